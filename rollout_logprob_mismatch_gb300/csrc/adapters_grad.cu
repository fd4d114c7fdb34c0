// adapters_grad.cu -- gradient of the low-rank adapters on a head's logits (sm_103a).
//
// For the logits' gradient dy [N, V], row i under adapter a, t_i = s_a A_a h_i:
//   dB_a = sum_i dy_i t_i^T        [V, R]
//   du_i = s_a B_a^T dy_i          [R]
//   dA_a = sum_i du_i h_i^T        [R, D]
//   dh_i (+)= A_a^T du_i           [D]
// dy is by far the largest operand and is read once: a CTA owns a slab of the vocabulary
// and walks all rows, adapter by adapter in steps of 16, so that dB's part of the slab
// stays in registers until the adapter's last row, and du of a step (the slab's part of
// the sum over V) goes to a partial array that a second launch folds in slab order.
// The eight warps split the slab's columns (mma.sync, bf16 operands, fp32 sums) and take
// turns to refill the ring of stages, with bulk copies of the rows' slabs and of t, after
// the one barrier of a step; a ninth warp for the copies would hold every thread to 168
// registers, too few for dB.  The adapter's factor comes by 16-byte asynchronous copies.
// Both products take the same tile from shared memory, dB with it transposed.  bf16 rows
// that start on 16 bytes are used as they land; others (fp16, fp32, odd rows) are first
// rewritten as one or two planes of bf16 parts: x = hi + lo leaves at most 2^-16 |x|.
// Every sum has one order, fixed by the rows' order and V: the same call gives the same bits.
#include <algorithm>
#include <type_traits>

#include "adapters.cuh"
#include "table_internal.h"

namespace tim {
namespace {

constexpr int WARPS = 8, STEP = AG_STEP;
constexpr int THREADS = WARPS * 32;

// Shared-memory layout and sizes of a variant.  RAW: stages hold rows as they are in
// memory (type T, any alignment) and are rewritten as planes; else they are bf16 rows.
template <typename T, bool RAW, int RP, int COLUMNS> struct Shape {
    static constexpr int COLS = COLUMNS;
    static constexpr int CW = COLS / WARPS;                    // columns of a warp
    static constexpr int PLANES = std::is_same<T, __nv_bfloat16>::value ? 1 : 2;
    static constexpr int ROW = COLS * static_cast<int>(sizeof(T)) + 16;   // bytes of a staged row
    static constexpr int PROW = COLS * 2 + 16;                 // bytes of a plane's row
    static constexpr int TROW = ag_t_pitch(RP == 64 ? 128 : RP) * 2;   // bytes of a row of t at most
    static constexpr int STAGE = STEP * (ROW + TROW);
    static constexpr int STAGES = 3;
    static constexpr int FROW = RP * 2 + 16;                   // bytes of a row of the factor
    static constexpr int FACTOR = COLS * FROW;
    static constexpr int RED = WARPS * STEP * (RP + 4) * 4;    // du's parts of the warps
    static constexpr int PLANE = RAW ? PLANES * STEP * PROW : 0;
    static constexpr int FIXED = PLANE + 2 * RED + 256;
    static constexpr int FACTORS = STAGES * STAGE + 2 * FACTOR + FIXED <= AG_SMEM ? 2 : 1;
    static constexpr int BYTES = STAGES * STAGE + FACTORS * FACTOR + FIXED;
    static_assert(BYTES <= AG_SMEM, "shared memory of a CTA");
    static_assert(STAGE % 16 == 0 && FACTOR % 16 == 0 && RED % 16 == 0 && PLANE % 16 == 0, "alignment");
};

__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t addr)
{
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
__device__ __forceinline__ void ldsm4t(uint32_t (&r)[4], uint32_t addr)
{
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}

// 16 bytes global -> shared (zeros where n = 0), counted by cp_async_arrive.
__device__ __forceinline__ void cp_async16(uint32_t dst, const void *src, uint32_t n)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(reinterpret_cast<uint64_t>(src)), "r"(n)
                 : "memory");
}
// One arrival on `bar` when this thread's asynchronous copies so far have landed.
__device__ __forceinline__ void cp_async_arrive(uint32_t bar)
{
    asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(bar) : "memory");
}

// The steps of a launch in order: STEP positions (fewer at an adapter's end) of one
// adapter.
struct Cursor {
    int ad, p, e;
    // the first step; false if there is none
    __device__ __forceinline__ bool start(const AdapterGradArgs &a)
    {
        ad = -1;
        return seek(a);
    }
    __device__ __forceinline__ bool seek(const AdapterGradArgs &a)   // the next adapter with positions
    {
        while (++ad < a.n) {
            p = max(a.plan.offsets[ad], a.p0);
            e = min(a.plan.offsets[ad + 1], a.p1);
            if (p < e)
                return true;
        }
        return false;
    }
    __device__ __forceinline__ bool skip(const AdapterGradArgs &a, int steps)
    {
        while (steps > 0) {
            const int here = (e - p + STEP - 1) / STEP;   // steps left of this adapter, this one included
            if (steps < here) {
                p += steps * STEP;
                return true;
            }
            steps -= here;
            if (!seek(a))
                return false;
        }
        return true;
    }
};

template <typename T, bool RAW, int RP, int COLUMNS>
__global__ void __launch_bounds__(THREADS, 1) adapters_grad_kernel(const AdapterGradArgs a)
{
    using S = Shape<T, RAW, RP, COLUMNS>;
    constexpr int CW = S::CW, MB = CW / 16, RB = RP / 8, PARTS = 2;
    extern __shared__ __align__(16) uint8_t smem[];
    const uint32_t base = smem_u32(smem);
    const uint32_t factor0 = base + S::STAGES * S::STAGE, plane0 = factor0 + S::FACTORS * S::FACTOR;
    uint8_t *red0 = smem + (plane0 - base) + S::PLANE;
    uint64_t *bars = reinterpret_cast<uint64_t *>(red0 + 2 * S::RED);
    const uint32_t bar0 = smem_u32(bars);
    auto full = [&](int i) { return bar0 + 8u * i; };
    auto ffull = [&](int i) { return bar0 + 8u * (S::STAGES + i); };
    volatile int *abort_flag = reinterpret_cast<volatile int *>(bars + S::STAGES + 2);

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, q = lane & 3;
    const int c0 = blockIdx.x * S::COLS, c1 = min(a.V, c0 + S::COLS);   // the slab's columns
    if (tid == 0) {
        for (int i = 0; i < S::STAGES; ++i)
            mbar_init(full(i), 1);
        for (int i = 0; i < 2; ++i)
            mbar_init(ffull(i), THREADS);
        *abort_flag = 0;
        fence_mbar_init();
    }
    if (!RAW) {
        // columns past the row's last whole 16 bytes are zeros: nothing below writes there
        // but a row's last elements
        const int whole = (c1 - c0) / 8 * 16;
        for (int i = tid; i < S::STAGES * STEP; i += THREADS)
            for (int b = whole; b < S::COLS * 2; b += 16)
                *reinterpret_cast<uint4 *>(smem + (i / STEP) * S::STAGE + (i % STEP) * S::ROW + b) = make_uint4(0u, 0u, 0u, 0u);
        fence_proxy_async_smem();
    }
    __syncthreads();
    pdl_wait();
    pdl_launch_dependents();
    const uint64_t budget = a.wait_budget_ns;
    const T *dy = static_cast<const T *>(a.dy);
    const uint32_t trow = static_cast<uint32_t>(ag_t_pitch(a.RT)) * 2;
    const uint64_t pol = l2_policy_evict_first(), pol_t = l2_policy_evict_last();

    // Each warp fills every eighth step, and has its next one's rows at hand.
    Cursor mine;
    bool more = mine.start(a) && mine.skip(a, warp);
    int row_of = 0;
    auto look_up = [&] {
        if (more && lane < min(STEP, mine.e - mine.p))
            row_of = a.plan.perm[mine.p + lane];
    };
    look_up();
    // One warp: bulk copies of its next step's rows and of their t into a stage.
    auto fill = [&](int stage) {
        const int rows = min(STEP, mine.e - mine.p);
        const uint32_t dst = base + stage * S::STAGE;
        RowCopy c{};
        uint8_t *st = smem + stage * S::STAGE + lane * S::ROW;
        if (lane < rows) {
            c = stage_row<T>(dy + static_cast<size_t>(row_of) * a.ld, c0, c1, a.V, st);
        } else if (lane < STEP && !RAW) {
            for (int k = 0; k < S::COLS * 2; k += 16)
                *reinterpret_cast<uint4 *>(st + k) = make_uint4(0u, 0u, 0u, 0u);
            fence_proxy_async_smem();
        }
        const uint32_t tbytes = static_cast<uint32_t>(rows) * trow;
        const uint32_t total = __reduce_add_sync(0xffffffffu, c.bytes) + tbytes;
        __syncwarp();
        if (lane == 0)
            mbar_arrive_expect_tx(full(stage), total);
        __syncwarp();
        if (c.bytes)
            bulk_load(dst + lane * S::ROW + c.off, c.src, c.bytes, full(stage), pol);
        if (lane == 0)
            bulk_load(dst + STEP * S::ROW, a.plan.t + static_cast<size_t>(mine.p) * (trow / 2), tbytes, full(stage), pol_t);
        more = mine.skip(a, WARPS);
        look_up();
    };
    // All threads: the slab of an adapter's factor, ranks r0 .. r0 + RP - 1, into buffer fb.
    auto load_factor = [&](int ad, int fb) {
        const uint16_t *B = a.B + static_cast<size_t>(ad) * a.V * a.R;
        for (int i = tid; i < S::COLS * (RP / 8); i += THREADS) {
            const int v = c0 + i / (RP / 8), r = a.r0 + i % (RP / 8) * 8;
            const bool on = v < a.V && r < a.R;
            cp_async16(factor0 + fb * S::FACTOR + (i / (RP / 8)) * S::FROW + (i % (RP / 8)) * 16,
                       B + static_cast<size_t>(on ? v : 0) * a.R + (on ? r : 0), on ? 16u : 0u);
        }
        cp_async_arrive(ffull(fb));
    };

    if (warp < S::STAGES && more)
        fill(warp);
    Cursor factors;   // the adapter whose factor is loaded next
    bool more_factors = factors.start(a);
    if (S::FACTORS == 2 && more_factors) {
        load_factor(factors.ad, 0);
        more_factors = factors.seek(a);
    }
    int stage = 0, fb = 0, rb = 0, turn = S::STAGES;   // turn: the warp that fills the next step
    uint32_t phase = 0, fphase = 0;
    // A wait that runs out sets the abort word and the status; the warps go on through
    // the same barriers (with what they find) and end.
    bool ok = true;
    const int w0 = warp * CW;   // the warp's columns in the slab
    for (int ad = 0; ad < a.n; ++ad) {
        const int ob = a.plan.offsets[ad], oe = a.plan.offsets[ad + 1];
        const int b = max(ob, a.p0), e = min(oe, a.p1);
        float db[MB][RB][4];
#pragma unroll
        for (int m = 0; m < MB; ++m)
#pragma unroll
            for (int r = 0; r < RB; ++r)
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    db[m][r][k] = 0.f;
        if (b < e) {
            // the other buffer's (or the only one's) last use is behind the last step's barrier
            if (S::FACTORS == 1) {
                load_factor(ad, 0);
            } else if (more_factors) {
                load_factor(factors.ad, fb ^ 1);
                more_factors = factors.seek(a);
            }
            if (ok)
                ok = mbar_wait_sleep(ffull(fb), fphase, abort_flag, budget);
        }
        for (int p = b; p < e; p += STEP) {
            if (ok)
                ok = mbar_wait_sleep(full(stage), phase, abort_flag, budget);
            const int rows = min(STEP, e - p);
            const uint32_t st = base + stage * S::STAGE, ts = st + STEP * S::ROW;
            uint32_t tile = st;
            if (RAW) {
                // 16 rows as planes of bf16 parts, eight columns at a time (the step before's
                // planes have been read: every warp has passed its barrier on du)
                for (int i = tid; i < STEP * (S::COLS / 8); i += THREADS) {
                    const int m = i / (S::COLS / 8), c = i % (S::COLS / 8) * 8;
                    uint32_t o[S::PLANES][4] = {};
                    if (m < rows && c0 + c < a.V) {
                        const uintptr_t lo = reinterpret_cast<uintptr_t>(dy + static_cast<size_t>(a.plan.perm[p + m]) * a.ld + c0);
                        const T *x = reinterpret_cast<const T *>(smem + stage * S::STAGE + m * S::ROW + (lo & 15)) + c;
#pragma unroll
                        for (int k = 0; k < 8; ++k) {
                            uint16_t part[S::PLANES];
                            split_bf16<S::PLANES>(c0 + c + k < a.V ? Elem<T>::load(x + k) : 0.f, part);
#pragma unroll
                            for (int i2 = 0; i2 < S::PLANES; ++i2)
                                o[i2][k >> 1] |= static_cast<uint32_t>(part[i2]) << ((k & 1) * 16);
                        }
                    }
#pragma unroll
                    for (int i2 = 0; i2 < S::PLANES; ++i2)
                        *reinterpret_cast<uint4 *>(smem + (plane0 - base) + (i2 * STEP + m) * S::PROW + c * 2) =
                            make_uint4(o[i2][0], o[i2][1], o[i2][2], o[i2][3]);
                }
                __syncthreads();
                tile = plane0;
            }
            constexpr int TPITCH = RAW ? S::PROW : S::ROW;
            // t's fragments: k = rows of the step, n = ranks.  Rows past the step's are
            // not in the stage: zeros
            uint32_t tf[PARTS][RB][2];
#pragma unroll
            for (int i = 0; i < PARTS; ++i)
#pragma unroll
                for (int r = 0; r < RB; r += 2) {
                    uint32_t x[4];
                    ldsm4t(x, ts + (lane & 15) * trow + (i * a.RT + a.r0 + r * 8 + (lane >> 4) * 8) * 2);
                    // a lane's two words hold rows 2q, 2q + 1 and 8 + 2q, 9 + 2q
                    const uint32_t k0 = (2 * q < rows ? 0xffffu : 0u) | (2 * q + 1 < rows ? 0xffff0000u : 0u);
                    const uint32_t k1 = (8 + 2 * q < rows ? 0xffffu : 0u) | (9 + 2 * q < rows ? 0xffff0000u : 0u);
                    tf[i][r][0] = x[0] & k0;
                    tf[i][r][1] = x[1] & k1;
                    tf[i][r + 1][0] = x[2] & k0;
                    tf[i][r + 1][1] = x[3] & k1;
                }
            float du[RB][4];
#pragma unroll
            for (int r = 0; r < RB; ++r)
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    du[r][k] = 0.f;
            const uint32_t fs = factor0 + fb * S::FACTOR;
#pragma unroll
            for (int m = 0; m < MB; ++m) {
                const int c = w0 + m * 16;
                uint32_t ff[RB][2];
#pragma unroll
                for (int r = 0; r < RB; r += 2) {
                    uint32_t x[4];
                    ldsm4t(x, fs + (c + (lane & 15)) * S::FROW + (r * 8 + (lane >> 4) * 8) * 2);
                    ff[r][0] = x[0];
                    ff[r][1] = x[1];
                    ff[r + 1][0] = x[2];
                    ff[r + 1][1] = x[3];
                }
#pragma unroll
                for (int i = 0; i < S::PLANES; ++i) {
                    const uint32_t pl = tile + i * (STEP * S::PROW);
                    uint32_t x[4];
                    // columns as rows: dB's operand
                    ldsm4t(x, pl + ((lane & 7) + (lane >> 4) * 8) * TPITCH + (c + ((lane >> 3) & 1) * 8) * 2);
#pragma unroll
                    for (int r = 0; r < RB; ++r) {
                        mma16816(db[m][r], x, tf[0][r][0], tf[0][r][1]);
                        if (i == 0)   // lo lo is of the size of what the parts leave
                            mma16816(db[m][r], x, tf[1][r][0], tf[1][r][1]);
                    }
                    ldsm4(x, pl + (lane & 15) * TPITCH + (c + (lane >> 4) * 8) * 2);
#pragma unroll
                    for (int r = 0; r < RB; ++r)
                        mma16816(du[r], x, ff[r][0], ff[r][1]);
                }
            }
            float *red = reinterpret_cast<float *>(red0 + rb * S::RED);
#pragma unroll
            for (int r = 0; r < RB; ++r) {
                *reinterpret_cast<float2 *>(red + (warp * STEP + g) * (RP + 4) + r * 8 + 2 * q) = make_float2(du[r][0], du[r][1]);
                *reinterpret_cast<float2 *>(red + (warp * STEP + g + 8) * (RP + 4) + r * 8 + 2 * q) = make_float2(du[r][2], du[r][3]);
            }
            __syncthreads();   // du's parts are there; the stage, and in an adapter's last step the factor, have been read
            if (warp == turn && more && ok)
                fill(stage);
            turn = turn + 1 == WARPS ? 0 : turn + 1;
            float *part = a.partial + (static_cast<size_t>(blockIdx.x) * (a.p1 - a.p0) + (p - a.p0)) * RP;
            for (int i = tid; i < rows * (RP / 4); i += THREADS) {
                const int m = i / (RP / 4), r = i % (RP / 4) * 4;
                float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
                for (int w = 0; w < WARPS; ++w) {
                    const float4 x = *reinterpret_cast<const float4 *>(red + (w * STEP + m) * (RP + 4) + r);
                    s.x += x.x;
                    s.y += x.y;
                    s.z += x.z;
                    s.w += x.w;
                }
                *reinterpret_cast<float4 *>(part + static_cast<size_t>(m) * RP + r) = s;
            }
            rb ^= 1;
            if (++stage == S::STAGES) {
                stage = 0;
                phase ^= 1u;
            }
        }
        if (b < e && ++fb == S::FACTORS) {
            fb = 0;
            fphase ^= 1u;
        }
        // an adapter whose rows began in an earlier part of the batch is added to; one
        // without rows is written (zeros) by the first part
        const bool add = a.accumulate || (ob < oe && ob < a.p0);
        if (b < e || (ob == oe && a.p0 == 0 && !a.accumulate)) {
            float *dB = a.dB + static_cast<size_t>(ad) * a.V * a.R;
#pragma unroll
            for (int m = 0; m < MB; ++m)
#pragma unroll
                for (int half = 0; half < 2; ++half) {
                    const int v = c0 + w0 + m * 16 + half * 8 + g;
                    if (v >= a.V)
                        continue;
#pragma unroll
                    for (int r = 0; r < RB; ++r) {
                        const int rr = a.r0 + r * 8 + 2 * q;
                        if (rr >= a.R)
                            continue;
                        float2 *p = reinterpret_cast<float2 *>(dB + static_cast<size_t>(v) * a.R + rr);
                        float2 x = make_float2(db[m][r][half * 2], db[m][r][half * 2 + 1]);
                        if (add) {
                            const float2 y = *p;
                            x.x += y.x;
                            x.y += y.y;
                        }
                        *p = x;
                    }
                }
        }
    }
    __syncthreads();
    if (*abort_flag) {   // copies may still be on their way
        asm volatile("cp.async.wait_all;" ::: "memory");
        if (tid == 0) {
            for (int i = 0; i < S::STAGES; ++i)
                drain_wait(full(i), i < stage ? phase : phase ^ 1u);
            atomicCAS(a.status, 0, static_cast<int>(TIM_ERR_TIMEOUT));
        }
        __syncthreads();
    }
}

// ---------------------------------------------------------------- fold
// du of positions p0 .. p1 - 1, ranks r0 .. r0 + RP - 1: the slabs' parts added in slab
// order by eight threads (slabs k, k + 8, ... each, then joined in order), times scale,
// in three bf16 parts.
template <int RP> __global__ void __launch_bounds__(256) adapters_fold_kernel(const AdapterGradArgs a)
{
    constexpr int SHARE = 8, ITEMS = 256 / SHARE;
    __shared__ float4 sums[SHARE][ITEMS];
    const int item = threadIdx.x % ITEMS, k = threadIdx.x / ITEMS;
    const int64_t count = a.p1 - a.p0;
    const int64_t i = (static_cast<int64_t>(blockIdx.x) * ITEMS + item);   // four ranks of a position
    pdl_wait();
    pdl_launch_dependents();
    const bool on = i < count * (RP / 4);
    float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
    if (on) {
        const float4 *p = reinterpret_cast<const float4 *>(a.partial) + i;
#pragma unroll 4
        for (int slab = k; slab < a.slabs; slab += SHARE) {
            const float4 x = p[slab * (count * (RP / 4))];
            s.x += x.x;
            s.y += x.y;
            s.z += x.z;
            s.w += x.w;
        }
    }
    sums[k][item] = s;
    __syncthreads();
    if (k != 0 || !on)
        return;
#pragma unroll
    for (int j = 1; j < SHARE; ++j) {
        const float4 x = sums[j][item];
        s.x += x.x;
        s.y += x.y;
        s.z += x.z;
        s.w += x.w;
    }
    const int pos = a.p0 + static_cast<int>(i / (RP / 4)), r = static_cast<int>(i % (RP / 4)) * 4;
    const int ad = a.plan.adapter[pos];
    if (ad >= a.n)
        return;   // no adapter: nothing was summed
    const float scale = a.scale ? a.scale[ad] : 1.f;
    uint16_t x0[3], x1[3], x2[3], x3[3];
    split_bf16<3>(s.x * scale, x0);
    split_bf16<3>(s.y * scale, x1);
    split_bf16<3>(s.z * scale, x2);
    split_bf16<3>(s.w * scale, x3);
    uint16_t *du = a.du + static_cast<size_t>(pos) * (3 * a.RT) + a.r0 + r;
#pragma unroll
    for (int j = 0; j < 3; ++j)
        *reinterpret_cast<uint2 *>(du + j * a.RT) =
            make_uint2(x0[j] | static_cast<uint32_t>(x1[j]) << 16, x2[j] | static_cast<uint32_t>(x3[j]) << 16);
}

// ---------------------------------------------------------------- dA
// CTA (x, a): dA of adapter a, columns x * 128 .. + 127 of D; a warp has 16 of them for
// all ranks.  Rows in chunks of 32 through shared memory (gathered in the plan's order).
template <int RT> __global__ void __launch_bounds__(256) adapters_dA_kernel(const AdapterGradArgs a)
{
    constexpr int ROWS = 32, COLS = 128, HROW = COLS * 2 + 16, UROW = 3 * RT * 2 + 16, RM = RT / 16;
    __shared__ __align__(16) uint8_t hs[ROWS * HROW], us[ROWS * UROW];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, q = lane & 3;
    const int ad = blockIdx.y, d0 = blockIdx.x * COLS;
    pdl_wait();
    pdl_launch_dependents();
    const int b = a.plan.offsets[ad], e = a.plan.offsets[ad + 1];
    if (b == e && a.accumulate)
        return;
    float acc[RM][2][4] = {};
    const uint32_t h0 = smem_u32(hs), u0 = smem_u32(us);
    const uint4 zero = make_uint4(0u, 0u, 0u, 0u);
    for (int p = b; p < e; p += ROWS) {
        __syncthreads();
        for (int i = tid; i < ROWS * (COLS / 8); i += 256) {
            const int m = i / (COLS / 8), c = i % (COLS / 8) * 8;
            const bool on = p + m < e && d0 + c < a.D;
            *reinterpret_cast<uint4 *>(hs + m * HROW + c * 2) =
                on ? __ldg(reinterpret_cast<const uint4 *>(a.h + static_cast<size_t>(a.plan.perm[p + m]) * a.D + d0 + c)) : zero;
        }
        for (int i = tid; i < ROWS * (3 * RT / 8); i += 256) {
            const int m = i / (3 * RT / 8), c = i % (3 * RT / 8) * 8;
            *reinterpret_cast<uint4 *>(us + m * UROW + c * 2) =
                p + m < e ? *reinterpret_cast<const uint4 *>(a.du + static_cast<size_t>(p + m) * (3 * RT) + c) : zero;
        }
        __syncthreads();
#pragma unroll
        for (int k = 0; k < ROWS; k += 16) {
            uint32_t x[4];   // k = rows, n = the warp's 16 columns
            ldsm4t(x, h0 + (k + (lane & 15)) * HROW + (warp * 16 + (lane >> 4) * 8) * 2);
#pragma unroll
            for (int i = 0; i < 3; ++i)
#pragma unroll
                for (int m = 0; m < RM; ++m) {
                    uint32_t u[4];   // ranks as rows
                    ldsm4t(u, u0 + (k + (lane & 7) + (lane >> 4) * 8) * UROW + (i * RT + m * 16 + ((lane >> 3) & 1) * 8) * 2);
                    mma16816(acc[m][0], u, x[0], x[1]);
                    mma16816(acc[m][1], u, x[2], x[3]);
                }
        }
    }
#pragma unroll
    for (int m = 0; m < RM; ++m)
#pragma unroll
        for (int half = 0; half < 2; ++half) {
            const int r = m * 16 + half * 8 + g;
            if (r >= a.R)
                continue;
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const int d = d0 + warp * 16 + j * 8 + 2 * q;
                if (d >= a.D)
                    continue;
                float2 *o = reinterpret_cast<float2 *>(a.dA + (static_cast<size_t>(ad) * a.R + r) * a.D + d);
                float2 x = make_float2(acc[m][j][half * 2], acc[m][j][half * 2 + 1]);
                if (a.accumulate) {
                    const float2 y = *o;
                    x.x += y.x;
                    x.y += y.y;
                }
                *o = x;
            }
        }
}

// ---------------------------------------------------------------- dh
// CTA (x, y): columns x * 256 .. + 255 of D (a warp 32) of positions y * chunk ...; the
// adapter's A slab is in shared memory while the rows' adapter is the same.
template <int RT> __global__ void __launch_bounds__(256) adapters_dh_kernel(const AdapterGradArgs a)
{
    constexpr int COLS = 256, AROW = COLS * 2 + 16, KS = RT / 16;
    extern __shared__ __align__(16) uint8_t as[];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, q = lane & 3;
    const int d0 = blockIdx.x * COLS, dw = d0 + warp * 32;
    pdl_wait();
    pdl_launch_dependents();
    const int live = a.plan.offsets[a.n];
    const int p0 = blockIdx.y * a.row_chunk, p1 = min(a.N, p0 + a.row_chunk);
    const uint32_t a0 = smem_u32(as);
    for (int p = p0; p < min(p1, live);) {   // adapter by adapter
        const int ad = a.plan.adapter[p];
        const int e = min(p1, a.plan.offsets[ad + 1]);
        __syncthreads();
        for (int i = tid; i < RT * (COLS / 8); i += 256) {
            const int r = i / (COLS / 8), c = i % (COLS / 8) * 8;
            const bool on = r < a.R && d0 + c < a.D;
            *reinterpret_cast<uint4 *>(as + r * AROW + c * 2) =
                on ? __ldg(reinterpret_cast<const uint4 *>(a.A + (static_cast<size_t>(ad) * a.R + r) * a.D + d0 + c))
                   : make_uint4(0u, 0u, 0u, 0u);
        }
        __syncthreads();
        for (; p < e; p += 16) {
            const bool on0 = p + g < e, on1 = p + g + 8 < e;
            float acc[4][4] = {};
            const uint16_t *u = a.du + static_cast<size_t>(p + g) * (3 * RT);
#pragma unroll 1
            for (int i = 0; i < 3; ++i)
#pragma unroll
                for (int k = 0; k < KS; ++k) {
                    const int r = i * RT + k * 16 + 2 * q;
                    uint32_t x[4];
                    x[0] = on0 ? *reinterpret_cast<const uint32_t *>(u + r) : 0u;
                    x[1] = on1 ? *reinterpret_cast<const uint32_t *>(u + 8 * (3 * RT) + r) : 0u;
                    x[2] = on0 ? *reinterpret_cast<const uint32_t *>(u + r + 8) : 0u;
                    x[3] = on1 ? *reinterpret_cast<const uint32_t *>(u + 8 * (3 * RT) + r + 8) : 0u;
#pragma unroll
                    for (int j = 0; j < 4; j += 2) {
                        uint32_t w[4];
                        ldsm4t(w, a0 + (k * 16 + (lane & 15)) * AROW + (warp * 32 + j * 8 + (lane >> 4) * 8) * 2);
                        mma16816(acc[j], x, w[0], w[1]);
                        mma16816(acc[j + 1], x, w[2], w[3]);
                    }
                }
#pragma unroll
            for (int half = 0; half < 2; ++half) {
                if (!(half ? on1 : on0))
                    continue;
                float *row = a.dh + static_cast<size_t>(a.plan.perm[p + g + half * 8]) * a.D;
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const int d = dw + j * 8 + 2 * q;
                    if (d >= a.D)
                        continue;
                    float2 *o = reinterpret_cast<float2 *>(row + d);
                    float2 x = make_float2(acc[j][half * 2], acc[j][half * 2 + 1]);
                    if (a.accumulate_dh) {
                        const float2 y = *o;
                        x.x += y.x;
                        x.y += y.y;
                    }
                    *o = x;
                }
            }
        }
        p = e;
    }
    if (a.accumulate_dh)
        return;
    // rows under no adapter
    for (int z = max(p0, live) + warp; z < p1; z += 8) {
        float *row = a.dh + static_cast<size_t>(a.plan.perm[z]) * a.D;
        for (int c = lane * 4; c < COLS; c += 128)
            if (d0 + c < a.D)
                *reinterpret_cast<float4 *>(row + d0 + c) = make_float4(0.f, 0.f, 0.f, 0.f);
    }
}

template <typename F>
cudaError_t launch(F kernel, dim3 grid, int threads, int smem, const AdapterGradArgs &a, cudaStream_t s)
{
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1] = {pdl_attribute()};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads, 1, 1);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, a);
}

template <typename T, bool RAW, int RP, int COLS> cudaError_t grad(const AdapterGradArgs &a, cudaStream_t s, bool set)
{
    using S = Shape<T, RAW, RP, COLS>;
    if (set)
        return cudaFuncSetAttribute(adapters_grad_kernel<T, RAW, RP, COLS>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                    S::BYTES);
    return launch(adapters_grad_kernel<T, RAW, RP, COLS>, dim3(static_cast<unsigned>(a.slabs)), THREADS, S::BYTES, a, s);
}

// The variant for the slab's width; set: its shared memory is granted instead.
template <typename T, bool RAW, int RP> cudaError_t grad(const AdapterGradArgs &a, int cols, cudaStream_t s, bool set)
{
    constexpr int WIDE = ag_cols(RP, RAW, true), NARROW = ag_cols(RP, RAW, false);
    return cols == WIDE ? grad<T, RAW, RP, WIDE>(a, s, set) : grad<T, RAW, RP, NARROW>(a, s, set);
}

template <int RP>
cudaError_t grad(const AdapterGradArgs &a, int dtype, bool raw, int cols, cudaStream_t s, bool set = false)
{
    if (dtype == TIM_F32)
        return grad<float, true, RP>(a, cols, s, set);
    if (dtype == TIM_F16)
        return grad<__half, true, RP>(a, cols, s, set);
    return raw ? grad<__nv_bfloat16, true, RP>(a, cols, s, set) : grad<__nv_bfloat16, false, RP>(a, cols, s, set);
}

template <int RP> cudaError_t prepare()
{
    const AdapterGradArgs a{};
    cudaError_t e = cudaSuccess;
    for (int wide = 0; wide < 2; ++wide) {
        for (int dtype : {TIM_F32, TIM_F16, TIM_BF16})
            if (e == cudaSuccess)
                e = grad<RP>(a, dtype, true, ag_cols(RP, true, wide), nullptr, true);
        if (e == cudaSuccess)
            e = grad<RP>(a, TIM_BF16, false, ag_cols(RP, false, wide), nullptr, true);
    }
    return e;
}

} // namespace

cudaError_t adapters_grad_prepare_device()
{
    cudaError_t e = prepare<16>();
    if (e == cudaSuccess)
        e = prepare<32>();
    if (e == cudaSuccess)
        e = prepare<64>();
    if (e == cudaSuccess)
        e = cudaFuncSetAttribute(adapters_dh_kernel<128>, cudaFuncAttributeMaxDynamicSharedMemorySize, 128 * 528);
    return e;
}

cudaError_t adapters_grad_launch(AdapterGradArgs a, int dtype, cudaStream_t s)
{
    const int RP = std::min(a.RT, 64);
    for (int64_t p0 = 0; p0 < a.N; p0 += a.row_part)
        for (a.r0 = 0; a.r0 < a.R; a.r0 += RP) {
            a.p0 = static_cast<int32_t>(p0);
            a.p1 = static_cast<int32_t>(std::min<int64_t>(a.N, p0 + a.row_part));
            cudaError_t e = RP == 16   ? grad<16>(a, dtype, a.raw, a.cols, s)
                            : RP == 32 ? grad<32>(a, dtype, a.raw, a.cols, s)
                                       : grad<64>(a, dtype, a.raw, a.cols, s);
            if (e != cudaSuccess)
                return e;
            const int64_t items = static_cast<int64_t>(a.p1 - a.p0) * (RP / 4);
            const dim3 grid(static_cast<unsigned>((items + 31) / 32));
            e = RP == 16   ? launch(adapters_fold_kernel<16>, grid, 256, 0, a, s)
                : RP == 32 ? launch(adapters_fold_kernel<32>, grid, 256, 0, a, s)
                           : launch(adapters_fold_kernel<64>, grid, 256, 0, a, s);
            if (e != cudaSuccess)
                return e;
        }
    const dim3 grid_a(static_cast<unsigned>((a.D + 127) / 128), static_cast<unsigned>(a.n));
    int64_t chunk = 128;
    while ((a.N + chunk - 1) / chunk > 65535)
        chunk *= 2;
    a.row_chunk = static_cast<int32_t>(chunk);
    const dim3 grid_h(static_cast<unsigned>((a.D + 255) / 256), static_cast<unsigned>((a.N + chunk - 1) / chunk));
    const int smem = a.RT * 528;
    cudaError_t e;
    switch (a.RT) {
    case 16:
        e = launch(adapters_dA_kernel<16>, grid_a, 256, 0, a, s);
        return e != cudaSuccess ? e : launch(adapters_dh_kernel<16>, grid_h, 256, smem, a, s);
    case 32:
        e = launch(adapters_dA_kernel<32>, grid_a, 256, 0, a, s);
        return e != cudaSuccess ? e : launch(adapters_dh_kernel<32>, grid_h, 256, smem, a, s);
    case 64:
        e = launch(adapters_dA_kernel<64>, grid_a, 256, 0, a, s);
        return e != cudaSuccess ? e : launch(adapters_dh_kernel<64>, grid_h, 256, smem, a, s);
    default:
        e = launch(adapters_dA_kernel<128>, grid_a, 256, 0, a, s);
        return e != cudaSuccess ? e : launch(adapters_dh_kernel<128>, grid_h, 256, smem, a, s);
    }
}

} // namespace tim
