// adapters.cu -- low-rank adapters of many requests beside the shared head (sm_103a).
//
// y_n = z_n + s_a B_a (A_a h_n), a = the adapter of row n: z are the shared head's
// logits, A_a [R, D] and B_a [V, R] the adapter's factors.  Two launches:
//   shrink  orders the rows by adapter (a CTA counts the ids below its own and takes
//           its own in order: no counter to clear, no atomics, the same order every
//           time) and writes t_n = s_a A_a h_n in bf16 parts; two launches for many rows;
//   map     y = z + t B^T, one pass over the logits.
// A row's products are formed with its own adapter's factors only: where a tile of 16
// rows meets several adapters, the tile is multiplied with each and every row keeps its
// own (masking t to zero instead would let an infinite or NaN factor of one tenant
// reach another's rows).
#include <algorithm>

#include "adapters.cuh"
#include "table_internal.h"
#include "tim_internal.h"

namespace tim {
namespace {

// ---------------------------------------------------------------- shrink
constexpr int WARPS = 16;   // of a CTA that orders or projects

// Calls f(row, position among the adapter's rows) for those of the warp's rows
// [r0, r1) that are under adapter `ad`, in order, `before` of them already counted.
template <typename F>
__device__ __forceinline__ void own_rows(const AdapterArgs &a, int ad, int r0, int r1, int before, F f)
{
    const int lane = threadIdx.x & 31;
#pragma unroll 4
    for (int r = r0; r < r1; r += 32) {
        const int id = r + lane < r1 ? a.rows[r + lane] : 0;
        const bool in = r + lane < r1 && (static_cast<unsigned>(id) < static_cast<unsigned>(a.n) ? id : a.n) == ad;
        const unsigned all = __ballot_sync(0xffffffffu, in);
        if (in)
            f(r + lane, before + __popc(all & ((1u << lane) - 1u)));
        before += __popc(all);
    }
}

// The warp's part [r0, r1) of the list of ids, and what lies before the rows of adapter
// ad: the rows of lower adapters (base), in all (count), in the warps before (before).
struct Own {
    int r0, r1, own, base, count, before;
};

__device__ __forceinline__ Own count_rows(const AdapterArgs &a, int ad)
{
    __shared__ int sb[WARPS], so[WARPS];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int per = ((a.N + 31) / 32 + WARPS - 1) / WARPS * 32;
    Own o;
    o.r0 = min(a.N, warp * per);
    o.r1 = min(a.N, o.r0 + per);
    int below = 0, own = 0;
#pragma unroll 8
    for (int r = o.r0 + lane; r < o.r1; r += 32) {
        int id = a.rows[r];
        id = static_cast<unsigned>(id) < static_cast<unsigned>(a.n) ? id : a.n;
        below += id < ad;
        own += id == ad;
    }
    below = __reduce_add_sync(0xffffffffu, below);
    own = __reduce_add_sync(0xffffffffu, own);
    if (lane == 0) {
        sb[warp] = below;
        so[warp] = own;
    }
    __syncthreads();
    o.own = own;
    o.base = o.count = o.before = 0;
#pragma unroll
    for (int w = 0; w < WARPS; ++w) {
        o.base += sb[w];
        o.count += so[w];
        o.before += w < warp ? so[w] : 0;
    }
    return o;
}

__device__ __forceinline__ void write_order(const AdapterArgs &a, int ad, const Own &o)
{
    TIM_DCHECK(o.base + o.count <= a.N && (ad < a.n || o.base + o.count == a.N), a.status, TIM_CHECK_UNIT, ad, o.base);
    if (threadIdx.x == 0) {
        a.plan.offsets[ad] = o.base;
        if (ad == a.n)
            a.plan.offsets[ad + 1] = a.N;
    }
    if (o.own > 0)
        own_rows(a, ad, o.r0, o.r1, o.base + o.before, [&](int r, int p) {
            TIM_DCHECK(p < o.base + o.count, a.status, TIM_CHECK_STORE, p, r);
            a.plan.perm[p] = r;
            a.plan.adapter[p] = ad;
        });
}

// t of up to 16 rows under adapter ad, written for rows lo .. hi - 1 of them at positions
// pos + lo ..  k is shared among the 16 warps (every 16th 32 of it each), whose sums are added up through shared memory in their order, so that a row's sum
// depends on D alone.  AHEAD: steps of 32 k whose loads are in flight together.
template <int RP, int PARTS, int AHEAD>
__device__ __forceinline__ void project(const AdapterArgs &a, int ad, const int32_t *rows, int lo, int hi, int pos)
{
    constexpr int NC = RP < 32 ? RP : 32;      // rank columns at a time
    __shared__ float sums[WARPS][16][NC + 1];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, q = lane & 3;
    const float scale = a.scale ? a.scale[ad] : 1.f;
    const uint16_t *A = a.A + static_cast<size_t>(ad) * a.R * a.D;
    const int kchunks = (a.D + 31) / 32;
    const uint4 zero = make_uint4(0u, 0u, 0u, 0u);
    const bool on0 = g >= lo && g < hi, on1 = g + 8 >= lo && g + 8 < hi;
    TIM_DCHECK((!on0 || static_cast<unsigned>(rows[g]) < static_cast<unsigned>(a.N)) &&
                   (!on1 || static_cast<unsigned>(rows[g + 8]) < static_cast<unsigned>(a.N)),
               a.status, TIM_CHECK_UNIT, pos + g, ad);
    TIM_DCHECK(static_cast<unsigned>(ad) < static_cast<unsigned>(a.n) && pos + hi <= a.N, a.status, TIM_CHECK_STORE, pos, ad);
    const uint16_t *h0 = a.h + static_cast<size_t>(on0 ? rows[g] : 0) * a.D;
    const uint16_t *h1 = a.h + static_cast<size_t>(on1 ? rows[g + 8] : 0) * a.D;
    for (int n0 = 0; n0 < RP; n0 += NC) {
        float acc[NC / 8][4] = {};
        if (n0 < a.R) {
            for (int kc0 = warp; kc0 < kchunks; kc0 += WARPS * AHEAD) {
                uint4 x0[AHEAD], x1[AHEAD], w[AHEAD][NC / 8];
#pragma unroll
                for (int i = 0; i < AHEAD; ++i) {
                    const int k = (kc0 + i * WARPS) * 32 + q * 8;   // D is a multiple of 8: the eight are in or out together
                    const bool in = k < a.D;
                    x0[i] = in && on0 ? __ldg(reinterpret_cast<const uint4 *>(h0 + k)) : zero;
                    x1[i] = in && on1 ? __ldg(reinterpret_cast<const uint4 *>(h1 + k)) : zero;
#pragma unroll
                    for (int j = 0; j < NC / 8; ++j) {
                        const int r = n0 + j * 8 + g;
                        w[i][j] = in && r < a.R ? __ldg(reinterpret_cast<const uint4 *>(A + static_cast<size_t>(r) * a.D + k)) : zero;
                    }
                }
#pragma unroll
                for (int i = 0; i < AHEAD; ++i)
#pragma unroll
                    for (int j = 0; j < NC / 8; ++j) {
                        // 32 k by themselves, then added: the tensor cores cut, rather than round, what they add up
                        float part[4] = {};
                        mma16816(part, {x0[i].x, x1[i].x, x0[i].y, x1[i].y}, w[i][j].x, w[i][j].y);
                        mma16816(part, {x0[i].z, x1[i].z, x0[i].w, x1[i].w}, w[i][j].z, w[i][j].w);
#pragma unroll
                        for (int k = 0; k < 4; ++k)
                            acc[j][k] += part[k];
                    }
            }
        }
        __syncthreads();   // the sums before have been read
#pragma unroll
        for (int j = 0; j < NC / 8; ++j) {
            float (&to)[16][NC + 1] = sums[warp];
            to[g][j * 8 + 2 * q] = acc[j][0];
            to[g][j * 8 + 2 * q + 1] = acc[j][1];
            to[g + 8][j * 8 + 2 * q] = acc[j][2];
            to[g + 8][j * 8 + 2 * q + 1] = acc[j][3];
        }
        __syncthreads();
        for (int i = tid; i < (hi - lo) * NC; i += WARPS * 32) {
            const int m = lo + i / NC, r = i % NC;
            float u = 0.f;
#pragma unroll
            for (int w = 0; w < WARPS; ++w)
                u += sums[w][m][r];
            uint16_t p[PARTS];
            split_bf16<PARTS>(u * scale, p);
            uint16_t *t = a.plan.t + (static_cast<size_t>(pos) + static_cast<size_t>(ad) * a.plan.t_pad + m) * a.plan.t_pitch + n0 + r;
#pragma unroll
            for (int k = 0; k < PARTS; ++k)
                t[k * RP] = p[k];
        }
    }
}

// The zeros behind the last of an adapter's `count` rows, whose positions end at `end`.
__device__ __forceinline__ void pad_rows(const AdapterArgs &a, int ad, int count, int end)
{
    if (a.plan.t_pad == 0)
        return;
    const int words = (-count & (AG_PAD - 1)) * (a.plan.t_pitch / 2);
    TIM_DCHECK(end <= a.N, a.status, TIM_CHECK_STORE, end, ad);
    uint32_t *t = reinterpret_cast<uint32_t *>(a.plan.t + (static_cast<size_t>(end) + static_cast<size_t>(ad) * a.plan.t_pad) * a.plan.t_pitch);
    for (int i = threadIdx.x; i < words; i += blockDim.x)
        t[i] = 0u;
}

// Few rows, one launch: a chain of loads (ids, rows, their products), 11 us for 64 rows of 4096 under
// 32 adapters of rank 16, 4.0 MB.  CTA (a, y): the rows of adapter a, 16 at a time from the y-th 16
// on; a = n: the rows under no adapter (only ordered).
template <int RP, int PARTS>
__global__ void __launch_bounds__(512, 1) adapters_shrink_kernel(const AdapterArgs a)
{
    __shared__ int32_t mine[16];
    const int ad = blockIdx.x;
    pdl_wait();
    pdl_launch_dependents();
    const Own o = count_rows(a, ad);
    if (blockIdx.y == 0)
        write_order(a, ad, o);
    if (ad == a.n)
        return;
    for (int c0 = blockIdx.y * 16; c0 < o.count; c0 += gridDim.y * 16) {
        const int rows = min(16, o.count - c0);
        if (o.own > 0 && o.before < c0 + rows && o.before + o.own > c0)
            own_rows(a, ad, o.r0, o.r1, o.before, [&](int r, int p) {
                if (p >= c0 && p < c0 + rows)
                    mine[p - c0] = r;
            });
        __syncthreads();
        project<RP, PARTS, RP == 16 ? 4 : 3>(a, ad, mine, 0, rows, o.base + c0);
        if (c0 + rows == o.count)
            pad_rows(a, ad, o.count, o.base + o.count);
        __syncthreads();
    }
}

// Many rows: the order in a launch of its own (8192 rows 6 us), then a CTA for every 16 positions:
// two an SM where there are that many (8192 rows of rank 16: whole call on 8192 columns 99 us, 104 with one
// an SM; at rank 64 one would win, 246 for 283), else one with more loads in flight (1000 rows of
// rank 64: 68 us, 104 with two).  8192 x 4096, rank 16, 25 us (h read at 2.7 TB/s; the factors come from
// L2 for every 16 rows).
__global__ void __launch_bounds__(512) adapters_order_kernel(const AdapterArgs a)
{
    pdl_wait();
    pdl_launch_dependents();
    const Own o = count_rows(a, blockIdx.x);
    write_order(a, blockIdx.x, o);
}

template <int RP, int PARTS, bool MANY>
__global__ void __launch_bounds__(512, MANY ? 2 : 1) adapters_project_kernel(const AdapterArgs a)
{
    __shared__ int32_t s_row[16], s_ad[17];
    pdl_wait();
    pdl_launch_dependents();
    const int p0 = blockIdx.x * 16, rows = min(16, a.plan.offsets[a.n] - p0);
    if (rows <= 0)
        return;
    if (threadIdx.x < rows) {
        s_row[threadIdx.x] = a.plan.perm[p0 + threadIdx.x];
        s_ad[threadIdx.x] = a.plan.adapter[p0 + threadIdx.x];
    }
    if (threadIdx.x == 0)
        s_ad[rows] = -1;
    __syncthreads();
    for (int s = 0; s < rows;) {
        int m = s + 1;
        while (s_ad[m] == s_ad[s])
            ++m;
        project<RP, PARTS, MANY ? (RP == 16 ? 2 : 1) : 4>(a, s_ad[s], s_row, s, m, p0);
        const int ad = s_ad[s], e = a.plan.offsets[ad + 1];
        if (p0 + m == e)
            pad_rows(a, ad, e - a.plan.offsets[ad], e);
        s = m;
    }
}

// ---------------------------------------------------------------- map
// Eight columns of a row from a quad's lane q: 32 columns from col - 8 q on in all;
// stores aligned 16-byte pieces whatever the row's alignment (the tail of one lane's
// columns goes to the next lane of the quad).  The whole warp calls it; on = the lane's
// row and columns exist, any = some row of the warp is not aligned.
template <typename T>
__device__ __forceinline__ void store_quad(T *row, int col, int V, const Raw8<T> &r, bool on, bool any)
{
    constexpr int W = Elem<T>::WORDS;
    const uint32_t shift = row_shift(row);
    const int q = threadIdx.x & 3;
    uint32_t w[W + 4], o[W];
    if (any) {
#pragma unroll
        for (int k = 0; k < 4; ++k)
            w[k] = __shfl_up_sync(0xffffffffu, r.w[W - 4 + k], 1, 4);
#pragma unroll
        for (int k = 0; k < W; ++k)
            w[4 + k] = r.w[k];
        shift_words<W, sizeof(T) == 2>(o, w, 16 - shift);
    }
    if (!on)
        return;
    if (shift == 0 ? col + 8 > V : col - 8 * q + 32 > V) {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (col + i < V)
                store1(row, col, r, i);
        return;
    }
    uint4 *p = reinterpret_cast<uint4 *>(reinterpret_cast<char *>(row + col) - shift);
    if (shift == 0) {
#pragma unroll
        for (int k = 0; k < W / 4; ++k)
            p[k] = make_uint4(r.w[4 * k], r.w[4 * k + 1], r.w[4 * k + 2], r.w[4 * k + 3]);
        return;
    }
    const int head = static_cast<int>((16 - shift) / sizeof(T));   // own elements in the first piece
    if (q != 0)
        p[0] = make_uint4(o[0], o[1], o[2], o[3]);
    if constexpr (W == 8)
        p[1] = make_uint4(o[4], o[5], o[6], o[7]);
    if (q == 0) {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (i < head)
                store1(row, col, r, i);
    }
    if (q == 3) {
        const int tail = static_cast<int>(shift / sizeof(T));
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (i >= 8 - tail)
                store1(row, col, r, i);
    }
}

// k groups of a lane: 32 ranks in 16 bytes (two products), or all 16 ranks in 8.
template <int RP> struct Ranks {
    static constexpr int STEP = RP == 16 ? 4 : 8;        // neighbouring ranks of a lane
    static constexpr int GROUPS = RP == 16 ? 1 : RP / 32;
    static constexpr int WORDS = STEP / 2;
    // A warp keeps its part of a factor in registers, so that the buffer is free at once (256 x 151936
    // bf16, rank 32 of 64: 154 us, 167 without).  At rank 16 it takes the room of the wide form
    // (8192 x 151936: 1190 us, 906 without) and gains nothing in the narrow one for bf16 (64 x 128256 of
    // 32: 54 us either way; 2048 x 151936 fp32 420 for 430); at 64 it gains 1 %; at 128 there is no room.
    static constexpr bool HELD = RP == 32;
};

template <int WORDS> __device__ __forceinline__ void lds_words(uint32_t (&w)[4], uint32_t addr)
{
    if constexpr (WORDS == 2) {
        asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(w[0]), "=r"(w[1]) : "r"(addr));
        w[2] = w[3] = 0u;
    } else {
        asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                     : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3])
                     : "r"(addr));
    }
}

// Shared memory of a CTA of the map: a ring of tiles (16 rows of the slab and their t),
// and one of the slabs of adapters' factors.
template <typename T, int RP, int PARTS, int CB> struct MapShape {
    static constexpr int COLS = 256 * CB;                              // columns of a slab
    static constexpr int ROW = COLS * static_cast<int>(sizeof(T)) + 64;   // bytes of a staged row: a warp's 16-byte reads meet no bank twice
    static constexpr int TROW = (PARTS * RP + 8) * 2;
    static constexpr int STAGE = 16 * (ROW + TROW);
    static constexpr int FACTOR = COLS * RP * 2;
    static constexpr int bytes(int stages, int factors) { return stages * STAGE + factors * FACTOR + 256; }
    static constexpr int MOST = bytes(4, 2) <= AD_MAP_SMEM ? 4 : 3;    // stages
    static_assert(bytes(MOST, 2) <= AD_MAP_SMEM, "shared memory of a CTA");
};

// A CTA: row_chunk positions, 256 CB columns, eight warps of 32 CB columns (the CTAs
// side by side in the grid share their rows), and a ninth that keeps the copies of the
// next tiles and factors in flight.  Product j (of four) of 32 columns has as its column n
// the logits' column 8 (n / 2) + 2 j + n % 2, so that lane q's eight results are eight
// neighbours.  Measured, inputs out of L2: 8192 x 151936 bf16, rank 16 of 4 adapters, 845 us
// (5.0 GB, 88 % of the copy rate); 64 x 128256 bf16 under 32 adapters 39 us (133 MB, a CTA's only
// tile waits for its factors); rank 64, 16384 x 32000 bf16, 1118 us against a floor of 311: the
// factor is read from shared memory for every 16 rows.
template <typename T, int RP, int PARTS, int CB, bool AL>
__global__ void __launch_bounds__(AD_MAP_THREADS, CB == 1 && RP <= 32 ? 3 : 2) adapters_map_kernel(const AdapterArgs a)
{
    using K = Ranks<RP>;
    using S = MapShape<T, RP, PARTS, CB>;
    constexpr int MAP_WARPS = AD_MAP_THREADS / 32 - 1;
    constexpr int W = Elem<T>::WORDS;
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ int32_t s_row[AD_MAP_ROWS], s_ad[AD_MAP_ROWS + 1];
    const uint32_t base = smem_u32(smem), factor0 = base + a.stages * S::STAGE;
    uint64_t *bars = reinterpret_cast<uint64_t *>(smem + a.stages * S::STAGE + a.factors * S::FACTOR);
    const uint32_t bar0 = smem_u32(bars);
    auto full = [&](int i) { return bar0 + 8u * i; };
    auto empty = [&](int i) { return bar0 + 8u * (4 + i); };
    auto ffull = [&](int i) { return bar0 + 8u * (8 + i); };
    auto fempty = [&](int i) { return bar0 + 8u * (12 + i); };
    volatile int *abort_flag = reinterpret_cast<volatile int *>(bars + 16);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, q = lane & 3;
    const int slabs = (a.V + S::COLS - 1) / S::COLS;
    const int c0 = static_cast<int>(blockIdx.x % slabs) * S::COLS, c1 = min(a.V, c0 + S::COLS);
    const int p0 = static_cast<int>(blockIdx.x / slabs) * a.row_chunk;
    if (tid == 0) {
        for (int i = 0; i < 4; ++i) {
            mbar_init(full(i), 1);
            mbar_init(empty(i), MAP_WARPS);
            mbar_init(ffull(i), 1);
            mbar_init(fempty(i), MAP_WARPS);
        }
        *abort_flag = 0;
        fence_mbar_init();
    }
    pdl_wait();
    pdl_launch_dependents();
    const int live = a.in_place ? a.plan.offsets[a.n] : a.N;   // rows under no adapter come last
    const int rows = min(live - p0, a.row_chunk);
    if (rows <= 0)
        return;
    for (int i = tid; i < rows; i += AD_MAP_THREADS) {
        s_row[i] = a.plan.perm[p0 + i];
        s_ad[i] = a.plan.adapter[p0 + i];
        TIM_DCHECK(static_cast<unsigned>(s_row[i]) < static_cast<unsigned>(a.N) && s_ad[i] >= 0 && s_ad[i] <= a.n, a.status,
                   TIM_CHECK_UNIT, p0 + i, s_ad[i]);
    }
    if (tid == 0)
        s_ad[rows] = -1;
    __syncthreads();
    const T *z = static_cast<const T *>(a.z);
    const uint64_t budget = a.wait_budget_ns;

    if (warp == MAP_WARPS) {
        // ------------------------------------------------------------ copies
        const uint64_t pol = l2_policy_evict_first(), pol_keep = l2_policy_evict_normal();
        int stage = 0, slot = 0, held = -1;   // held: the adapter of the last factor copied
        uint32_t phase = 0, fphase = 0;
        uint32_t used = 0, parity = 0;   // barriers filled (stages from bit 0, factors from bit 8 on), parity of their last fill
        auto filled = [&](int bit, uint32_t p) {
            used |= 1u << bit;
            parity = (parity & ~(1u << bit)) | p << bit;
        };
        bool ok = true;
        for (int p = 0; ok && p < rows; p += 16) {
            ok = warp_wait(empty(stage), phase ^ 1u, abort_flag, budget);
            if (!ok)
                break;
            const int m = min(16, rows - p);
            const uint32_t dst = base + stage * S::STAGE;
            RowCopy c{};
            if (lane < m)
                c = stage_row<T>(z + static_cast<size_t>(s_row[p + lane]) * a.ld, c0, c1, a.V, smem + stage * S::STAGE + lane * S::ROW);
            const uint32_t tbytes = static_cast<uint32_t>(m) * S::TROW;
            const uint32_t total = __reduce_add_sync(0xffffffffu, c.bytes) + tbytes;
            __syncwarp();
            if (lane == 0)
                mbar_arrive_expect_tx(full(stage), total);
            __syncwarp();
            TIM_DCHECK(((reinterpret_cast<uintptr_t>(c.src) | c.off | c.bytes | tbytes |
                         reinterpret_cast<uintptr_t>(a.plan.t + static_cast<size_t>(p0 + p) * (S::TROW / 2))) & 15) == 0 &&
                           c.off + c.bytes <= S::ROW && (lane >= m || c.bytes == 0 ||
                           (c.src >= reinterpret_cast<const char *>(z + static_cast<size_t>(s_row[p + lane]) * a.ld) &&
                            c.src + c.bytes <= reinterpret_cast<const char *>(z + static_cast<size_t>(s_row[p + lane]) * a.ld + a.V))),
                       a.status, TIM_CHECK_BULK, p0 + p + lane, c.bytes);
            if (c.bytes)
                bulk_load(dst + lane * S::ROW + c.off, c.src, c.bytes, full(stage), pol);
            if (lane == 0)
                bulk_load(dst + 16 * S::ROW, a.plan.t + static_cast<size_t>(p0 + p) * (S::TROW / 2), tbytes, full(stage), pol_keep);
            filled(stage, phase);
            if (++stage == a.stages) {
                stage = 0;
                phase ^= 1u;
            }
            // the factors of the adapters that begin in this tile
            const int mine = lane < m ? s_ad[p + lane] : a.n;
            const int before = lane == 0 ? held : lane < m ? s_ad[p + lane - 1] : mine;
            unsigned starts = __ballot_sync(0xffffffffu, mine < a.n && mine != before);
            while (starts) {
                const int i = __ffs(starts) - 1;
                starts &= starts - 1;
                held = s_ad[p + i];
                ok = warp_wait(fempty(slot), fphase ^ 1u, abort_flag, budget);
                if (!ok)
                    break;
                if (lane == 0) {
                    const uint32_t bytes = static_cast<uint32_t>(c1 - c0) * a.R * 2;
                    TIM_DCHECK((bytes & 15) == 0 && bytes <= S::FACTOR, a.status, TIM_CHECK_BULK, held, bytes);
                    mbar_arrive_expect_tx(ffull(slot), bytes);
                    bulk_load(factor0 + slot * S::FACTOR, a.B + (static_cast<size_t>(held) * a.V + c0) * a.R, bytes, ffull(slot),
                              pol_keep);
                }
                filled(8 + slot, fphase);
                if (++slot == a.factors) {
                    slot = 0;
                    fphase ^= 1u;
                }
            }
        }
        // no copy is in flight when the CTA leaves
        if (lane == 0) {
            for (int i = 0; i < 16; ++i)
                if (used >> i & 1u)
                    drain_wait(bar0 + 8u * i, parity >> i & 1u);
        }
        __syncwarp();
    } else {
        // ------------------------------------------------------------ products
        const int w0 = warp * 32 * CB;   // the warp's columns in the slab
        T *out = static_cast<T *>(a.out);
        int stage = 0, held = -1, slot = a.factors - 1;   // slot: of the factor held
        uint32_t phase = 0, fphase = 1;
        bool ok = true;
        const uint32_t frow = static_cast<uint32_t>(a.R) * 2;
        uint32_t f[K::HELD ? K::GROUPS : 1][CB][4][4];   // the factor's columns and ranks of this lane
        const uint32_t fcol = static_cast<uint32_t>(w0 + 8 * (g >> 1) + (g & 1)) * frow + q * (K::STEP * 2);
        auto load_factor = [&](uint32_t (&w)[4], int from, int k, int c, int j) {
            w[0] = w[1] = w[2] = w[3] = 0u;
            if (k * 32 + q * K::STEP < a.R)   // ranks past R: zeros
                lds_words<K::WORDS>(w, factor0 + from * S::FACTOR + fcol + static_cast<uint32_t>(c * 32 + 2 * j) * frow + k * 64);
        };
        for (int p = 0; p < rows; p += 16) {
            ok = warp_wait(full(stage), phase, abort_flag, budget);
            if (!ok)
                break;
            const uint32_t st = base + stage * S::STAGE, ts = st + 16 * S::ROW;
            const int e = min(p + 16, rows);
            float keep[CB][4][4] = {};
            for (int s = p; s < e;) {
                // the positions of this tile under one adapter: s .. m - 1
                const int ad = s_ad[s];
                int m = e;
                if (s_ad[e - 1] != ad)
                    for (m = s + 1; s_ad[m] == ad;)
                        ++m;
                if (ad < a.n) {
                    if (ad != held) {
                        if (!K::HELD) {
                            __syncwarp();
                            if (held >= 0 && lane == 0)
                                mbar_arrive(fempty(slot));
                        }
                        held = ad;
                        if (++slot == a.factors) {
                            slot = 0;
                            fphase ^= 1u;
                        }
                        ok = warp_wait(ffull(slot), fphase, abort_flag, budget);
                        if (!ok)
                            break;
                        if constexpr (K::HELD) {   // the buffer is free again as soon as every warp has its part
#pragma unroll
                            for (int k = 0; k < K::GROUPS; ++k)
#pragma unroll
                                for (int c = 0; c < CB; ++c)
#pragma unroll
                                    for (int j = 0; j < 4; ++j)
                                        load_factor(f[k][c][j], slot, k, c, j);
                            __syncwarp();
                            if (lane == 0)
                                mbar_arrive(fempty(slot));
                        }
                    }
                    float acc[CB][4][4] = {};
#pragma unroll
                    for (int k = 0; k < K::GROUPS; ++k) {
                        uint32_t t[PARTS][2][4];   // rows g and g + 8 of t
#pragma unroll
                        for (int i = 0; i < PARTS; ++i)
#pragma unroll
                            for (int half = 0; half < 2; ++half)
                                lds_words<K::WORDS>(t[i][half], ts + (g + half * 8) * S::TROW + (i * RP + k * 32 + q * K::STEP) * 2);
#pragma unroll
                        for (int c = 0; c < CB; ++c)
#pragma unroll
                            for (int j = 0; j < 4; ++j) {
                                uint32_t (&w)[4] = f[K::HELD ? k : 0][c][j];
                                if (!K::HELD)
                                    load_factor(w, slot, k, c, j);
#pragma unroll
                                for (int i = 0; i < PARTS; ++i) {
                                    mma16816(acc[c][j], {t[i][0][0], t[i][1][0], t[i][0][1], t[i][1][1]}, w[0], w[1]);
                                    if (K::WORDS == 4)
                                        mma16816(acc[c][j], {t[i][0][2], t[i][1][2], t[i][0][3], t[i][1][3]}, w[2], w[3]);
                                }
                            }
                    }
                    const bool in0 = p + g >= s && p + g < m, in1 = p + g + 8 >= s && p + g + 8 < m;
#pragma unroll
                    for (int c = 0; c < CB; ++c)
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            keep[c][j][0] = in0 ? acc[c][j][0] : keep[c][j][0];
                            keep[c][j][1] = in0 ? acc[c][j][1] : keep[c][j][1];
                            keep[c][j][2] = in1 ? acc[c][j][2] : keep[c][j][2];
                            keep[c][j][3] = in1 ? acc[c][j][3] : keep[c][j][3];
                        }
                }
                s = m;
            }
            if (!ok)
                break;
#pragma unroll
            for (int half = 0; half < 2; ++half) {
                const int i = p + g + half * 8;
                const bool on = i < e, has = on && s_ad[on ? i : p] < a.n;
                const int n = on ? s_row[i] : 0;
                T *row = out + static_cast<size_t>(n) * a.ldo;
                const bool any = !AL && __any_sync(0xffffffffu, row_shift(row) != 0);
                const uint32_t shift = AL ? 0u : row_shift(z + static_cast<size_t>(n) * a.ld);
#pragma unroll
                for (int c = 0; c < CB; ++c) {
                    const int col = c0 + w0 + c * 32 + q * 8;
                    const uint8_t *src = smem + stage * S::STAGE + (g + half * 8) * S::ROW + (w0 + c * 32 + q * 8) * sizeof(T);
                    Raw8<T> y;
                    uint32_t x[W + 4];
#pragma unroll
                    for (int k = 0; k < W / 4 + (AL ? 0 : 1); ++k) {
                        const uint4 v = reinterpret_cast<const uint4 *>(src)[k];
                        x[4 * k] = v.x;
                        x[4 * k + 1] = v.y;
                        x[4 * k + 2] = v.z;
                        x[4 * k + 3] = v.w;
                    }
                    if (AL) {
#pragma unroll
                        for (int k = 0; k < W; ++k)
                            y.w[k] = x[k];
                    } else {
                        shift_words<W, sizeof(T) == 2>(y.w, x, shift);
                    }
                    float v[8];
#pragma unroll
                    for (int k = 0; k < 8; ++k)
                        v[k] = Elem<T>::get(y.w, k) + keep[c][k >> 1][2 * half + (k & 1)];
                    Raw8<T> w = pack8<T>(v);
                    if (!has)
                        w = y;   // a row under no adapter keeps its bits
                    store_quad<T>(row, col, a.V, w, on && col < a.V, any);
                }
            }
            __syncwarp();
            if (lane == 0)
                mbar_arrive(empty(stage));
            if (++stage == a.stages) {
                stage = 0;
                phase ^= 1u;
            }
        }
    }
    __syncthreads();
    if (tid == 0 && *abort_flag)
        atomicCAS(a.status, 0, static_cast<int>(TIM_ERR_TIMEOUT));
}

template <typename F>
cudaError_t launch(F kernel, dim3 grid, int threads, int smem, const AdapterArgs &a, cudaStream_t s)
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

template <int RP, int PARTS> cudaError_t shrink(const AdapterArgs &a, int num_sms, cudaStream_t s)
{
    if (a.N > AD_FEW_ROWS) {
        const cudaError_t e = launch(adapters_order_kernel, dim3(static_cast<unsigned>(a.n + 1)), 512, 0, a, s);
        if (e != cudaSuccess)
            return e;
        const int ctas = (a.N + 15) / 16;
        return launch(ctas > num_sms ? adapters_project_kernel<RP, PARTS, true> : adapters_project_kernel<RP, PARTS, false>,
                      dim3(static_cast<unsigned>(ctas)), 512, 0, a, s);
    }
    const int ys = std::max(1, std::min((a.N + 15) / 16, (2 * num_sms + a.n) / (a.n + 1)));
    return launch(adapters_shrink_kernel<RP, PARTS>, dim3(static_cast<unsigned>(a.n + 1), static_cast<unsigned>(ys)),
                  512, 0, a, s);
}

template <int PARTS> cudaError_t shrink(const AdapterArgs &a, int num_sms, cudaStream_t s)
{
    switch (ad_rank_pad(a.R)) {
    case 16: return shrink<16, PARTS>(a, num_sms, s);
    case 32: return shrink<32, PARTS>(a, num_sms, s);
    case 64: return shrink<64, PARTS>(a, num_sms, s);
    default: return shrink<128, PARTS>(a, num_sms, s);
    }
}

template <typename T, int PARTS, int RP, int CB> cudaError_t map(AdapterArgs a, int num_sms, cudaStream_t s, bool set)
{
    using S = MapShape<T, RP, PARTS, CB>;
    auto aligned = adapters_map_kernel<T, RP, PARTS, CB, true>, any = adapters_map_kernel<T, RP, PARTS, CB, false>;
    if (set) {
        const cudaError_t e = cudaFuncSetAttribute(aligned, cudaFuncAttributeMaxDynamicSharedMemorySize, AD_MAP_SMEM);
        return e != cudaSuccess ? e : cudaFuncSetAttribute(any, cudaFuncAttributeMaxDynamicSharedMemorySize, AD_MAP_SMEM);
    }
    const int slabs = (a.V + S::COLS - 1) / S::COLS;
    // few rows: a tile a CTA, so that the adapters' factors come in parallel, and more of them at a time
    int64_t rows = AD_MAP_ROWS;
    while (rows > 16 && slabs * ((a.N + rows - 1) / rows) < int64_t(8) * num_sms)
        rows /= 2;
    a.row_chunk = static_cast<int32_t>(rows);
    a.stages = std::min<int>(a.N > AD_FEW_ROWS ? S::MOST : 2, static_cast<int>(rows / 16));
    // and then most of what is read are factors: as many as leave room for three CTAs an SM
    // (256 x 151936 bf16, rank 32 of 64: 167 us with three factors and two tiles, 198 with two and four)
    a.factors = 2;
    while (a.N <= AD_FEW_ROWS && a.factors < 4 && S::bytes(a.stages, a.factors + 1) <= AD_MAP_SMEM / 3)
        ++a.factors;
    const dim3 grid(static_cast<unsigned>(slabs * ((a.N + rows - 1) / rows)));
    auto starts16 = [](const void *p, int64_t ld, int64_t N) {
        return (reinterpret_cast<uintptr_t>(p) & 15) == 0 && (N == 1 || ld * sizeof(T) % 16 == 0);
    };
    return launch(starts16(a.z, a.ld, a.N) && starts16(a.out, a.ldo, a.N) ? aligned : any, grid, AD_MAP_THREADS,
                  S::bytes(a.stages, a.factors), a, s);
}

// A warp has 32 columns, or 64 (128 bytes of a row) of 16-bit logits at the smallest ranks, where a
// batch is large enough to be bound by them (8192 x 151936 bf16: 910 us, 1150 with 32; 2400 x 8192, below
// the rule, 48 us with 32 columns, 56 with 64).
template <typename T, int PARTS, int RP> cudaError_t map(const AdapterArgs &a, int num_sms, cudaStream_t s, bool set)
{
    if constexpr (sizeof(T) == 2 && RP == 16) {
        if (set) {
            const cudaError_t e = map<T, PARTS, RP, 1>(a, num_sms, s, true);
            return e != cudaSuccess ? e : map<T, PARTS, RP, 2>(a, num_sms, s, true);
        }
        if (static_cast<int64_t>(a.N) * a.V >= int64_t(num_sms) * 512 * AD_MAP_ROWS)
            return map<T, PARTS, RP, 2>(a, num_sms, s, false);
    }
    return map<T, PARTS, RP, 1>(a, num_sms, s, set);
}

template <typename T, int PARTS> cudaError_t map(const AdapterArgs &a, int num_sms, cudaStream_t s)
{
    switch (ad_rank_pad(a.R)) {
    case 16: return map<T, PARTS, 16>(a, num_sms, s, false);
    case 32: return map<T, PARTS, 32>(a, num_sms, s, false);
    case 64: return map<T, PARTS, 64>(a, num_sms, s, false);
    default: return map<T, PARTS, 128>(a, num_sms, s, false);
    }
}

template <typename T, int PARTS> cudaError_t prepare()
{
    const AdapterArgs a{};
    cudaError_t e = map<T, PARTS, 16>(a, 1, nullptr, true);
    if (e == cudaSuccess)
        e = map<T, PARTS, 32>(a, 1, nullptr, true);
    if (e == cudaSuccess)
        e = map<T, PARTS, 64>(a, 1, nullptr, true);
    return e != cudaSuccess ? e : map<T, PARTS, 128>(a, 1, nullptr, true);
}

} // namespace

cudaError_t adapters_prepare_device()
{
    cudaError_t e = prepare<float, 3>();
    if (e == cudaSuccess)
        e = prepare<__nv_bfloat16, 2>();
    return e != cudaSuccess ? e : prepare<__half, 2>();
}

cudaError_t adapters_shrink_launch(const AdapterArgs &a, int parts, int num_sms, cudaStream_t s)
{
    return parts == 3 ? shrink<3>(a, num_sms, s) : shrink<2>(a, num_sms, s);
}

cudaError_t adapters_expand_launch(AdapterArgs a, int dtype, int num_sms, cudaStream_t s)
{
    if (dtype == TIM_F32)
        return map<float, 3>(a, num_sms, s);
    if (dtype == TIM_BF16)
        return map<__nv_bfloat16, 2>(a, num_sms, s);
    return map<__half, 2>(a, num_sms, s);
}

} // namespace tim
