// adapters_grad.cu -- gradient of the low-rank adapters on a head's logits (sm_103a).
//
// For the logits' gradient dy [N, V], row i under adapter a, t_i = s_a A_a h_i:
//   dB_a = sum_i dy_i t_i^T        [V, R]
//   du_i = s_a B_a^T dy_i          [R]
//   dA_a = sum_i du_i h_i^T        [R, D]
//   dh_i (+)= A_a^T du_i           [D]
// dy is by far the largest operand and is read once for every 64 ranks: a CTA owns a slab of the
// vocabulary (up to 1024 columns) and walks all rows, adapter by adapter in steps of 128 rows
// (bf16), 64 (fp16) or 32 (fp32).  du of a step (the slab's part of the sum over V) goes to a
// partial array that a second launch folds in slab order.  dB's part of the slab stays in
// TMEM for up to a.link rows of the adapter and then goes to memory, where the next link's is
// added: the tensor cores cut what they add up, and one sum over all of 8200 rows lost 4e-6 to
// 5e-5 of dB.  Both products take the same tile, 128 columns of a step, from shared memory
// (tcgen05.mma, bf16 -> fp32; a step's planes of bf16 parts lie behind each other as its 128
// rows): du with the rows as M and the columns as K (K-major), dB with the columns as M and
// the rows as K (MN-major, the same bytes).
//   warp 0      the adapter's factor and t, by TMA
//   warp 1      issues the products, one lane of the converged warp
//   warps 2-5   du and dB from TMEM to memory
//   warps 6-    the tiles (the rows of an adapter lie anywhere).  COPY, bf16 rows that start on
//               16 bytes: 16-byte asynchronous copies to their swizzled places.  LOAD (fp32 and
//               fp16 rows that start there) and ANY: such copies into a ring of whole rows, a
//               row's ends by plain loads, and from there as planes of bf16 parts: one, two
//               (fp16, exactly), or three (fp32: 2^-24 of it is left at most)
// (TMA gathers of four rows brought the same tiles at 2 us a tile of 32 KB and SM.)
// Measured, dy's pass alone, inputs out of L2: 4096 x 128256 bf16, rank 16 of 8 adapters, 207 us
// (1.02 GB, 62 % of DRAM's nominal peak; what is left are the drains of dB and slabs that fill
// 143 of 152 SMs); 1024 x 129280 fp32, rank 32 of 3, 223 us (issue slots 51 %: the rewriting, and
// nine products of parts a tile); 500 x 50261 fp16 off 16 bytes 64 us.
// Every sum has one order, fixed by the rows' order and V: the same call gives the same bits.
#include <algorithm>
#include <type_traits>

#include "adapters.cuh"
#include "table_internal.h"
#include "tim_internal.h"

namespace tim {
namespace {

constexpr int BC = AG_BLOCK;            // columns of a tile
constexpr int PARTS = 3;                // of t

// How tiles are brought: COPY, bf16 rows from 16-byte boundaries on; LOAD, other types'
// rows from there; ANY, rows that start anywhere.
enum { COPY, LOAD, ANY };

template <typename T, int HOW, int RP> struct Shape {
    static constexpr int PLANES = sizeof(T) == 4 ? 3 : std::is_same<T, __nv_bfloat16>::value ? 1 : 2;
    static constexpr int STEP = PLANES == 1 ? 128 : PLANES == 2 ? 64 : 32;   // rows of a tile; the planes lie behind each other as its rows
    static constexpr int SUB = 128 * 128;                      // bytes of 64 columns of it
    static constexpr int SPAN = RP * 2;                        // bytes of a row of the factor, or of a part of t
    static constexpr int SPAN2 = SPAN == 128 ? 128 : 2 * SPAN; // of two parts of t side by side (ranks up to 32)
    static constexpr int BLOCKS = ag_blocks(RP);               // tiles of a slab at most
    static constexpr int TILE = 2 * SUB;
    static constexpr int FACTORS = (RP == 16 && HOW == COPY ? 2 : 1) * BLOCKS * BC * SPAN;   // bytes for factors: two where they fit
    static constexpr int TT = (RP <= 32 ? 4 : PARTS) * STEP * SPAN;
    static constexpr int TS = RP == 64 && PLANES == 1 && HOW != COPY ? 1 : 2;
    static constexpr int REST = AG_SMEM - 2048 - FACTORS - TS * TT;
    // not COPY: rows on their way to the warps that rewrite them, 32 NR in a batch
    static constexpr int SROW = BC * static_cast<int>(sizeof(T)) + (HOW == ANY ? 16 : 0);
    static constexpr int NR = PLANES == 2 ? 2 : 1, BATCH = NR * 32 * SROW;
    static constexpr int FIT = (REST - 2 * TILE) / BATCH, BATCHES = FIT < 4 ? FIT : 4;
    static constexpr int STAGING = HOW == COPY ? 0 : BATCHES * BATCH;
    static constexpr int STAGES = (REST - STAGING) / TILE < 4 ? (REST - STAGING) / TILE : 4;
    static constexpr int BYTES = AG_SMEM;
    static constexpr int WRITERS = HOW == COPY ? 8 : 16;       // warps that bring tiles
    static constexpr int THREADS = (6 + WRITERS) * 32;
    static constexpr uint32_t TMEM = 512;                      // du twice, dB's blocks
    static constexpr int CHAIN = 4;                            // tiles of a sum of du in TMEM
    // tiles whose sums of dB are free again together: one (4096 x 128256, rank 64 of 2: bf16 612 us, 681 with
    // four; fp16 1035, 1139), or four where the issue of the products is the narrow part (fp32, rank 32:
    // 1024 x 129280 302 us, 308 with one)
    static constexpr int FREED = PLANES == 3 && RP <= 32 ? CHAIN : 1;
    static_assert(RP <= 32 || CHAIN >= BLOCKS, "ranks beyond 32 are not added up in registers");
    static_assert(STAGES >= 2 && (HOW == COPY || BATCHES >= 2) && (2 + BLOCKS) * RP <= 512, "shared memory, TMEM");
};

// An adapter's positions [begin, end) of a part [p0, p1) of the batch: parts meet at a
// multiple of 16 rows of the adapter (t has zeros behind its last row only).
struct Part {
    int begin, end;
    __device__ __forceinline__ Part(int first, int last, int p0, int p1)
        : begin(min(last, cut(first, p0))), end(min(last, cut(first, p1)))
    {
    }
    static __device__ __forceinline__ int cut(int first, int p) { return p <= first ? first : first + (p - first + 15) / 16 * 16; }
};

// ldmatrix, for the smaller products below
__device__ __forceinline__ void ldsm4t(uint32_t (&r)[4], uint32_t addr)
{
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}

// `bytes` of 16 global -> shared, zeros in the rest.
__device__ __forceinline__ void cp_async16(uint32_t dst, const void *src, uint32_t bytes)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(reinterpret_cast<uint64_t>(src)), "r"(bytes)
                 : "memory");
}

// One arrival on `bar` when this thread's asynchronous copies so far have landed.
__device__ __forceinline__ void cp_async_arrive(uint32_t bar)
{
    asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(bar) : "memory");
}

// A ring's place: its slot, and the parity of the slot's current use.
struct Ring {
    int slots, slot = 0;
    uint32_t parity = 0;
    __device__ __forceinline__ explicit Ring(int n) : slots(n) {}
    __device__ __forceinline__ void next()
    {
        if (++slot == slots) {
            slot = 0;
            parity ^= 1u;
        }
    }
};

// High words of the operands' descriptors (their low words: the address / 16, and the
// leading offset / 16 from bit 16 on) as of sdesc_kmajor_sw128, sdesc_mnmajor_sw128, and of
// one swizzle span (32, 64 or 128 bytes, modes 6, 4, 2) as the M or N extent: a row of
// `span` bytes for each k, 8-row groups 8 span bytes apart.
__host__ __device__ constexpr uint32_t desc_kmajor_hi() { return 1024u / 16 | 1u << 14 | 2u << 29; }
__host__ __device__ constexpr uint32_t desc_mnmajor_hi() { return desc_kmajor_hi(); }
__host__ __device__ constexpr uint32_t desc_span_hi(int span)
{
    return static_cast<uint32_t>(8 * span) / 16 | 1u << 14 | (span == 128 ? 2u : span == 64 ? 4u : 6u) << 29;
}

__device__ __forceinline__ float4 plus(float4 x, float4 y) { return make_float4(x.x + y.x, x.y + y.y, x.z + y.z, x.w + y.w); }

// *p += x without waiting for *p (loads of it held the products up: 8192 x 151936 under one
// adapter of rank 32 936 us, 863 so).  One thread alone adds to p, so the order is its own.
// Sums below 2^-126 may count as zero.
__device__ __forceinline__ void red_add4(float4 *p, float4 x)
{
    asm volatile("red.relaxed.gpu.global.add.v4.f32 [%0], {%1, %2, %3, %4};" ::"l"(p), "f"(x.x), "f"(x.y), "f"(x.z), "f"(x.w)
                 : "memory");
}

template <int RC> __device__ __forceinline__ void tmem_row(uint32_t taddr, float (&v)[RC])
{
    static_assert(RC == 16 || RC == 32, "columns of one load");
    if constexpr (RC == 16)
        tmem_load16(taddr, v);
    else
        tmem_load32(taddr, v);
}

template <typename T, int HOW, int RP>
__global__ void __launch_bounds__(Shape<T, HOW, RP>::THREADS, 1)
    adapters_grad_kernel(const __grid_constant__ CUtensorMap map_b, const __grid_constant__ CUtensorMap map_t,
                         const __grid_constant__ AdapterGradArgs a)
{
    using S = Shape<T, HOW, RP>;
    constexpr int STEP = S::STEP, SUB = S::SUB;
    // M = 128 in both: du's rows are the tile's (each plane's product is a part of the sum)
    constexpr uint32_t IDESC_DU = idesc_bf16_f32(128, RP, false, true), IDESC_DB = idesc_bf16_f32(BC, RP, true, true),
                       IDESC_DB2 = idesc_bf16_f32(BC, 2 * RP, true, true);
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const uint32_t tiles = smem_u32(smem), factors = tiles + S::STAGES * S::TILE, ts = factors + S::FACTORS;
    const uint32_t staging = ts + S::TS * S::TT;
    uint64_t *bars = reinterpret_cast<uint64_t *>(smem + S::STAGES * S::TILE + S::FACTORS + S::TS * S::TT + S::STAGING);
    const uint32_t bar0 = smem_u32(bars);
    auto full = [&](int i) { return bar0 + 8u * i; };
    auto empty = [&](int i) { return bar0 + 8u * (4 + i); };
    auto tfull = [&](int i) { return bar0 + 8u * (8 + i); };
    auto tempty = [&](int i) { return bar0 + 8u * (10 + i); };
    auto ffull = [&](int i) { return bar0 + 8u * (12 + i); };
    auto fempty = [&](int i) { return bar0 + 8u * (14 + i); };
    auto dufull = [&](int i) { return bar0 + 8u * (16 + i); };
    auto duempty = [&](int i) { return bar0 + 8u * (18 + i); };
    auto dbfull = [&](int i) { return bar0 + 8u * (20 + i); };
    const uint32_t drain = bar0 + 8u * 22;
    auto dbempty = [&](int i, int block) { return bar0 + 8u * (23 + i * S::BLOCKS + block); };
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(bars + 23 + 2 * S::BLOCKS);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_slot + 1);

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int c0 = blockIdx.x * a.cols;                                   // the slab's columns
    const int blocks = (min(a.V, c0 + a.cols) - c0 + BC - 1) / BC;
    // two factors, and dB's sums of two adapters, where a slab's are small enough
    const int factor_bytes = a.cols * S::SPAN, num_factors = 2 * factor_bytes <= S::FACTORS ? 2 : 1;
    // t's first two parts side by side as one operand (N = 2 RP, the second's products in columns of their own) where TMEM has room
    const int db_block = a.merged ? 2 * RP : RP, db_chain = a.cols / BC * db_block;
    const int db_columns = (a.chains + a.low) * db_chain, num_db = 2 * RP + 2 * db_columns <= 512 ? 2 : 1;
    if (tid == 0) {
        for (int i = 0; i < S::STAGES; ++i) {
            mbar_init(full(i), HOW == COPY ? S::WRITERS * 32 : S::WRITERS);
            mbar_init(empty(i), 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(tfull(i), 1);
            mbar_init(tempty(i), 1);
            mbar_init(ffull(i), 1);
            mbar_init(fempty(i), 1);
            mbar_init(dufull(i), 1);
            mbar_init(duempty(i), 4);
            mbar_init(dbfull(i), 1);
            for (int c = 0; c < S::BLOCKS; ++c)
                mbar_init(dbempty(i, c), 4);
        }
        mbar_init(drain, 1);
        *abort_flag = 0;
        fence_mbar_init();
    }
    if (warp == 0 && lane == 0) {
        tma_prefetch_desc(&map_b);
        tma_prefetch_desc(&map_t);
    }
    pdl_wait();
    pdl_launch_dependents();
    if (warp == 1) {
        tmem_alloc(smem_u32(tmem_slot), S::TMEM);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;   // du: 2 x RP columns, then dB: RP columns a block
    const uint64_t budget = a.wait_budget_ns;
    const T *dy = static_cast<const T *>(a.dy);

    // The adapters with positions in this part, in order: f(adapter, first, end); false ends.
    auto segments = [&](auto f) {
        for (int ad = 0; ad < a.n; ++ad) {
            const Part r(a.plan.offsets[ad], a.plan.offsets[ad + 1], a.p0, a.p1);
            if (r.begin < r.end && !f(ad, r.begin, r.end))
                break;
        }
    };

    if (warp == 0) {
        // ------------------------------------------------------------ copies
        const uint64_t pol_keep = l2_policy_evict_normal();
        Ring tr(S::TS), fr(num_factors);
        uint32_t used_t = 0, used_f = 0, par_t = 0, par_f = 0;   // slots filled, parity of their last fill
        segments([&](int ad, int b, int e) {
            if (!warp_wait(fempty(fr.slot), fr.parity ^ 1u, abort_flag, budget))
                return false;
            if (lane == 0) {
                mbar_arrive_expect_tx(ffull(fr.slot), static_cast<uint32_t>(blocks) * BC * S::SPAN);
                for (int c = 0; c < blocks; ++c)
                    tma_load_3d(factors + fr.slot * factor_bytes + c * BC * S::SPAN, &map_b, ffull(fr.slot), a.r0, c0 + c * BC, ad,
                                pol_keep);
            }
            used_f |= 1u << fr.slot;
            par_f = (par_f & ~(1u << fr.slot)) | (fr.parity << fr.slot);
            fr.next();
            for (int p = b; p < e; p += STEP) {
                if (!warp_wait(tempty(tr.slot), tr.parity ^ 1u, abort_flag, budget))
                    return false;
                // t has its zeros up to a multiple of 16 of the adapter's rows
                TIM_DCHECK(p + ad * AG_PAD + (min(STEP, e - p) + 15) / 16 * 16 <= a.N + a.n * AG_PAD && a.r0 % 8 == 0, a.status,
                           TIM_CHECK_TMA_COORD, p, ad);
                if (lane == 0) {
                    mbar_arrive_expect_tx(tfull(tr.slot), (a.merged ? 4 : PARTS) * STEP * S::SPAN);
                    // part by part; or the first two side by side, then the third beside zeros (past t's last column)
                    const int boxes = a.merged ? 2 : PARTS, width = a.merged ? 2 * RP : RP;
                    for (int i = 0; i < boxes; ++i)
                        tma_load_2d(ts + tr.slot * S::TT + i * STEP * width * 2, &map_t, tfull(tr.slot),
                                    a.merged ? i * width : i * a.RT + a.r0, p + ad * AG_PAD, pol_keep);
                }
                used_t |= 1u << tr.slot;
                par_t = (par_t & ~(1u << tr.slot)) | (tr.parity << tr.slot);
                tr.next();
            }
            return true;
        });
        // no copy is in flight when the CTA leaves
        if (lane == 0) {
            for (int i = 0; i < 2; ++i) {
                if (used_t >> i & 1u)
                    drain_wait(tfull(i), par_t >> i & 1u);
                if (used_f >> i & 1u)
                    drain_wait(ffull(i), par_f >> i & 1u);
            }
        }
        __syncwarp();
    } else if (warp == 1) {
        // ------------------------------------------------------------ products
        // the whole warp, one lane issues
        const uint32_t lead = elect_one();
        Ring st(S::STAGES), tr(S::TS), fr(num_factors), du(2), db(num_db);
        constexpr uint32_t KHI = static_cast<uint32_t>(desc_kmajor_hi()), MHI = static_cast<uint32_t>(desc_mnmajor_hi());
        // du += tile x factor, 16 columns at a time, and dB += tile^T x t, 16 rows at a time,
        // in turn (neither waits for itself); products of parts of 2^-24 of the first's are left out.
        // The first parts' products go to tb, all others to low: the tensor cores cut, rather
        // than round, what they add up, and the chain of the first is as short as can be.
        auto tile_products = [&](auto merged, auto whole, uint32_t tile, uint32_t td, uint32_t tb, uint32_t low, uint32_t fd,
                                 uint32_t tt, int steps, uint32_t first_du, uint32_t first_db, uint32_t first_low) {
            constexpr bool MERGED = decltype(merged)::value, WHOLE = decltype(whole)::value;
            constexpr int TSPAN = MERGED ? S::SPAN2 : S::SPAN;
            const uint32_t a0 = tile >> 4, am = a0 | (static_cast<uint32_t>(SUB) >> 4) << 16;
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                umma_bf16_lead(lead, td, (a0 | 1u << 16) + (k / 4) * (SUB / 16) + 2 * (k % 4), KHI,
                               fd + k * S::SPAN, desc_span_hi(S::SPAN), IDESC_DU, k == 0 ? first_du : 1u);
                const int kr = k % (STEP / 16), plane = k / (STEP / 16);
                if (plane < S::PLANES && (WHOLE || kr < steps)) {
                    const uint32_t more = k == 0 ? first_db : 1u;
                    if (plane == 0)   // merged: part 1 of t beside it, whose columns are `low`
                        umma_bf16_lead(lead, tb, am + 128 * k, MHI, tt + kr * TSPAN, desc_span_hi(TSPAN), MERGED ? IDESC_DB2 : IDESC_DB,
                                       more);
#pragma unroll
                    for (int j = plane > 0 ? 0 : MERGED ? 2 : 1; j < PARTS - plane; ++j) {
                        // merged: parts 0 and 1 share rows of 2 RP, part 2 lies behind them
                        const uint32_t at = MERGED ? (j == 2 ? (STEP / 16 + kr) * TSPAN : kr * TSPAN + j * (S::SPAN / 16))
                                                   : (j * STEP / 16 + kr) * TSPAN;
                        umma_bf16_lead(lead, MERGED ? tb + RP : low, am + 128 * k, MHI, tt + at, desc_span_hi(TSPAN), IDESC_DB,
                                       !MERGED && k == 0 && j == 1 && low != tb ? first_low : 1u);
                    }
                }
            }
        };
        constexpr std::integral_constant<bool, true> yes{};
        constexpr std::integral_constant<bool, false> no{};
        segments([&](int, int b, int e) {
            if (!warp_wait(ffull(fr.slot), fr.parity, abort_flag, budget))
                return false;
            const uint32_t fd = ((factors + fr.slot * factor_bytes) >> 4) | 1u << 16;
            int link = b, chain = 0;   // where dB's sums began; the steps' products go to them in turn
            for (int p = b; p < e; p += STEP) {
                if (p == link + a.link) {   // long enough: what they have goes to memory
                    umma_commit_lead(lead, dbfull(db.slot));
                    db.next();
                    link = p;
                    chain = 0;
                }
                if (!warp_wait(tfull(tr.slot), tr.parity, abort_flag, budget))
                    return false;
                const int steps = (min(STEP, e - p) + 15) / 16;   // of 16 rows
                const uint32_t tt = ((ts + tr.slot * S::TT) >> 4) | 1u << 16;
                const uint32_t tdb0 = tmem + 2 * RP + db.slot * db_columns + chain * db_chain;
                const uint32_t first_db = p >= link + a.chains * STEP, first_low = a.merged ? first_db : p != link;
                const uint32_t low = a.low ? (a.chains - chain) * db_chain : 0;   // merged: beside the first part's columns
                chain = chain + 1 == a.chains ? 0 : chain + 1;
                for (int c = 0; c < blocks; ++c) {
                    if (c % S::CHAIN == 0) {
                        if (!warp_wait(duempty(du.slot), du.parity ^ 1u, abort_flag, budget))
                            return false;
                        // the first tiles go on while the last ones' sums are written
                        if (S::FREED == S::CHAIN && p == link && !warp_wait(dbempty(db.slot, c / S::CHAIN), db.parity ^ 1u, abort_flag, budget))
                            return false;
                    }
                    if (S::FREED == 1 && p == link && !warp_wait(dbempty(db.slot, c), db.parity ^ 1u, abort_flag, budget))
                        return false;
                    const uint32_t td = tmem + du.slot * RP;
                    if (!warp_wait(full(st.slot), st.parity, abort_flag, budget))
                        return false;
                    // the writers' shared memory for the products: the fence stands here, since a
                    // writer's would wait for its copies of later tiles too
                    fence_proxy_async_smem();
                    tc_fence_after();
                    const uint32_t tile = tiles + st.slot * S::TILE, f = fd + c * (BC * S::SPAN / 16);
                    const uint32_t tb = tdb0 + c * db_block, first_du = c % S::CHAIN != 0;
                    if (a.merged) {
                        if (steps == STEP / 16)
                            tile_products(yes, yes, tile, td, tb, tb + low, f, tt, steps, first_du, first_db, first_low);
                        else
                            tile_products(yes, no, tile, td, tb, tb + low, f, tt, steps, first_du, first_db, first_low);
                    } else {
                        if (steps == STEP / 16)
                            tile_products(no, yes, tile, td, tb, tb + low, f, tt, steps, first_du, first_db, first_low);
                        else
                            tile_products(no, no, tile, td, tb, tb + low, f, tt, steps, first_du, first_db, first_low);
                    }
                    umma_commit_lead(lead, empty(st.slot));
                    st.next();
                    if ((c + 1) % S::CHAIN == 0 || c + 1 == blocks) {
                        umma_commit_lead(lead, dufull(du.slot));
                        du.next();
                    }
                }
                umma_commit_lead(lead, tempty(tr.slot));
                tr.next();
            }
            umma_commit_lead(lead, fempty(fr.slot));
            umma_commit_lead(lead, dbfull(db.slot));
            fr.next();
            db.next();
            return true;
        });
        umma_commit_lead(lead, drain);   // every product has finished before TMEM is released
        if (lead)
            drain_wait(drain, 0);
        __syncwarp();
    } else if (warp < 6) {
        // ------------------------------------------------------------ results
        constexpr int RC = RP < 32 ? RP : 32, DC = 16;   // ranks of du, of dB at a time
        const int m = (warp & 3) * 32 + lane;   // row of du, column of dB's block
        const uint32_t mine = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16);
        Ring du(2), db(num_db);
        bool ok = true;
        for (int ad = 0; ok && ad < a.n; ++ad) {
            const int ob = a.plan.offsets[ad], oe = a.plan.offsets[ad + 1];
            const Part r(ob, oe, a.p0, a.p1);
            const int b = r.begin, e = r.end;
            const bool some = b < e;
            // an adapter whose rows began in an earlier part of the batch is added to; one
            // without rows is written (zeros) by the first part
            const bool add = a.accumulate || b > ob;
            if (!some && !(ob == oe && a.p0 == 0 && !a.accumulate))
                continue;
            for (int link = b; ok && link < max(e, b + 1); link += a.link) {   // dB's sums, from begun to written
                const int link_end = min(e, link + a.link);
                const int chains = min(a.chains, (link_end - link + STEP - 1) / STEP);   // dB's sums that have something
                for (int p = link; p < link_end; p += STEP) {
                    const int at = p + m % STEP;
                    // [part][four ranks][position]: a warp's rows lie together
                    const size_t count = a.p1 - a.p0 + 16;
                    float4 *o = reinterpret_cast<float4 *>(a.partial) +
                                static_cast<size_t>(blockIdx.x * S::PLANES + m / STEP) * (RP / 4) * count + (at - a.p0);
                    auto put = [&](int r0, const float (&v)[RC]) {
                        if (at < e && m / STEP < S::PLANES) {
                            TIM_DCHECK(at >= a.p0 && at - a.p0 < static_cast<int>(count) && r0 + RC <= RP, a.status, TIM_CHECK_STORE, at, ad);
#pragma unroll
                            for (int r = 0; r < RC / 4; ++r)
                                o[(r0 / 4 + r) * count] = make_float4(v[4 * r], v[4 * r + 1], v[4 * r + 2], v[4 * r + 3]);
                        }
                    };
                    float sum[RC] = {};   // of the chains of a slab (more than one where RP = RC)
                    for (int c = 0; c < blocks; c += S::CHAIN) {
                        ok = warp_wait(dufull(du.slot), du.parity, abort_flag, budget);
                        if (!ok)
                            break;
                        tc_fence_after();
#pragma unroll
                        for (int r0 = 0; r0 < RP; r0 += RC) {
                            float v[RC];
                            __syncwarp();
                            tmem_row<RC>(mine + du.slot * RP + r0, v);
                            if constexpr (RP == RC) {
#pragma unroll
                                for (int r = 0; r < RC; ++r)
                                    sum[r] += v[r];
                            } else {
                                put(r0, v);
                            }
                        }
                        tc_fence_before();
                        __syncwarp();
                        if (lane == 0)
                            mbar_arrive(duempty(du.slot));
                        du.next();
                    }
                    if (!ok)
                        break;
                    if (RP == RC)
                        put(0, sum);
                }
                if (!ok)
                    break;
                if (some) {
                    ok = warp_wait(dbfull(db.slot), db.parity, abort_flag, budget);
                    if (!ok)
                        break;
                    tc_fence_after();
                }
                for (int c = 0; c < blocks; ++c) {
                    const int col = c0 + c * BC + m;
                    const uint32_t tb = mine + 2 * RP + db.slot * db_columns + c * db_block;
                    float4 *o = reinterpret_cast<float4 *>(a.dB + (static_cast<size_t>(ad) * a.V + col) * a.R + a.r0);
#pragma unroll
                    for (int r0 = 0; r0 < RP; r0 += DC) {
                        if (a.r0 + r0 >= a.R)
                            break;
                        float v[DC] = {};
                        if (some) {
                            __syncwarp();
                            tmem_row<DC>(tb + r0, v);
                            auto add_up = [&](uint32_t from) {
                                float x[DC];
                                tmem_row<DC>(from, x);
#pragma unroll
                                for (int r = 0; r < DC; ++r)
                                    v[r] += x[r];
                            };
                            for (int i = 1; i < chains; ++i)
                                add_up(tb + i * db_chain + r0);
                            if (RP <= 32 && a.merged) {
                                for (int i = 0; i < chains; ++i)
                                    add_up(tb + i * db_chain + RP + r0);
                            } else if (a.low) {
                                add_up(tb + a.chains * db_chain + r0);
                            }
                        }
                        if (some && r0 + DC >= min(RP, a.R - a.r0) && ((c + 1) % S::FREED == 0 || c + 1 == blocks)) {   // the last ranks are read
                            tc_fence_before();
                            __syncwarp();
                            if (lane == 0)
                                mbar_arrive(dbempty(db.slot, c / S::FREED));
                        }
                        if (col >= a.V)
                            continue;
#pragma unroll
                        for (int r = 0; r < DC / 4; ++r) {
                            if (a.r0 + r0 + 4 * r >= a.R)
                                break;
                            float4 x = make_float4(v[4 * r], v[4 * r + 1], v[4 * r + 2], v[4 * r + 3]);
                            if (link > b) {
                                red_add4(o + r0 / 4 + r, x);
                                continue;
                            }
                            if (add)
                                x = plus(x, o[r0 / 4 + r]);
                            o[r0 / 4 + r] = x;
                        }
                    }
                }
                if (some)
                    db.next();
            }
        }
    } else {
        // ------------------------------------------------------------ tiles
        // a thread has columns 8 (t % 16) .. of every EACH-th row of a tile; 128-byte swizzle:
        // the 16-byte pieces of row m are exchanged by m % 8
        constexpr int EACH = S::WRITERS * 2, ROWS = STEP / EACH;   // 16, or 32 rows apart
        const int t = tid - 6 * 32, chunk = t & 15, r0 = t >> 4;
        auto place = [&](int m) {
            return static_cast<uint32_t>((chunk >> 3) * SUB + m * 128 + (((chunk & 7) ^ (m & 7)) << 4));
        };
        auto in_batch = [&](int r) {
            TIM_DCHECK(static_cast<unsigned>(r) < static_cast<unsigned>(a.N), a.status, TIM_CHECK_UNIT, r, blockIdx.x);
            return static_cast<size_t>(r);
        };
        const T *row[ROWS];   // of the step, from the slab's (COPY: the thread's) first column on; null: past its last
        const int mine = HOW == COPY ? chunk * 8 : 0;
        auto look_up = [&](int p, int rows) {
#pragma unroll
            for (int i = 0; i < ROWS; ++i)
                row[i] = r0 + EACH * i < rows ? dy + in_batch(a.plan.perm[p + r0 + EACH * i]) * a.ld + c0 + mine : nullptr;
        };
        if constexpr (HOW == COPY) {
            Ring st(S::STAGES);
            segments([&](int, int b, int e) {
                for (int p = b; p < e; p += STEP) {
                    const int rows = min(STEP, e - p), padded = (rows + 15) / 16 * 16;
                    look_up(p, rows);
                    for (int c = 0; c < blocks; ++c) {
                        const int col = c0 + c * BC + chunk * 8;
                        const uint32_t bytes = col < a.V ? static_cast<uint32_t>(min(8, a.V - col)) * 2u : 0u;
                        if (!warp_wait(empty(st.slot), st.parity ^ 1u, abort_flag, budget))
                            return false;
                        const uint32_t dst = tiles + st.slot * S::TILE;
#pragma unroll
                        for (int i = 0; i < ROWS; ++i)   // zeros past the row's end and past the step's last row
                            if (r0 + EACH * i < padded)
                                cp_async16(dst + place(r0 + EACH * i), row[i] && bytes ? row[i] + c * BC : dy, row[i] ? bytes : 0u);
                        cp_async_arrive(full(st.slot));
                        st.next();
                    }
                }
                return true;
            });
            asm volatile("cp.async.wait_all;" ::: "memory");   // no copy is in flight when the CTA leaves
        } else {
            // Half a warp has a row of the staging ring, brings it in whole 16-byte pieces and
            // rewrites it, so that no warp waits for another; a batch is 32 NR rows, and up to
            // BATCHES are on their way.
            constexpr int NR = S::NR;
            static_assert(EACH == 32, "half a warp a row of 32");
            struct Cursor {   // batch `part` (rows 32 NR part ..) of the tile (p, c) of an adapter
                int ad = -1, p = 0, e = 0, c = 0, part = 0;
                __device__ __forceinline__ bool seek(const AdapterGradArgs &a)
                {
                    while (++ad < a.n) {
                        const Part r(a.plan.offsets[ad], a.plan.offsets[ad + 1], a.p0, a.p1);
                        p = r.begin;
                        e = r.end;
                        if (p < e)
                            return true;
                    }
                    return false;
                }
                __device__ __forceinline__ int rows() const { return min(STEP, e - p); }
                __device__ __forceinline__ bool last() const { return (part + 1) * 32 * S::NR >= rows(); }
                __device__ __forceinline__ bool next(const AdapterGradArgs &a, int blocks)
                {
                    if (!last()) {
                        ++part;
                        return true;
                    }
                    part = 0;
                    if (++c < blocks)
                        return true;
                    c = 0;
                    p += STEP;
                    return p < e || seek(a);
                }
            };
            constexpr int ES = static_cast<int>(sizeof(T)), P = ES / 2;   // 16-byte pieces of a thread's eight columns
            auto staged = [&](int batch, int i) { return staging + static_cast<uint32_t>(((batch * NR + i) * 32 + r0) * S::SROW); };
            Cursor head;
            bool more = head.seek(a);
            Cursor tail = head;
            bool left = more;
            Ring st(S::STAGES), in(S::BATCHES), out(S::BATCHES);
            uint32_t shifts = 0;   // a nibble a row, the latest lowest: its bytes past a 16-byte boundary
            auto ask = [&] {       // for the pieces of the head's batch
                uint32_t bits = 0;
                if (more) {
                    if (head.c == 0 && head.part == 0)
                        look_up(head.p, head.rows());
                    const int col = c0 + head.c * BC;
#pragma unroll
                    for (int i = 0; i < NR; ++i) {
                        const T *from = row[i];
#pragma unroll
                        for (int k = 1; k < ROWS / NR; ++k)
                            from = head.part == k ? row[k * NR + i] : from;
                        if (!from || col >= a.V)
                            continue;
                        from += head.c * BC;   // the tile's first column of the row
                        const uint32_t shift = HOW == ANY ? row_shift(from) : 0u;
                        bits |= shift << (4 * i);
                        const char *src = reinterpret_cast<const char *>(from) - shift;
                        const uint32_t dst = staged(in.slot, i);
                        // columns of piece k of the tile: first .. first + 16 / ES - 1
                        auto bring = [&](int k) {
                            const int first = col + (16 * k - static_cast<int>(shift)) / ES;
                            if (first >= 0 && first + 16 / ES <= a.V) {
                                cp_async16(dst + 16 * k, src + 16 * k, 16u);
                            } else {   // a row's ends, one by one
                                for (int x = 0; x < 16 / ES; ++x)
                                    if (first + x >= 0 && first + x < a.V)
                                        reinterpret_cast<T *>(smem + (dst - tiles) + 16 * k)[x] = reinterpret_cast<const T *>(src + 16 * k)[x];
                            }
                        };
#pragma unroll
                        for (int k = 0; k < P; ++k)
                            bring(k * 16 + chunk);
                        if (HOW == ANY && chunk == 0 && shift != 0)
                            bring(P * 16);
                    }
                    more = head.next(a, blocks);
                }
                asm volatile("cp.async.commit_group;" ::: "memory");
                shifts = shifts << (4 * NR) | bits;
                in.next();
            };
            for (int i = 0; i < S::BATCHES - 1; ++i)
                ask();
            while (left) {
                ask();
                asm volatile("cp.async.wait_group %0;" ::"n"(S::BATCHES - 1) : "memory");
                __syncwarp();   // every lane's pieces of the warp's rows
                const int rows = tail.rows(), padded = (rows + 15) / 16 * 16, col = c0 + tail.c * BC + chunk * 8;
                if (tail.part == 0 && !warp_wait(empty(st.slot), st.parity ^ 1u, abort_flag, budget))
                    break;
#pragma unroll
                for (int i = 0; i < NR; ++i) {
                    const int m = (tail.part * NR + i) * 32 + r0;
                    if (m >= padded)
                        continue;
                    uint32_t o[S::PLANES][4] = {};
                    if (m < rows && col < a.V) {
                        constexpr int W = Elem<T>::WORDS;
                        uint32_t x[W + 4] = {};
                        const uint4 *in_row = reinterpret_cast<const uint4 *>(smem + (staged(out.slot, i) - tiles)) + chunk * P;
#pragma unroll
                        for (int k = 0; k < P + (HOW == ANY ? 1 : 0); ++k) {
                            const uint4 v = in_row[k];
                            x[4 * k] = v.x;
                            x[4 * k + 1] = v.y;
                            x[4 * k + 2] = v.z;
                            x[4 * k + 3] = v.w;
                        }
                        Raw8<T> w;
                        if (HOW == ANY) {
                            shift_words<W, ES == 2>(w.w, x, shifts >> (4 * (NR * (S::BATCHES - 1) + i)) & 15u);
                        } else {
#pragma unroll
                            for (int k = 0; k < W; ++k)
                                w.w[k] = x[k];
                        }
                        float v[8];
#pragma unroll
                        for (int k = 0; k < 8; ++k)
                            v[k] = Elem<T>::get(w.w, k);
                        if (col + 8 > a.V) {
#pragma unroll
                            for (int k = 0; k < 8; ++k)
                                v[k] = col + k < a.V ? v[k] : 0.f;
                        }
                        split8<S::PLANES>(v, o);
                    }
#pragma unroll
                    for (int j = 0; j < S::PLANES; ++j)
                        *reinterpret_cast<uint4 *>(smem + st.slot * S::TILE + place(j * STEP + m)) =
                            make_uint4(o[j][0], o[j][1], o[j][2], o[j][3]);
                }
                __syncwarp();   // the rows have been read, the tile's part is written
                if (tail.last()) {
                    if (lane == 0)
                        mbar_arrive(full(st.slot));
                    st.next();
                }
                out.next();
                left = tail.next(a, blocks);
            }
            asm volatile("cp.async.wait_all;" ::: "memory");
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 1)
        tmem_dealloc(tmem, S::TMEM);
    if (tid == 0 && *abort_flag)
        atomicCAS(a.status, 0, static_cast<int>(TIM_ERR_TIMEOUT));
}

// ---------------------------------------------------------------- fold
// du of a part's positions, ranks r0 .. r0 + RP - 1: the slabs' parts added in slab
// order by 16 threads (slabs k, k + 16, ... each, then joined in order), times scale,
// in three bf16 parts.  Bound by its loads: 143 slabs x 4096 positions
// x 16 ranks, 37 MB, 11 us.
template <int RP> __global__ void __launch_bounds__(256) adapters_fold_kernel(const AdapterGradArgs a)
{
    constexpr int SHARE = 16, ITEMS = 256 / SHARE;
    __shared__ float4 sums[SHARE][ITEMS];
    const int item = threadIdx.x % ITEMS, k = threadIdx.x / ITEMS;
    const int64_t count = a.p1 - a.p0 + 16;   // a part may end up to 15 positions past p1
    const int64_t i = (static_cast<int64_t>(blockIdx.x) * ITEMS + item);   // four ranks of a position, positions side by side
    pdl_wait();
    pdl_launch_dependents();
    const int pos = a.p0 + static_cast<int>(i % count), r = static_cast<int>(i / count) * 4;
    int ad = a.n;
    if (i < count * (RP / 4) && pos < a.N) {
        ad = a.plan.adapter[pos];
        if (ad < a.n) {
            const Part in(a.plan.offsets[ad], a.plan.offsets[ad + 1], a.p0, a.p1);
            ad = pos >= in.begin && pos < in.end ? ad : a.n;
        }
    }
    const bool on = ad < a.n;
    float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
    if (on) {
        const float4 *p = reinterpret_cast<const float4 *>(a.partial) + i;
#pragma unroll 4
        for (int slab = k; slab < a.du_parts; slab += SHARE) {
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
    const float scale = a.scale ? a.scale[ad] : 1.f;
    uint16_t x0[3], x1[3], x2[3], x3[3];
    split_bf16<3>(s.x * scale, x0);
    split_bf16<3>(s.y * scale, x1);
    split_bf16<3>(s.z * scale, x2);
    split_bf16<3>(s.w * scale, x3);
    TIM_DCHECK(a.r0 + r + 4 <= a.RT, a.status, TIM_CHECK_STORE, pos, a.r0 + r);
    uint16_t *du = a.du + static_cast<size_t>(pos) * (3 * a.RT) + a.r0 + r;
#pragma unroll
    for (int j = 0; j < 3; ++j)
        *reinterpret_cast<uint2 *>(du + j * a.RT) =
            make_uint2(x0[j] | static_cast<uint32_t>(x1[j]) << 16, x2[j] | static_cast<uint32_t>(x3[j]) << 16);
}

// ---------------------------------------------------------------- dA
// dA of an adapter, 128 columns of D from 128 x on, by a CTA; a warp has 16 of them for
// all ranks.  Rows in chunks of 64 (gathered in the plan's order) by asynchronous copies
// into a ring of three stages.  With dh in one launch: 4096 x 4096, rank 16 of 8 adapters, 30 us
// (two launches 41); tensor pipes 21 %, an adapter's chunks one after the other.
template <int RT> struct DaShape {
    static constexpr int ROWS = 64, COLS = 128, STAGES = 3;
    static constexpr int HROW = COLS * 2 + 16, UROW = 3 * RT * 2 + 16;   // padded: no bank twice
    static constexpr int STAGE = ROWS * (HROW + UROW), BYTES = STAGES * STAGE;
    static_assert(BYTES >= RT * 528, "dh's slab of A lies there too");
};

template <int RT> __device__ __forceinline__ void dA_part(const AdapterGradArgs &a, int column_block, int ad, uint8_t *ring)
{
    using S = DaShape<RT>;
    constexpr int ROWS = S::ROWS, COLS = S::COLS, HROW = S::HROW, UROW = S::UROW, RM = RT / 16;
    const uint32_t ring0 = smem_u32(ring);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, q = lane & 3;
    const int d0 = column_block * COLS;
    const int b = a.plan.offsets[ad], e = a.plan.offsets[ad + 1];
    if (b == e && a.accumulate)
        return;
    float acc[RM][2][4] = {};
    const int hc = tid % 16 * 8;   // this thread's piece of rows tid / 16, tid / 16 + 16, .. of a chunk
    int row[ROWS / 16];
    auto look_up = [&](int p) {
#pragma unroll
        for (int i = 0; i < ROWS / 16; ++i) {
            const int at = p + tid / 16 + i * 16;
            row[i] = at < e ? a.plan.perm[at] : -1;
            TIM_DCHECK(row[i] < a.N && (at >= e || row[i] >= 0), a.status, TIM_CHECK_UNIT, at, row[i]);
        }
    };
    auto fill = [&](int stage, int p) {
        const uint32_t h0 = ring0 + stage * S::STAGE, u0 = h0 + ROWS * HROW;
        if (p < e) {
#pragma unroll
            for (int i = 0; i < ROWS / 16; ++i) {
                const bool on = row[i] >= 0 && d0 + hc < a.D;
                cp_async16(h0 + (tid / 16 + i * 16) * HROW + hc * 2, a.h + (on ? static_cast<size_t>(row[i]) * a.D + d0 + hc : 0), on ? 16u : 0u);
            }
            for (int i = tid; i < ROWS * (3 * RT / 8); i += 256) {
                const int m = i / (3 * RT / 8), c = i % (3 * RT / 8) * 8;
                const bool on = p + m < e;
                cp_async16(u0 + m * UROW + c * 2, a.du + (on ? static_cast<size_t>(p + m) * (3 * RT) + c : 0), on ? 16u : 0u);
            }
            look_up(p + ROWS);
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
    look_up(b);
    for (int i = 0; i < S::STAGES - 1; ++i)
        fill(i, b + i * ROWS);
    int stage = 0;
    for (int p = b; p < e; p += ROWS) {
        asm volatile("cp.async.wait_group %0;" ::"n"(S::STAGES - 2) : "memory");
        __syncthreads();   // the chunk is there; the one before has been read
        fill(stage == 0 ? S::STAGES - 1 : stage - 1, p + (S::STAGES - 1) * ROWS);
        const uint32_t h0 = ring0 + stage * S::STAGE, u0 = h0 + ROWS * HROW;
        // a chunk's sums by themselves, then added: the tensor cores cut, rather than round,
        // what they add up, and a long chain of that leans to one side
        uint32_t x[ROWS / 16][4];   // k = rows, n = the warp's 16 columns
#pragma unroll
        for (int k = 0; k < ROWS / 16; ++k)
            ldsm4t(x[k], h0 + (k * 16 + (lane & 15)) * HROW + (warp * 16 + (lane >> 4) * 8) * 2);
#pragma unroll
        for (int m = 0; m < RM; ++m) {
            float part[2][4] = {};
#pragma unroll
            for (int i = 2; i >= 0; --i)   // the smallest first, so that they are not cut off the large sum
#pragma unroll
                for (int k = 0; k < ROWS / 16; ++k) {
                    uint32_t u[4];   // ranks as rows
                    ldsm4t(u, u0 + (k * 16 + (lane & 7) + (lane >> 4) * 8) * UROW + (i * RT + m * 16 + ((lane >> 3) & 1) * 8) * 2);
                    mma16816(part[0], u, x[k][0], x[k][1]);
                    mma16816(part[1], u, x[k][2], x[k][3]);
                }
#pragma unroll
            for (int j = 0; j < 2; ++j)
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    acc[m][j][k] += part[j][k];
        }
        stage = stage + 1 == S::STAGES ? 0 : stage + 1;
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
// dh in 256 columns (a warp 32) of row_chunk positions, by a CTA; the
// adapter's A slab is in registers while the rows' adapter is the same, and the next 16
// rows' du is on its way while the products of the 16 before are written.  A lane has
// four neighbouring ranks (8 bytes) of du where the product's order of k is two pairs; A's
// rows are taken in the same order.
template <int RT> __device__ __forceinline__ void dh_part(const AdapterGradArgs &a, int column_block, int64_t chunk, uint8_t *as)
{
    constexpr int COLS = 256, AROW = COLS * 2 + 16, KS = RT / 16;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, q = lane & 3;
    const int d0 = column_block * COLS, dw = d0 + warp * 32;
    const int live = a.plan.offsets[a.n];
    const int p0 = static_cast<int>(chunk * a.row_chunk), p1 = min(a.N, p0 + a.row_chunk);
    const uint32_t a0 = smem_u32(as);
    const int kr = lane & 15;   // k of the lane's row address: 2 q + i is rank 4 q + i, 2 q + 8 + i is 4 q + 2 + i
    const int rank = (kr & 7) / 2 * 4 + (kr & 1) + (kr >= 8 ? 2 : 0);
    for (int p = p0; p < min(p1, live);) {   // adapter by adapter
        const int ad = a.plan.adapter[p];
        const int e = min(p1, a.plan.offsets[ad + 1]);
        uint2 u[3][KS][2];   // rows g and g + 8
        int row[2];
        auto fetch = [&](int at) {
#pragma unroll
            for (int half = 0; half < 2; ++half) {
                const int i = at + g + half * 8;
                row[half] = i < e ? a.plan.perm[i] : -1;
                TIM_DCHECK(row[half] < a.N && (i >= e || row[half] >= 0), a.status, TIM_CHECK_STORE, i, row[half]);
#pragma unroll
                for (int part = 0; part < 3; ++part)
#pragma unroll
                    for (int k = 0; k < KS; ++k)
                        u[part][k][half] = i < e ? *reinterpret_cast<const uint2 *>(a.du + static_cast<size_t>(i) * (3 * RT) +
                                                                                     part * RT + k * 16 + 4 * q)
                                                 : make_uint2(0u, 0u);
            }
        };
        if (KS <= 4)
            fetch(p);
        __syncthreads();
        for (int i = tid; i < RT * (COLS / 8); i += 256) {
            const int r = i / (COLS / 8), c = i % (COLS / 8) * 8;
            const bool on = r < a.R && d0 + c < a.D;
            *reinterpret_cast<uint4 *>(as + r * AROW + c * 2) =
                on ? __ldg(reinterpret_cast<const uint4 *>(a.A + (static_cast<size_t>(ad) * a.R + r) * a.D + d0 + c))
                   : make_uint4(0u, 0u, 0u, 0u);
        }
        __syncthreads();
        uint32_t w[KS][4][2];
#pragma unroll
        for (int k = 0; k < KS; ++k)
#pragma unroll
            for (int j = 0; j < 4; j += 2) {
                uint32_t x[4];
                ldsm4t(x, a0 + (k * 16 + rank) * AROW + (warp * 32 + j * 8 + (lane >> 4) * 8) * 2);
                w[k][j][0] = x[0];
                w[k][j][1] = x[1];
                w[k][j + 1][0] = x[2];
                w[k][j + 1][1] = x[3];
            }
        for (; p < e; p += 16) {
            if (KS > 4)   // no room for the next ones
                fetch(p);
            float acc[4][4] = {};
#pragma unroll
            for (int part = 2; part >= 0; --part)   // the smallest first
#pragma unroll
                for (int k = 0; k < KS; ++k)
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        mma16816(acc[j], {u[part][k][0].x, u[part][k][1].x, u[part][k][0].y, u[part][k][1].y}, w[k][j][0], w[k][j][1]);
            const int to[2] = {row[0], row[1]};
            if (KS <= 4 && p + 16 < e)
                fetch(p + 16);
#pragma unroll
            for (int half = 0; half < 2; ++half) {
                if (to[half] < 0)
                    continue;
                float *out = a.dh + static_cast<size_t>(to[half]) * a.D;
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const int d = dw + j * 8 + 2 * q;
                    if (d >= a.D)
                        continue;
                    float2 *o = reinterpret_cast<float2 *>(out + d);
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

// Both, which wait for du alone: the first CTAs dA (fewer, and longer), the others dh.
template <int RT> __global__ void __launch_bounds__(256) adapters_outer_kernel(const AdapterGradArgs a)
{
    extern __shared__ __align__(16) uint8_t shared[];
    const int blocks_a = (a.D + 127) / 128, blocks_h = (a.D + 255) / 256;
    const int64_t first_h = static_cast<int64_t>(blocks_a) * a.n;
    pdl_wait();
    pdl_launch_dependents();
    if (blockIdx.x < first_h)
        dA_part<RT>(a, static_cast<int>(blockIdx.x % blocks_a), static_cast<int>(blockIdx.x / blocks_a), shared);
    else
        dh_part<RT>(a, static_cast<int>((blockIdx.x - first_h) % blocks_h), (blockIdx.x - first_h) / blocks_h, shared);
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

// The gradient's launch; maps = null: the kernel's shared memory is granted instead.
template <typename T, int HOW, int RP> cudaError_t grad(const CUtensorMap *maps, const AdapterGradArgs &a, cudaStream_t s)
{
    using S = Shape<T, HOW, RP>;
    auto kernel = adapters_grad_kernel<T, HOW, RP>;
    if (!maps)
        return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, S::BYTES);
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1] = {pdl_attribute()};
    cfg.gridDim = dim3(static_cast<unsigned>(a.slabs), 1, 1);
    cfg.blockDim = dim3(S::THREADS, 1, 1);
    cfg.dynamicSmemBytes = S::BYTES;
    cfg.stream = s;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, maps[0], maps[1], a);
}

template <int RP> cudaError_t grad(const CUtensorMap *maps, const AdapterGradArgs &a, int dtype, bool aligned, cudaStream_t s)
{
    if (dtype == TIM_F32)
        return aligned ? grad<float, LOAD, RP>(maps, a, s) : grad<float, ANY, RP>(maps, a, s);
    if (dtype == TIM_F16)
        return aligned ? grad<__half, LOAD, RP>(maps, a, s) : grad<__half, ANY, RP>(maps, a, s);
    return aligned ? grad<__nv_bfloat16, COPY, RP>(maps, a, s) : grad<__nv_bfloat16, ANY, RP>(maps, a, s);
}

template <int RP> cudaError_t prepare()
{
    const AdapterGradArgs a{};
    cudaError_t e = cudaSuccess;
    for (int dtype : {TIM_F32, TIM_F16, TIM_BF16})
        for (bool aligned : {true, false})
            if (e == cudaSuccess)
                e = grad<RP>(nullptr, a, dtype, aligned, nullptr);
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
    auto set = [&](auto kernel, int bytes) {
        if (e == cudaSuccess)
            e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    };
    set(adapters_outer_kernel<16>, DaShape<16>::BYTES);
    set(adapters_outer_kernel<32>, DaShape<32>::BYTES);
    set(adapters_outer_kernel<64>, DaShape<64>::BYTES);
    set(adapters_outer_kernel<128>, DaShape<128>::BYTES);
    return e;
}

cudaError_t adapters_grad_launch(const CUtensorMap (&maps)[2], AdapterGradArgs a, int dtype, int num_sms, cudaStream_t s)
{
    const int RP = std::min(a.RT, 64);
    for (int64_t p0 = 0; p0 < a.N; p0 += a.row_part)
        for (a.r0 = 0; a.r0 < a.R; a.r0 += RP) {
            a.p0 = static_cast<int32_t>(p0);
            a.p1 = static_cast<int32_t>(std::min<int64_t>(a.N, p0 + a.row_part));
            cudaError_t e = RP == 16   ? grad<16>(maps, a, dtype, a.aligned, s)
                            : RP == 32 ? grad<32>(maps, a, dtype, a.aligned, s)
                                       : grad<64>(maps, a, dtype, a.aligned, s);
            if (e != cudaSuccess)
                return e;
            const int64_t items = static_cast<int64_t>(a.p1 - a.p0 + 16) * (RP / 4);
            const dim3 grid(static_cast<unsigned>((items + 15) / 16));
            e = RP == 16   ? launch(adapters_fold_kernel<16>, grid, 256, 0, a, s)
                : RP == 32 ? launch(adapters_fold_kernel<32>, grid, 256, 0, a, s)
                           : launch(adapters_fold_kernel<64>, grid, 256, 0, a, s);
            if (e != cudaSuccess)
                return e;
        }
    const int64_t columns = (a.D + 255) / 256;
    int64_t chunk = 128;
    while (chunk > 16 && columns * ((a.N + chunk - 1) / chunk) < 4 * num_sms)
        chunk /= 2;
    a.row_chunk = static_cast<int32_t>(chunk);
    const dim3 grid(static_cast<unsigned>((a.D + 127) / 128 * static_cast<int64_t>(a.n) + columns * ((a.N + chunk - 1) / chunk)));
    switch (a.RT) {
    case 16: return launch(adapters_outer_kernel<16>, grid, 256, DaShape<16>::BYTES, a, s);
    case 32: return launch(adapters_outer_kernel<32>, grid, 256, DaShape<32>::BYTES, a, s);
    case 64: return launch(adapters_outer_kernel<64>, grid, 256, DaShape<64>::BYTES, a, s);
    default: return launch(adapters_outer_kernel<128>, grid, 256, DaShape<128>::BYTES, a, s);
    }
}

} // namespace tim
