// logits_process.cu -- the sampler's rules on a head's logits: the processed
// logits themselves, the chosen token's log-probability under them, and its
// gradient with respect to the raw logits.
//
// For row i and column v, with c the number of times v is among the row's
// generated tokens (history from the spans' second entry on) and "seen" if v is
// anywhere in the row's history:
//   x = z + bias_v                               (0 where the row has no bias for v)
//   x = x > 0 ? x / rho : x rho                  if seen
//   x = x - alpha_f c - alpha_p                  if c > 0
//   y = x / tau,  y = -inf where the row's grammar does not allow v.
// logp_a = y_a - lse(y); d logp_a / d z_v = (1[v = a] - e^(y_v - lse)) dy_v/dz_v
// with dy/dz = (1 / tau) (1, 1 / rho or rho), and 0 where y = -inf.
//
// What bounds it: every operation streams the row (and its mask, V / 8 bytes)
// once; only the few touched columns (history and biased ids) need more.  So the
// columns are streamed as if none were touched, and a table in shared memory
// holds the touched ones: a bitmap of the CTA's columns, the number of bits
// before each group of four of its words, and an entry per touched column, in column
// order.  Building it takes two scans of the row's history (set the bits; count
// with shared-memory integer atomics, which have no order) and one gather per
// distinct id; no sort, no hash, any history length (where more columns are touched
// than a table holds, the columns are handled in halves).  The log-probability takes
// the touched columns out of the stream and adds the table's entries of the same
// slice; the others write their columns first and the touched ones over them.
//
// Measured on a GB300 against the bytes each has to move at 6760 GB/s (inputs not in L2):
//   process   512 x 151936 bf16, histories of 1000 tokens   79 us of 47 us: the tables
//             (86 us in place, fp32 126 us of 93 us, bf16 to fp32 106 us of 70 us)
//   process   64 x 128256 bf16 -> fp32, half under a grammar 26 us of 7 us: one table's
//             chain of loads and barriers (rules, history, counts, gathers), then the stream
//   logprob   8192 x 151936 bf16, packed sequences of 512   439 us of 368 us: issue slots
//             (6 instructions a column for the sum, 3 more for table and touched columns)
//             (fp32 1024 x 129280 110 us of 78 us: registers, see launch_logp)
//   gradient  4096 x 128256 bf16, a quarter under a grammar 341 us of 313 us: memory
//             (371 us in place; fp32 1024 x 129280 165 us of 157 us)
#include <algorithm>

#include "logits_rows.cuh"

namespace tim {
namespace {

// A table entry while it is counted: seen in the prompt, listed with a bias, and
// the number of times among the generated tokens (the host keeps it below 2^30).
constexpr uint32_t kPrompt = 0x80000000u, kBiased = 0x40000000u, kCount = 0x3fffffffu;

struct RowRules {
    float tau, inv_tau, rho, pres, freq;
    float grad, lse;           // GRAD
    int target;                // LOGP, GRAD
    int h0, hg, h1;            // history span
    int b0, b1;                // bias entries
    const uint8_t *mask;       // the row's bits, or null
    bool bad;
};

// One warp reads a row's scalars for its CTA, each lane one of them: the loads
// overlap (one thread's chain of conditional loads cost 6 us a row).
__device__ __forceinline__ void read_rules(const ProcArgs &a, int row, RowRules &out)
{
    const int lane = threadIdx.x & 31;
    const void *p = nullptr;
    int64_t at = row;
    uint32_t v = 0;
    switch (lane) {
    case 0: p = a.temperature; v = 0x3f800000u; break;
    case 1: p = a.repetition; v = 0x3f800000u; break;
    case 2: p = a.presence; break;
    case 3: p = a.frequency; break;
    case 4: p = a.grad; break;
    case 5: p = a.lse; break;
    case 6: p = a.targets; v = 0xffffffffu; break;
    case 7: p = a.allowed_rows; v = a.allowed ? static_cast<uint32_t>(row) : 0xffffffffu; break;
    case 8: p = a.bias_offsets; break;
    case 9: p = a.bias_offsets; at = static_cast<int64_t>(row) + 1; break;
    case 10: case 11: case 12: p = a.spans; at = static_cast<int64_t>(row) * 3 + (lane - 10); break;
    default: break;
    }
    if (p)
        v = static_cast<const uint32_t *>(p)[at];
    auto f = [&](int k) { return __uint_as_float(__shfl_sync(0xffffffffu, v, k)); };
    auto i = [&](int k) { return static_cast<int>(__shfl_sync(0xffffffffu, v, k)); };
    RowRules r;
    r.tau = f(0);
    r.rho = f(1);
    r.pres = f(2);
    r.freq = f(3);
    r.grad = f(4);
    r.lse = f(5);
    r.target = i(6);
    int m = i(7);
    r.b0 = i(8);
    r.b1 = i(9);
    r.h0 = i(10);
    r.hg = i(11);
    r.h1 = i(12);
    r.inv_tau = 1.f / r.tau;
    r.bad = !(r.tau > 0.f) || !isfinite(r.tau) || !isfinite(r.inv_tau) || !(r.rho > 0.f) || !isfinite(r.rho) ||
            !isfinite(1.f / r.rho) || !isfinite(r.pres) || !isfinite(r.freq);
    if (r.h0 < 0 || r.hg < r.h0 || r.h1 < r.hg || r.h1 > a.history_len) {
        r.bad = true;
        r.h0 = r.hg = r.h1 = 0;
    }
    if (r.b0 < 0 || r.b1 < r.b0 || r.b1 > a.num_bias || r.b1 - r.b0 > a.V) {
        r.bad = true;
        r.b0 = r.b1 = 0;
    }
    if (a.allowed && m >= a.num_allowed) {
        r.bad = true;
        m = -1;
    }
    r.mask = a.allowed && m >= 0 ? reinterpret_cast<const uint8_t *>(a.allowed + m * a.allowed_ld) : nullptr;
    if (lane == 0)
        out = r;
}

__device__ __forceinline__ bool is_allowed(const uint8_t *mask, int id)
{
    return !mask || (mask[id >> 3] >> (id & 7) & 1);
}

// A touched column before the temperature: x, and its slope dx/dz.
__device__ __forceinline__ float touched_value(const RowRules &r, float z, float bias, uint32_t word, float &slope)
{
    float x = z + bias;
    slope = 1.f;
    if (word != 0) {
        slope = x > 0.f ? 1.f / r.rho : r.rho;
        x = x > 0.f ? x / r.rho : x * r.rho;
    }
    const uint32_t c = word & kCount;
    if (c != 0)
        x = x - r.freq * static_cast<float>(c) - r.pres;
    return x;
}

// ---------------------------------------------------------------- touched columns
template <typename C> struct Table {
    uint32_t *value;     // [cap]: counts, then the column's replacement (fp32 bits)
    uint32_t *bitmap;    // [columns / 32]
    uint16_t *before;    // [columns / 128]: bits set in the four-word groups before
    C *column;           // [cap]: relative to the table's first
    int *bad;            // a bias list that breaks its limits
    int cap;
    int groups, used;    // of the columns in hand
};

// Bytes of a table over `columns` columns (a multiple of 1024).
template <typename C> __host__ __device__ inline size_t table_bytes(int columns, int cap)
{
    return static_cast<size_t>(cap) * (4 + sizeof(C)) + columns / 8 + columns / 64 + 16;
}

template <typename C> __device__ __forceinline__ Table<C> carve(uint32_t *smem, int columns, int cap)
{
    Table<C> t;
    t.cap = cap;
    t.value = smem;
    t.bitmap = smem + cap;
    t.before = reinterpret_cast<uint16_t *>(t.bitmap + columns / 32);
    t.column = reinterpret_cast<C *>(t.before + columns / 128);
    t.bad = reinterpret_cast<int *>(t.column + cap);
    t.groups = t.used = 0;
    return t;
}

// Entry of column k (relative), whose bit is set.
template <typename C> __device__ __forceinline__ int rank_of(const Table<C> &t, unsigned k)
{
    const uint4 w = reinterpret_cast<const uint4 *>(t.bitmap)[k >> 7];
    const unsigned in = k >> 5 & 3;
    const uint32_t mine = in == 0 ? w.x : in == 1 ? w.y : in == 2 ? w.z : w.w;
    return t.before[k >> 7] + (in > 0 ? __popc(w.x) : 0) + (in > 1 ? __popc(w.y) : 0) + (in > 2 ? __popc(w.z) : 0) +
           __popc(mine & ((1u << (k & 31)) - 1));
}

template <typename C> __device__ __forceinline__ bool is_touched(const Table<C> &t, int k)
{
    return t.bitmap[k >> 5] >> (k & 31) & 1;
}

// f(position, id relative to c0) for the entries ids[j0 .. j1) within [c0, c0 + width);
// four loads at a time, so that a long history does not wait for each.
template <typename F>
__device__ __forceinline__ void scan_ids(int nt, const int32_t *ids, int j0, int j1, int c0, int width, F f)
{
    for (int j = j0 + static_cast<int>(threadIdx.x); j < j1; j += 4 * nt) {
        unsigned k[4];
#pragma unroll
        for (int u = 0; u < 4; ++u)
            k[u] = j + u * nt < j1 ? static_cast<unsigned>(ids[j + u * nt]) - static_cast<unsigned>(c0) : 0xffffffffu;
#pragma unroll
        for (int u = 0; u < 4; ++u)
            if (k[u] < static_cast<unsigned>(width))
                f(j + u * nt, k[u]);
    }
}

// Empties the table for `width` columns: the first nt threads; a barrier before use.
template <typename C> __device__ __forceinline__ void clear_table(int nt, Table<C> &t, int width)
{
    const uint4 zero = make_uint4(0u, 0u, 0u, 0u);
    t.groups = (width + 127) / 128;
    for (int j = threadIdx.x; j < t.groups; j += nt)
        reinterpret_cast<uint4 *>(t.bitmap)[j] = zero;
    if (threadIdx.x == 0)
        *t.bad = 0;
}

// Builds the cleared table of columns c0 .. c0 + width - 1 with replacement(id, x,
// slope) for each.  The CTA's first nt threads (whole warps), which meet at
// barrier 1, and the same answer in all: kBad where the row's bias ids are out of range or order, kFull
// where more columns are touched than the table holds (never for a width up to its
// capacity).  Ends with a barrier.
enum TableState { kBuilt, kBad, kFull };

template <typename T, typename C, typename F>
__device__ __forceinline__ TableState build_table(int nt, const ProcArgs &a, const RowRules &r, const T *z, int c0, int width, Table<C> &t,
                                  F replacement)
{
    __shared__ int warp_bits[LP_WARPS];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    auto mark = [&](int, unsigned k) { atomicOr(t.bitmap + (k >> 5), 1u << (k & 31)); };
    scan_ids(nt, a.history, r.h0, r.h1, c0, width, mark);
    bool bad = false;
    for (int j = r.b0 + static_cast<int>(threadIdx.x); j < r.b1; j += nt) {
        const int id = a.bias_ids[j];
        bad |= id < 0 || id >= a.V || (j > r.b0 && a.bias_ids[j - 1] >= id);
        const unsigned k = static_cast<unsigned>(id) - static_cast<unsigned>(c0);
        if (k < static_cast<unsigned>(width))
            mark(j, k);
    }
    if (bad)
        *t.bad = 1;
    named_sync(1, nt);
    if (*t.bad)
        return kBad;
    // bits before each group of four words: a run of groups per thread
    const uint4 *groups = reinterpret_cast<const uint4 *>(t.bitmap);
    const int run = (t.groups + nt - 1) / nt;
    const int q0 = min(t.groups, static_cast<int>(threadIdx.x) * run), q1 = min(t.groups, q0 + run);
    auto bits_of = [&](int q) {
        const uint4 w = groups[q];
        return __popc(w.x) + __popc(w.y) + __popc(w.z) + __popc(w.w);
    };
    int bits = 0;
    for (int q = q0; q < q1; ++q)
        bits += bits_of(q);
    int upto = bits;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const int v = __shfl_up_sync(0xffffffffu, upto, d);
        upto += lane >= d ? v : 0;
    }
    if (lane == 31)
        warp_bits[warp] = upto;
    named_sync(1, nt);
    int base = upto - bits;
    t.used = 0;
#pragma unroll
    for (int w = 0; w < LP_WARPS; ++w) {
        const int n = w < nt / 32 ? warp_bits[w] : 0;
        base += w < warp ? n : 0;
        t.used += n;
    }
    if (t.used > t.cap) {
        named_sync(1, nt);   // warp_bits is written again
        return kFull;
    }
    for (int q = q0; q < q1; ++q) {
        t.before[q] = static_cast<uint16_t>(base);
        base += bits_of(q);
    }
    for (int n = threadIdx.x; n < t.used; n += nt)
        t.value[n] = 0;
    named_sync(1, nt);
    scan_ids(nt, a.history, r.h0, r.h1, c0, width, [&](int j, unsigned k) {
        const int n = rank_of(t, k);
        t.column[n] = static_cast<C>(k);   // the same from every token with this id
        if (j >= r.hg)
            atomicAdd(t.value + n, 1u);
        else
            atomicOr(t.value + n, kPrompt);
    });
    scan_ids(nt, a.bias_ids, r.b0, r.b1, c0, width, [&](int, unsigned k) {
        const int n = rank_of(t, k);
        t.column[n] = static_cast<C>(k);
        atomicOr(t.value + n, kBiased);
    });
    named_sync(1, nt);
    auto finish = [&](int n, int id, float logit, float bias) {
        float slope;
        float x = touched_value(r, logit, bias, t.value[n] & ~kBiased, slope);
        if (!is_allowed(r.mask, id))
            x = neg_inf();
        t.value[n] = __float_as_uint(replacement(id, x, slope));
    };
    for (int n = threadIdx.x; n < t.used; n += 2 * nt) {
        const int n1 = n + nt;
        const bool in0 = !(t.value[n] & kBiased), in1 = n1 < t.used && !(t.value[n1] & kBiased);
        const int id0 = c0 + t.column[n], id1 = in1 ? c0 + t.column[n1] : 0;
        const float z0 = in0 ? Elem<T>::load(z + id0) : 0.f, z1 = in1 ? Elem<T>::load(z + id1) : 0.f;
        if (in0)
            finish(n, id0, z0, 0.f);
        if (in1)
            finish(n1, id1, z1, 0.f);
    }
    named_sync(1, nt);
    if (r.b1 > r.b0) {   // the biased ones, by their bias entry
        scan_ids(nt, a.bias_ids, r.b0, r.b1, c0, width, [&](int j, unsigned k) {
            const int id = c0 + static_cast<int>(k);
            finish(rank_of(t, k), id, Elem<T>::load(z + id), a.bias_values[j]);
        });
        named_sync(1, nt);
    }
    return kBuilt;
}

// Half as many columns, in whole slices.
__device__ __forceinline__ int half(int columns) { return (columns / 2 + LG_SLICE - 1) / LG_SLICE * LG_SLICE; }

// ---------------------------------------------------------------- kernels
// WRITE and GRAD: one CTA per (row, segment); no column depends on another.  Its
// first nb threads build the table while the others stream the columns (512 at a
// time, claimed from a counter), then join them; the touched columns go over the
// streamed ones at the end.  In place the table, which reads the touched logits,
// comes first, and the others wait for it.  nb is half of the threads where the stream
// hides the table, all where a segment is short or the row's history long.  All / half,
// processing 512 rows of 151936 bf16 (50 slices a segment): histories of some 400 tokens
// 69.2 / 64.1 us, 3500 92.8 / 87.4 us, 7000 111.5 / 121.6 us, 14000 241 / 333 us; gradient of
// 4096 x 128256 bf16 350 / 344 us; processing 64 rows of 128256 (11 slices) 22.0 / 23.8 us; at
// 17 to 25 slices the two are within 2 %.
//
// A column's x / tau is the same operation whether the column is touched or not, so that
// equal logits stay equal: for fp32 outputs the corrected quotient, for 16-bit ones the
// product with the rounded reciprocal, whose 1.5 units of fp32's last place are nothing
// beside the output's rounding (with the quotient 2048 x 151936 bf16 took 202 us, not 197).
template <typename T, typename TO, int OP, bool TOUCH>
__global__ void __launch_bounds__(LP_MAP_THREADS, LP_MAP_CTAS) process_map_kernel(const ProcArgs a)
{
    constexpr int NT = LP_MAP_THREADS, WARPS = NT / 32;
    static_assert(WARPS <= LP_WARPS);
    extern __shared__ __align__(16) uint32_t smem[];
    __shared__ RowRules r;
    __shared__ HalfMasks masks;
    __shared__ int s_next, s_state, s_used;
    const int row = static_cast<int>(blockIdx.x / static_cast<unsigned>(a.segs));
    const int seg = static_cast<int>(blockIdx.x % static_cast<unsigned>(a.segs));
    const int seg0 = seg * a.seg_slices * LG_SLICE, seg1 = min(a.V, seg0 + a.seg_slices * LG_SLICE);
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const T *z = static_cast<const T *>(a.z) + row * a.ld;
    TO *out = static_cast<TO *>(a.out) + row * a.ldo;
    const uint32_t shift = row_shift(z), shift_out = row_shift(out);
    using C = uint16_t;   // a segment has at most 65536 columns
    Table<C> t = carve<C>(smem, a.table_columns, a.table_cap);
    if (warp == 0)
        read_rules(a, row, r);
    if (sizeof(TO) == 2 && a.allowed)
        masks.fill();
    if constexpr (TOUCH)
        clear_table(NT, t, seg1 - seg0);
    if (threadIdx.x == 0)
        s_next = seg0;
    __syncthreads();
    const int nb = a.seg_slices <= LP_SHORT || r.h1 - r.h0 > LP_LONG ? NT : NT / 2;
    const float inv_tau = r.inv_tau, gi = r.grad * inv_tau;
    const float lse = r.lse == neg_inf() ? -neg_inf() : r.lse;   // an empty row: every probability is 0
    const uint8_t *const mask = r.mask;
    const int target = OP == LP_GRAD ? r.target : -1;
    TIM_DCHECK(threadIdx.x != 0 || seg != 0 || target < a.V, a.status, TIM_CHECK_TARGET, row, target);
    TIM_DCHECK(OP != LP_GRAD || threadIdx.x != 0 || seg != 0 || r.bad || (isfinite(r.grad) && r.lse < INFINITY), a.status,
               TIM_CHECK_BACKWARD_INPUT, row, __float_as_uint(r.lse));

    auto fill = [&](float value) {
        float v[8];
#pragma unroll
        for (int i = 0; i < 8; ++i)
            v[i] = value;
        const Raw8<TO> f = pack8<TO>(v);
        for (int b = seg0 + warp * 256; b < seg1; b += WARPS * 256)
            store8<TO>(out, b + lane * 8, seg1, shift_out, f);
    };
    if (r.bad || (OP == LP_GRAD && r.grad == 0.f)) {
        fill(r.bad ? quiet_nan() : 0.f);
        if (r.bad && threadIdx.x == 0)
            report_bad_input(a.status);
        return;
    }
    const Pair inv2 = pair(inv_tau, inv_tau), tau2 = pair(-r.tau, -r.tau), lse2 = pair(-lse, -lse), e2 = pair(LG_LOG2E, LG_LOG2E), g2 = pair(-gi, -gi);
    auto chunks = [&](int b, int end) {   // columns b .. b + 511
        Raw8<T> raw[2];
        uint32_t drop[2] = {0u, 0u};
        load_chunks<T, 2>(raw, z, b, end, shift);
        if (mask) {
#pragma unroll
            for (int u = 0; u < 2; ++u)
                if (b + u * 256 + lane * 8 < end)
                    drop[u] = ~static_cast<uint32_t>(mask[(b + u * 256 + lane * 8) >> 3]) & 0xffu;
        }
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            float v[8];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const Pair x = get2<T>(raw[u], k);
                if constexpr (OP == LP_WRITE) {
                    if constexpr (sizeof(TO) == 4)
                        quotient2(x, tau2, inv2, v[2 * k], v[2 * k + 1]);
                    else
                        unpair(mul2(x, inv2), v[2 * k], v[2 * k + 1]);
                } else {
                    float lo, hi;
                    unpair(mul2(fma2(x, inv2, lse2), e2), lo, hi);
                    unpair(mul2(pair(prob2(lo), prob2(hi)), g2), v[2 * k], v[2 * k + 1]);
                }
            }
            Raw8<TO> o = pack8<TO>(v);
            if (drop[u])
                drop8<TO>(o, drop[u], masks, OP == LP_WRITE ? Elem<TO>::NEG_INF : 0u);
            store8<TO>(out, b + u * 256 + lane * 8, end, shift_out, o);
        }
    };
    auto stream = [&](int end) {   // until nothing is left to claim below `end`
        int b = 0;
        if (lane == 0)
            b = atomicAdd(&s_next, 512);
        b = __shfl_sync(0xffffffffu, b, 0);
        while (b < end) {
            int next = 0;
            if (lane == 0)
                next = atomicAdd(&s_next, 512);
            chunks(b, end);
            b = __shfl_sync(0xffffffffu, next, 0);
        }
    };
    // an untouched target's one-hot term (read before anything is written)
    float target_v = 0.f;
    const bool target_mine = target >= seg0 && target < seg1 && threadIdx.x == NT - 1;
    if (target_mine) {
        const float x = Elem<T>::load(z + target);
        target_v = is_allowed(mask, target) && x != neg_inf()
                       ? (1.f - prob2(fmaf(x, inv_tau, -lse) * LG_LOG2E)) * gi
                       : 0.f;
    }
    if constexpr (!TOUCH) {
        if (OP == LP_GRAD)
            __syncthreads();   // (in place)
        for (int b = seg0 + warp * 512; b < seg1; b += WARPS * 512)
            chunks(b, seg1);
        if constexpr (OP == LP_GRAD) {
            __syncthreads();
            if (target_mine)
                out[target] = Elem<TO>::from(target_v);
        }
    } else {
        bool streamed = a.in_place == 0;   // the whole segment, along with the first table
        for (int c0 = seg0, c1, width = seg1 - seg0; c0 < seg1;) {
            c1 = min(seg1, c0 + width);
            if (threadIdx.x < nb) {
                const TableState state = build_table(nb, a, r, z, c0, c1 - c0, t, [&](int id, float x, float slope) {
                    const float y = sizeof(TO) == 4 || OP == LP_GRAD ? quotient(x, r.tau, inv_tau) : __fmul_rn(x, inv_tau);
                    if constexpr (OP == LP_GRAD)
                        return y == neg_inf() ? 0.f
                                              : ((id == target ? 1.f : 0.f) - prob2((y - lse) * LG_LOG2E)) *
                                                    (r.grad * (slope / r.tau));
                    else
                        return y;
                });
                if (threadIdx.x == 0) {
                    s_state = state;
                    s_used = t.used;
                }
            }
            if (streamed)
                stream(seg1);
            __syncthreads();
            const int state = s_state, used = s_used;
            if (state == kBad) {
                fill(quiet_nan());
                if (threadIdx.x == 0)
                    report_bad_input(a.status);
                return;
            }
            if (state == kBuilt) {
                if (!streamed) {   // in place: these columns now, after their table
                    stream(c1);
                    __syncthreads();
                }
                if (OP == LP_GRAD && target_mine && target >= c0 && target < c1 && !is_touched(t, target - c0))
                    out[target] = Elem<TO>::from(target_v);
                for (int n = threadIdx.x; n < used; n += NT)
                    out[c0 + t.column[n]] = Elem<TO>::from(__uint_as_float(t.value[n]));
                c0 = c1;
            } else {
                width = half(c1 - c0);
            }
            if (c0 < seg1) {
                __syncthreads();   // the table has been read
                if (threadIdx.x < nb)
                    clear_table(nb, t, min(seg1, c0 + width) - c0);
                if (threadIdx.x == 0 && !streamed)
                    s_next = c0;
                __syncthreads();
            }
        }
    }
}

// LOGP: a cluster per row; each rank reduces seg_slices slices, one warp per
// slice.  The slices' partials go to rank 0's shared memory, which folds them.
template <typename T, bool TOUCH, int NT, int CTAS>
__global__ void __launch_bounds__(NT, CTAS) process_logp_kernel(const ProcArgs a)
{
    constexpr int WARPS = NT / 32;
    extern __shared__ __align__(16) uint32_t smem[];
    __shared__ RowRules r;
    __shared__ HalfMasks masks;
    __shared__ float target_x;
    const int rank = static_cast<int>(blockIdx.x % static_cast<unsigned>(a.segs));
    const int row = static_cast<int>(blockIdx.x / static_cast<unsigned>(a.segs));
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int slices = (a.V + LG_SLICE - 1) / LG_SLICE;
    const int s0 = min(slices, rank * a.seg_slices), s1 = min(slices, s0 + a.seg_slices);
    using C = int32_t;
    Table<C> t = carve<C>(smem, a.table_columns, a.table_cap);
    float2 *part = reinterpret_cast<float2 *>(smem + (TOUCH ? table_bytes<C>(a.table_columns, a.table_cap) / 4 : 0));   // [slices]
    const T *z = static_cast<const T *>(a.z) + row * a.ld;
    const uint32_t shift = row_shift(z);
    if (a.segs > 1)
        cluster_arrive_relaxed();   // waited for before the first store into rank 0's shared memory
    if (warp == 0)
        read_rules(a, row, r);
    if (sizeof(T) == 2 && (TOUCH || a.allowed))
        masks.fill();
    if constexpr (TOUCH)
        clear_table(NT, t, min(LP_TABLE, min(a.V, s1 * LG_SLICE) - s0 * LG_SLICE));
    __syncthreads();
    bool bad = r.bad;
    const float inv_tau = r.inv_tau, k2 = LG_LOG2E * inv_tau;
    const uint8_t *const mask = r.mask;
    const int target = r.target;
    TIM_DCHECK(threadIdx.x != 0 || rank != 0 || target < a.V, a.status, TIM_CHECK_TARGET, row, target);
    const bool has_target = target >= s0 * LG_SLICE && target < min(a.V, s1 * LG_SLICE);
    if (has_target && threadIdx.x == NT - 1)
        target_x = is_allowed(mask, target) ? Elem<T>::load(z + target) : neg_inf();
    for (int f0 = s0, f1, step = LP_TABLE / LG_SLICE; f0 < s1 && !bad; f0 = f1) {
        f1 = min(s1, f0 + step);
        const int c0 = f0 * LG_SLICE, c1 = min(a.V, f1 * LG_SLICE);
        if constexpr (TOUCH) {
            if (f0 != s0 || step != LP_TABLE / LG_SLICE) {
                __syncthreads();   // the table before has been read
                clear_table(NT, t, c1 - c0);
                __syncthreads();
            }
            const TableState state = build_table(NT, a, r, z, c0, c1 - c0, t, [](int, float x, float) { return x; });
            bad = state == kBad;
            if (bad)
                break;
            if (state == kFull) {
                step = half(c1 - c0) / LG_SLICE;
                f1 = f0;
                continue;
            }
            if (threadIdx.x == NT - 1 && target >= c0 && target < c1 && is_touched(t, target - c0))
                target_x = __uint_as_float(t.value[rank_of(t, target - c0)]);
        }
        for (int s = f0 + warp; s < f1; s += WARPS) {
            Raw8<T> raw[4];
            load_chunks<T, 4>(raw, z, s * LG_SLICE, a.V, shift);
            int n0 = 0, n1 = 0;   // the slice's touched columns
            if constexpr (TOUCH) {
                const int group = (s - f0) * (LG_SLICE / 128);
                n0 = t.before[group];
                n1 = group + LG_SLICE / 128 < t.groups ? t.before[group + LG_SLICE / 128] : t.used;
            }
            if (mask || n1 > n0) {
#pragma unroll
                for (int u = 0; u < 4; ++u) {
                    const int col = s * LG_SLICE + u * 256 + lane * 8;
                    uint32_t drop = 0u;
                    if (col < a.V) {
                        if (mask)
                            drop = ~static_cast<uint32_t>(mask[col >> 3]) & 0xffu;
                        if (TOUCH)
                            drop |= reinterpret_cast<const uint8_t *>(t.bitmap)[(col - c0) >> 3];
                    }
                    if (drop)
                        drop8(raw[u], drop, masks);
                }
            }
            float m, sum;
            warp_sums<T, 4>(raw, k2, t.value + n0, n1 - n0, m, sum);
            if (lane == 0)
                part[s] = make_float2(m, sum);
        }
    }
    __syncthreads();
    if (a.segs > 1) {
        cluster_wait();
        if (rank != 0) {
            const uint32_t part0 = mapa_shared(smem_u32(part), 0);
            for (int s = s0 + static_cast<int>(threadIdx.x); s < s1; s += NT)
                st_cluster_f2(part0 + s * 8, part[s].x, part[s].y);
            if (threadIdx.x == NT - 1 && has_target)
                st_shared_cluster(mapa_shared(smem_u32(&target_x), 0), __float_as_int(target_x));
        }
        __syncwarp();
        cluster_arrive();
        cluster_wait();
    }
    if (rank == 0 && warp == 0) {
        float m = neg_inf(), sum = 0.f;
        if (!bad) {   // in slice order: lane l takes slices l, l + 32, ...
            for (int s = lane; s < slices; s += 32)
                join(m, sum, part[s].x, part[s].y, k2);
            warp_join(m, sum, k2);
        }
        if (lane == 0) {
            const bool in = target >= 0 && target < a.V;
            a.out_lse[row] = bad ? quiet_nan() : row_lse(m, sum, inv_tau);
            a.out_logp[row] = bad || !in ? quiet_nan() : row_logp(target_x, m, sum, inv_tau);
            if (bad)
                report_bad_input(a.status);
        }
    }
}

template <typename F> cudaError_t set_smem(F *kernel)
{
    const size_t logp = table_bytes<int32_t>(LP_TABLE, LP_LOGP_CAP) + LG_MAX_SLICES * 8;
    const size_t map = table_bytes<uint16_t>(LP_MAP_SLICES * LG_SLICE, LP_HEAVY_CAP);
    return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                static_cast<int>(std::max(logp, map)));
}

template <typename T, typename TO, int OP> cudaError_t launch_map(ProcArgs a, int num_sms, cudaStream_t s)
{
    const bool touch = a.spans || a.bias_offsets;
    const int slices = lg_slices(a.V);
    // segments of at most LP_MAP_SLICES, and of at least four; five CTAs for every SM if
    // the rows do not give them (of 3, 4, 5 and 6 the best for 64 rows of 128256 and 333
    // of 32003)
    const int want = static_cast<int>((int64_t(5) * num_sms + a.N - 1) / a.N);
    const int segs = std::max((slices + LP_MAP_SLICES - 1) / LP_MAP_SLICES, std::min((slices + 3) / 4, want));
    a.seg_slices = (slices + segs - 1) / segs;
    a.segs = (slices + a.seg_slices - 1) / a.seg_slices;
    a.table_columns = a.seg_slices * LG_SLICE;
    // Rows with long histories of their own (on average: rows that share theirs count
    // little) touch more columns than the usual table holds.  The host sees the length of
    // the array only: a padded token buffer counts whole.
    const bool heavy = a.history_len / LP_HEAVY >= a.N;
    a.table_cap = heavy ? LP_HEAVY_CAP : LP_MAP_CAP;
    const unsigned grid = static_cast<unsigned>(a.N) * static_cast<unsigned>(a.segs);
    if (touch)
        process_map_kernel<T, TO, OP, true>
            <<<grid, LP_MAP_THREADS, table_bytes<uint16_t>(a.table_columns, a.table_cap), s>>>(a);
    else
        process_map_kernel<T, TO, OP, false><<<grid, LP_MAP_THREADS, 0, s>>>(a);
    return cudaGetLastError();
}

template <typename T, bool TOUCH, int NT, int CTAS> cudaError_t launch_logp_kernel(const ProcArgs &a, cudaStream_t s)
{
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(static_cast<unsigned>(a.N) * static_cast<unsigned>(a.segs));
    cfg.blockDim = dim3(NT);
    cfg.dynamicSmemBytes = static_cast<size_t>(lg_slices(a.V)) * 8 +
                           (TOUCH ? table_bytes<int32_t>(a.table_columns, a.table_cap) : 0);
    cfg.stream = s;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = static_cast<unsigned>(a.segs);
    at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = a.segs > 1 ? 1 : 0;   // a plain launch where one CTA has the row
    return cudaLaunchKernelEx(&cfg, process_logp_kernel<T, TOUCH, NT, CTAS>, a);
}

template <typename T> cudaError_t launch_logp(ProcArgs a, int num_sms, cudaStream_t s)
{
    const bool touch = a.spans || a.bias_offsets;
    const int slices = lg_slices(a.V);
    int ranks = 1;   // CTAs of a row: more while the rows alone leave SMs idle
    while (ranks < LG_CLUSTER && ranks * 2 <= slices && static_cast<int64_t>(a.N) * ranks < 4 * num_sms)
        ranks *= 2;
    a.seg_slices = (slices + ranks - 1) / ranks;
    a.segs = (slices + a.seg_slices - 1) / a.seg_slices;
    a.table_columns = std::min(LP_TABLE, a.seg_slices * LG_SLICE);
    // The shorter a CTA's part of the row, the more of its time is the table's, and the
    // more CTAs an SM needs to fill it.  128 threads against 384: 55 us against 75 us for
    // 2916 rows of 20544 fp16; 192 against 384: 118 us against 138 us for 4096 of 50304
    // bf16; 256 against 384: 439 us against 460 us for 8192 of 151936 bf16.  The tables
    // are kept small because the loads in flight live in what shared memory leaves of
    // L1 (2048 entries for 1024: 128 us for 118 us at 50304 columns).  The limits on
    // registers were set for 16-bit logits; a warp's slice of fp32 ones is 32 registers by
    // itself, and those kernels spill: 44 to 52 bytes a thread, 204 at 192 threads.
    a.table_cap = a.seg_slices <= 110 ? 1024 : LP_LOGP_CAP;
    if (a.seg_slices <= 40)
        return touch ? launch_logp_kernel<T, true, 128, 10>(a, s) : launch_logp_kernel<T, false, 128, 10>(a, s);
    if (a.seg_slices <= 110)
        return touch ? launch_logp_kernel<T, true, 192, 7>(a, s) : launch_logp_kernel<T, false, 192, 7>(a, s);
    return touch ? launch_logp_kernel<T, true, 256, 5>(a, s) : launch_logp_kernel<T, false, 256, 5>(a, s);
}

template <typename T> cudaError_t launch_op(const ProcArgs &a, int op, int out_dtype, int num_sms, cudaStream_t s)
{
    if (op == LP_LOGP)
        return launch_logp<T>(a, num_sms, s);
    if (op == LP_GRAD)
        return launch_map<T, T, LP_GRAD>(a, num_sms, s);
    if (out_dtype == TIM_F32)
        return launch_map<T, float, LP_WRITE>(a, num_sms, s);
    return launch_map<T, T, LP_WRITE>(a, num_sms, s);
}

template <typename T> cudaError_t prepare()
{
    for (cudaError_t e : {set_smem(process_map_kernel<T, T, LP_WRITE, true>), set_smem(process_map_kernel<T, float, LP_WRITE, true>),
                          set_smem(process_map_kernel<T, T, LP_GRAD, true>),
                          set_smem(process_logp_kernel<T, true, 192, 7>), set_smem(process_logp_kernel<T, true, 256, 5>)})
        if (e != cudaSuccess)
            return e;
    return cudaSuccess;
}

} // namespace

cudaError_t logits_process_launch(ProcArgs a, int op, int dtype, int out_dtype, int num_sms, cudaStream_t s)
{
    if (dtype == TIM_F32)
        return launch_op<float>(a, op, out_dtype, num_sms, s);
    if (dtype == TIM_BF16)
        return launch_op<__nv_bfloat16>(a, op, out_dtype, num_sms, s);
    return launch_op<__half>(a, op, out_dtype, num_sms, s);
}

cudaError_t logits_process_prepare_device()
{
    cudaError_t e = prepare<float>();
    if (e == cudaSuccess)
        e = prepare<__nv_bfloat16>();
    if (e == cudaSuccess)
        e = prepare<__half>();
    return e;
}

} // namespace tim
