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
// before each of its words, and one 4-byte entry per touched column, in column
// order.  Building it takes two scans of the row's history (set the bits; count
// with shared-memory integer atomics, which have no order) and one gather per
// distinct id; no sort, no hash, any history length (a history that could fill
// more than LP_CAP entries is handled LP_CAP columns at a time).  The log-probability
// takes the touched columns out of the stream and adds the table's entries of the
// same slice; the others write their columns first and the touched ones over them.
#include <algorithm>

#include "logits_rows.cuh"

namespace tim {
namespace {

// A table entry while it is counted: seen in the prompt, listed with a bias, and
// the number of times among the generated tokens (the host keeps it below 2^30).
constexpr uint32_t kPrompt = 0x80000000u, kBiased = 0x40000000u, kCount = 0x3fffffffu;

struct RowRules {
    float tau, inv_tau, rho, pres, freq;
    int h0, hg, h1;            // history span
    int b0, b1;                // bias entries
    const uint8_t *mask;       // the row's bits, or null
    bool bad;
};

__device__ __forceinline__ RowRules row_rules(const ProcArgs &a, int row)
{
    RowRules r;
    r.tau = a.temperature ? a.temperature[row] : 1.f;
    r.rho = a.repetition ? a.repetition[row] : 1.f;
    r.pres = a.presence ? a.presence[row] : 0.f;
    r.freq = a.frequency ? a.frequency[row] : 0.f;
    r.h0 = r.hg = r.h1 = r.b0 = r.b1 = 0;
    if (a.spans) {
        const int32_t *s = a.spans + static_cast<int64_t>(row) * 3;
        r.h0 = s[0];
        r.hg = s[1];
        r.h1 = s[2];
    }
    if (a.bias_offsets) {
        r.b0 = a.bias_offsets[row];
        r.b1 = a.bias_offsets[row + 1];
    }
    int m = -1;
    if (a.allowed)
        m = a.allowed_rows ? a.allowed_rows[row] : row;
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
    if (m >= a.num_allowed && a.allowed) {
        r.bad = true;
        m = -1;
    }
    r.mask = m >= 0 ? reinterpret_cast<const uint8_t *>(a.allowed + m * a.allowed_ld) : nullptr;
    return r;
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
struct Table {
    uint32_t *value;     // [LP_CAP]: counts, then the column's replacement (fp32 bits)
    uint32_t *bitmap;    // [LP_TABLE / 32]
    uint16_t *before;    // [LP_TABLE / 32]: bits set in the words before
    int words, used;     // of the columns in hand
};

__device__ __forceinline__ int rank_of(const Table &t, unsigned k)
{
    const uint32_t w = t.bitmap[k >> 5];
    return t.before[k >> 5] + __popc(w & ((1u << (k & 31)) - 1));
}

// Column (relative to the table's first) of entry n.
__device__ __forceinline__ int column_of(const Table &t, int n)
{
    int lo = 0, hi = t.words - 1;   // the last word with before <= n
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (t.before[mid] <= n)
            lo = mid;
        else
            hi = mid - 1;
    }
    uint32_t w = t.bitmap[lo];
    for (int skip = n - t.before[lo]; skip > 0; --skip)
        w &= w - 1;
    return lo * 32 + __ffs(static_cast<int>(w)) - 1;
}

// f(position, id relative to c0) for the entries ids[j0 .. j1) within [c0, c0 + width).
template <typename F>
__device__ __forceinline__ void scan_ids(const int32_t *ids, int j0, int j1, int c0, int width, F f)
{
    for (int j = j0 + static_cast<int>(threadIdx.x); j < j1; j += LP_THREADS) {
        const unsigned k = static_cast<unsigned>(ids[j]) - static_cast<unsigned>(c0);
        if (k < static_cast<unsigned>(width))
            f(j, k);
    }
}

// Builds the table of columns c0 .. c0 + width - 1 with replacement(id, x, slope)
// for each.  All threads of the CTA; false (in all) where the row's bias ids are
// out of range or order.  Ends with a barrier.
template <typename T, typename F>
__device__ bool build_table(const ProcArgs &a, const RowRules &r, const T *z, int c0, int width, Table &t, F replacement)
{
    __shared__ int warp_bits[LP_WARPS];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    t.words = (width + 31) / 32;
    for (int j = threadIdx.x; j < t.words; j += LP_THREADS)
        t.bitmap[j] = 0;
    for (int j = threadIdx.x; j < min(LP_CAP, r.h1 - r.h0 + r.b1 - r.b0); j += LP_THREADS)
        t.value[j] = 0;
    bool bad = false;
    for (int j = r.b0 + static_cast<int>(threadIdx.x); j < r.b1; j += LP_THREADS) {
        const int id = a.bias_ids[j];
        bad |= id < 0 || id >= a.V || (j > r.b0 && a.bias_ids[j - 1] >= id);
    }
    if (__syncthreads_or(bad))
        return false;
    auto mark = [&](int, unsigned k) { atomicOr(t.bitmap + (k >> 5), 1u << (k & 31)); };
    scan_ids(a.history, r.h0, r.h1, c0, width, mark);
    scan_ids(a.bias_ids, r.b0, r.b1, c0, width, mark);
    __syncthreads();
    // bits before each word: a run of words per thread
    const int run = (t.words + LP_THREADS - 1) / LP_THREADS;
    const int w0 = min(t.words, static_cast<int>(threadIdx.x) * run), w1 = min(t.words, w0 + run);
    int bits = 0;
    for (int w = w0; w < w1; ++w)
        bits += __popc(t.bitmap[w]);
    int upto = bits;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const int v = __shfl_up_sync(0xffffffffu, upto, d);
        upto += lane >= d ? v : 0;
    }
    if (lane == 31)
        warp_bits[warp] = upto;
    __syncthreads();
    int base = upto - bits;
    t.used = 0;
#pragma unroll
    for (int w = 0; w < LP_WARPS; ++w) {
        base += w < warp ? warp_bits[w] : 0;
        t.used += warp_bits[w];
    }
    for (int w = w0; w < w1; ++w) {
        t.before[w] = static_cast<uint16_t>(base);
        base += __popc(t.bitmap[w]);
    }
    __syncthreads();
    scan_ids(a.history, r.h0, r.h1, c0, width, [&](int j, unsigned k) {
        uint32_t *v = t.value + rank_of(t, k);
        if (j >= r.hg)
            atomicAdd(v, 1u);
        else
            atomicOr(v, kPrompt);
    });
    scan_ids(a.bias_ids, r.b0, r.b1, c0, width, [&](int, unsigned k) { atomicOr(t.value + rank_of(t, k), kBiased); });
    __syncthreads();
    auto finish = [&](int n, int id, float bias) {
        float slope;
        float x = touched_value(r, Elem<T>::load(z + id), bias, t.value[n] & ~kBiased, slope);
        if (r.mask && !(r.mask[id >> 3] >> (id & 7) & 1))
            x = neg_inf();
        t.value[n] = __float_as_uint(replacement(id, x, slope));
    };
    for (int n = threadIdx.x; n < t.used; n += LP_THREADS)
        if (!(t.value[n] & kBiased))
            finish(n, c0 + column_of(t, n), 0.f);
    __syncthreads();
    if (r.b1 > r.b0) {   // the biased ones, by their bias entry
        scan_ids(a.bias_ids, r.b0, r.b1, c0, width,
                 [&](int j, unsigned k) { finish(rank_of(t, k), c0 + static_cast<int>(k), a.bias_values[j]); });
        __syncthreads();
    }
    return true;
}

// Columns a table covers at a time.
__device__ __forceinline__ int table_step(const RowRules &r)
{
    return r.h1 - r.h0 + r.b1 - r.b0 <= LP_CAP ? LP_TABLE : LP_CAP;
}

__device__ __forceinline__ Table carve(uint32_t *smem, int table_columns)
{
    Table t;
    t.value = smem;
    t.bitmap = smem + LP_CAP;
    t.before = reinterpret_cast<uint16_t *>(t.bitmap + table_columns / 32);
    t.words = t.used = 0;
    return t;
}

// ---------------------------------------------------------------- kernels
// WRITE and GRAD: one CTA per (row, segment); no column depends on another.
template <typename T, typename TO, int OP, bool TOUCH>
__global__ void __launch_bounds__(LP_THREADS) process_map_kernel(const ProcArgs a)
{
    extern __shared__ uint32_t smem[];
    const int row = static_cast<int>(blockIdx.x / static_cast<unsigned>(a.segs));
    const int seg = static_cast<int>(blockIdx.x % static_cast<unsigned>(a.segs));
    const int seg0 = seg * a.seg_slices * LG_SLICE, seg1 = min(a.V, seg0 + a.seg_slices * LG_SLICE);
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const T *z = static_cast<const T *>(a.z) + row * a.ld;
    TO *out = static_cast<TO *>(a.out) + row * a.ldo;
    const uint32_t shift = row_shift(z), shift_out = row_shift(out);

    const RowRules r = row_rules(a, row);
    bool bad = r.bad;
    float g = 1.f, lse = 0.f, target_v = 0.f;
    int target = -1;
    if constexpr (OP == LP_GRAD) {
        g = a.grad[row];
        lse = a.lse[row];
        if (lse == neg_inf())
            lse = -neg_inf();   // nothing is left of the row: every probability is 0
        target = a.targets[row];
    }
    auto probability = [&](float y) { return exp2_approx((y - lse) * LG_LOG2E); };
    const float gi = g * r.inv_tau;
    const int step = TOUCH ? table_step(r) : LP_TABLE;
    Table t = carve(smem, a.table_columns);
    for (int c0 = seg0; c0 < seg1; c0 += step) {
        const int c1 = min(seg1, c0 + step);
        const bool zero = OP == LP_GRAD && g == 0.f;
        const bool has_target = OP == LP_GRAD && target >= c0 && target < c1;
        if constexpr (OP == LP_GRAD) {
            if (has_target && threadIdx.x == 0) {   // an untouched target's one-hot term
                const float x = Elem<T>::load(z + target);
                const bool in = !r.mask || (r.mask[target >> 3] >> (target & 7) & 1);
                target_v = in && x != neg_inf() ? (1.f - exp2_approx(fmaf(x, r.inv_tau, -lse) * LG_LOG2E)) * gi : 0.f;
            }
            if constexpr (!TOUCH)
                __syncthreads();   // read before it is written over in place
        }
        if constexpr (TOUCH) {
            if (!bad && !zero) {
                if (c0 != seg0)
                    __syncthreads();   // the table before has been written out
                bad = !build_table(a, r, z, c0, c1 - c0, t, [&](int id, float x, float slope) {
                    const float y = x / r.tau;
                    if constexpr (OP == LP_GRAD)
                        return y == neg_inf() ? 0.f : ((id == target ? 1.f : 0.f) - probability(y)) * (g * (slope / r.tau));
                    else
                        return y;
                });
            }
        }
        if (bad || zero) {
            float v[8];
            const float fill = bad ? quiet_nan() : 0.f;
#pragma unroll
            for (int i = 0; i < 8; ++i)
                v[i] = fill;
            for (int b = c0 + warp * 256; b < c1; b += LP_WARPS * 256)
                store8<TO>(out, b + lane * 8, c1, shift_out, v);
            continue;
        }
        const Pair inv2 = pair(r.inv_tau, r.inv_tau), lse2 = pair(-lse, -lse), e2 = pair(LG_LOG2E, LG_LOG2E),
                   g2 = pair(-gi, -gi);
        for (int b = c0 + warp * 512; b < c1; b += LP_WARPS * 512) {
            Raw8<T> raw[2];
            uint32_t ok[2] = {0xffu, 0xffu};
            load_chunks<T, 2>(raw, z, b, c1, shift);
            if (r.mask) {
#pragma unroll
                for (int u = 0; u < 2; ++u)
                    if (b + u * 256 + lane * 8 < c1)
                        ok[u] = r.mask[(b + u * 256 + lane * 8) >> 3];
            }
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                float v[8];
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const Pair x = get2<T>(raw[u], k);
                    if constexpr (OP == LP_WRITE) {
                        unpair(mul2(x, inv2), v[2 * k], v[2 * k + 1]);
                    } else {
                        float lo, hi;
                        unpair(mul2(fma2(x, inv2, lse2), e2), lo, hi);
                        unpair(mul2(pair(exp2_approx(lo), exp2_approx(hi)), g2), v[2 * k], v[2 * k + 1]);
                    }
                }
                if (ok[u] != 0xffu) {
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        if (!(ok[u] >> i & 1))
                            v[i] = OP == LP_WRITE ? neg_inf() : 0.f;
                }
                store8<TO>(out, b + u * 256 + lane * 8, c1, shift_out, v);
            }
        }
        if (TOUCH || OP == LP_GRAD) {
            __syncthreads();   // the touched columns go over what has just been written
            if (OP == LP_GRAD && has_target && threadIdx.x == 0 &&
                !(TOUCH && (t.bitmap[(target - c0) >> 5] >> ((target - c0) & 31) & 1)))
                out[target] = Elem<TO>::from(target_v);
        }
        if constexpr (TOUCH) {
            for (int n = threadIdx.x; n < t.used; n += LP_THREADS)
                out[c0 + column_of(t, n)] = Elem<TO>::from(__uint_as_float(t.value[n]));
        }
    }
    if (bad && threadIdx.x == 0)
        report_bad_input(a.status);
}

// LOGP: a cluster per row; each rank reduces seg_slices slices, one warp per
// slice.  The slices' partials go to rank 0's shared memory, which folds them.
template <typename T, bool TOUCH>
__global__ void __launch_bounds__(LP_THREADS) process_logp_kernel(const ProcArgs a)
{
    extern __shared__ uint32_t smem[];
    __shared__ float2 part[LG_MAX_SLICES];
    __shared__ float target_x;
    const int rank = static_cast<int>(cluster_ctarank());
    const int row = static_cast<int>(blockIdx.x / static_cast<unsigned>(a.segs));
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int slices = (a.V + LG_SLICE - 1) / LG_SLICE;
    const int s0 = min(slices, rank * a.seg_slices), s1 = min(slices, s0 + a.seg_slices);
    const T *z = static_cast<const T *>(a.z) + row * a.ld;
    const uint32_t shift = row_shift(z);
    if (a.segs > 1)
        cluster_arrive();   // waited for before the first store into rank 0's shared memory

    const RowRules r = row_rules(a, row);
    bool bad = r.bad;
    const int target = a.targets[row];
    const bool has_target = target >= s0 * LG_SLICE && target < min(a.V, s1 * LG_SLICE);
    const float k2 = LG_LOG2E * r.inv_tau;
    const int step = (TOUCH ? table_step(r) : LP_TABLE) / LG_SLICE;
    Table t = carve(smem, a.table_columns);
    for (int f0 = s0; f0 < s1 && !bad; f0 += step) {
        const int f1 = min(s1, f0 + step);
        const int c0 = f0 * LG_SLICE;
        if constexpr (TOUCH) {
            if (f0 != s0)
                __syncthreads();   // the table before has been read
            bad = !build_table(a, r, z, c0, min(a.V, f1 * LG_SLICE) - c0, t, [](int, float x, float) { return x; });
            if (bad)
                break;
        }
        if (threadIdx.x == 0 && target >= c0 && target < min(a.V, f1 * LG_SLICE)) {
            const bool in = !r.mask || (r.mask[target >> 3] >> (target & 7) & 1);
            if (!in)
                target_x = neg_inf();
            else if (TOUCH && (t.bitmap[(target - c0) >> 5] >> ((target - c0) & 31) & 1))
                target_x = __uint_as_float(t.value[rank_of(t, target - c0)]);
            else
                target_x = Elem<T>::load(z + target);
        }
        for (int s = f0 + warp; s < f1; s += LP_WARPS) {
            Raw8<T> raw[4];
            load_chunks<T, 4>(raw, z, s * LG_SLICE, a.V, shift);
            int n0 = 0, n1 = 0;   // the slice's touched columns
            if constexpr (TOUCH) {
                const int word = (s - f0) * (LG_SLICE / 32);
                n0 = t.before[word];
                n1 = word + LG_SLICE / 32 < t.words ? t.before[word + LG_SLICE / 32] : t.used;
            }
            if (r.mask || n1 > n0) {
#pragma unroll
                for (int u = 0; u < 4; ++u) {
                    const int col = s * LG_SLICE + u * 256 + lane * 8;
                    uint32_t drop = 0u;
                    if (col < a.V) {
                        if (r.mask)
                            drop = ~static_cast<uint32_t>(r.mask[col >> 3]) & 0xffu;
                        if (TOUCH)
                            drop |= reinterpret_cast<const uint8_t *>(t.bitmap)[(col - c0) >> 3];
                    }
                    if (drop)
                        drop8(raw[u], drop);
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
            for (int s = s0 + static_cast<int>(threadIdx.x); s < s1; s += LP_THREADS)
                st_cluster_f2(part0 + s * 8, part[s].x, part[s].y);
            if (threadIdx.x == 0 && has_target)
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
            a.out_lse[row] = bad ? quiet_nan() : row_lse(m, sum, r.inv_tau);
            a.out_logp[row] = bad || !in ? quiet_nan() : row_logp(target_x, m, sum, r.inv_tau);
            if (bad)
                report_bad_input(a.status);
        }
    }
}

// Dynamic shared memory of a table over `columns` columns (a multiple of 1024).
size_t table_bytes(int columns) { return LP_CAP * 4 + columns / 32 * 6; }

template <typename F> cudaError_t set_smem(F *kernel)
{
    return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                static_cast<int>(table_bytes(LP_TABLE)));
}

template <typename T, typename TO, int OP> cudaError_t launch_map(ProcArgs a, int num_sms, cudaStream_t s)
{
    const bool touch = a.spans || a.bias_offsets;
    const int slices = lg_slices(a.V);
    // segments of at most 64 slices, fewer while there are not four CTAs for every SM
    int per = std::min(64, slices);
    while (per > 4 && static_cast<int64_t>(a.N) * ((slices + per - 1) / per) < 4 * num_sms)
        per = (per + 1) / 2;
    a.seg_slices = per;
    a.segs = (slices + per - 1) / per;
    a.table_columns = std::min(LP_TABLE, per * LG_SLICE);
    const unsigned grid = static_cast<unsigned>(a.N) * static_cast<unsigned>(a.segs);
    if (touch)
        process_map_kernel<T, TO, OP, true><<<grid, LP_THREADS, table_bytes(a.table_columns), s>>>(a);
    else
        process_map_kernel<T, TO, OP, false><<<grid, LP_THREADS, 0, s>>>(a);
    return cudaGetLastError();
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
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(static_cast<unsigned>(a.N) * static_cast<unsigned>(a.segs));
    cfg.blockDim = dim3(LP_THREADS);
    cfg.dynamicSmemBytes = touch ? table_bytes(a.table_columns) : 0;
    cfg.stream = s;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = static_cast<unsigned>(a.segs);
    at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    return touch ? cudaLaunchKernelEx(&cfg, process_logp_kernel<T, true>, a)
                 : cudaLaunchKernelEx(&cfg, process_logp_kernel<T, false>, a);
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
    cudaError_t e = set_smem(process_map_kernel<T, T, LP_WRITE, true>);
    if (e == cudaSuccess)
        e = set_smem(process_map_kernel<T, float, LP_WRITE, true>);
    if (e == cudaSuccess)
        e = set_smem(process_map_kernel<T, T, LP_GRAD, true>);
    if (e == cudaSuccess)
        e = set_smem(process_logp_kernel<T, true>);
    return e;
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
