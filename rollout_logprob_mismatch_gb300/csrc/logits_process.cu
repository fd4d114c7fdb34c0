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
// columns are treated as untouched, with one multiplication each, and the
// touched ones are replaced from a table in shared memory: a CTA owns a segment
// of at most 16384 columns with one 4-byte slot each (64 KB, so that two CTAs fit an
// SM and one's table phase runs under the other's loads).  It scans the row's
// history three times: the slots of its ids are set to zero, then counted with
// shared-memory atomics (integers: no order), then one thread per distinct id
// (the one that sets its bit in a bitmap) turns the count into the column's
// final value.  Nothing has to be cleared between segments, no sort, no hash, any
// history length.  The first slice of each warp is loaded before the scans.
#include <algorithm>

#include "logits_rows.cuh"

namespace tim {
namespace {

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
    if (r.b0 < 0 || r.b1 < r.b0 || r.b1 > a.num_bias) {
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

// A touched column: processed value y (mask apart) and its slope dy/dz.
__device__ __forceinline__ float touched_value(const RowRules &r, float z, float bias, uint32_t word, float &slope)
{
    float x = z + bias;
    slope = 1.f;
    if (word != 0) {
        slope = x > 0.f ? 1.f / r.rho : r.rho;
        x = x > 0.f ? x / r.rho : x * r.rho;
    }
    const uint32_t c = word & 0x7fffffffu;
    if (c != 0)
        x = x - r.freq * static_cast<float>(c) - r.pres;
    slope /= r.tau;
    return x / r.tau;
}

__device__ __forceinline__ float bias_of(const ProcArgs &a, const RowRules &r, int id)
{
    int lo = r.b0, hi = r.b1;
    while (lo < hi) {
        const int mid = (lo + hi) >> 1;
        if (a.bias_ids[mid] < id)
            lo = mid + 1;
        else
            hi = mid;
    }
    return lo < r.b1 && a.bias_ids[lo] == id ? a.bias_values[lo] : 0.f;
}

// Fills the table of columns c0 .. c0 + width - 1: bit set and slot = the
// replacement, as op needs it.  All threads of the CTA.
template <typename T, int OP>
__device__ void fill_table(const ProcArgs &a, const RowRules &r, const T *z, int c0, int width, uint32_t *slot,
                           uint32_t *bitmap, int target, float g, float lse)
{
    const unsigned w = static_cast<unsigned>(width);
    for (int j = threadIdx.x; j < (width + 31) / 32; j += LP_THREADS)
        bitmap[j] = 0;
    for (int j = r.h0 + static_cast<int>(threadIdx.x); j < r.h1; j += LP_THREADS) {
        const unsigned k = static_cast<unsigned>(a.history[j]) - static_cast<unsigned>(c0);
        if (k < w)
            slot[k] = 0;
    }
    for (int j = r.b0 + static_cast<int>(threadIdx.x); j < r.b1; j += LP_THREADS) {
        const unsigned k = static_cast<unsigned>(a.bias_ids[j]) - static_cast<unsigned>(c0);
        if (k < w)
            slot[k] = 0;
    }
    __syncthreads();
    for (int j = r.h0 + static_cast<int>(threadIdx.x); j < r.h1; j += LP_THREADS) {
        const unsigned k = static_cast<unsigned>(a.history[j]) - static_cast<unsigned>(c0);
        if (k < w) {
            if (j >= r.hg)
                atomicAdd(slot + k, 1u);
            else
                atomicOr(slot + k, 0x80000000u);
        }
    }
    __syncthreads();
    auto claim = [&](unsigned k, int id, float bias) {
        float slope;
        float y = touched_value(r, Elem<T>::load(z + id), bias, slot[k], slope);
        if constexpr (OP == LP_LOGP)
            y *= LG_LOG2E;
        if constexpr (OP == LP_GRAD) {
            const float p = exp2_approx((y - lse) * LG_LOG2E);
            y = y == neg_inf() ? 0.f : ((id == target ? 1.f : 0.f) - p) * (g * slope);
        }
        slot[k] = __float_as_uint(y);
    };
    for (int j = r.h0 + static_cast<int>(threadIdx.x); j < r.h1; j += LP_THREADS) {
        const int id = a.history[j];
        const unsigned k = static_cast<unsigned>(id) - static_cast<unsigned>(c0);
        if (k < w) {
            const uint32_t bit = 1u << (k & 31);
            if (!(atomicOr(bitmap + (k >> 5), bit) & bit))
                claim(k, id, r.b1 > r.b0 ? bias_of(a, r, id) : 0.f);
        }
    }
    for (int j = r.b0 + static_cast<int>(threadIdx.x); j < r.b1; j += LP_THREADS) {
        const int id = a.bias_ids[j];
        const unsigned k = static_cast<unsigned>(id) - static_cast<unsigned>(c0);
        if (k < w) {
            const uint32_t bit = 1u << (k & 31);
            if (!(atomicOr(bitmap + (k >> 5), bit) & bit))
                claim(k, id, a.bias_values[j]);
        }
    }
    __syncthreads();
}

// Whether any of the row's bias ids is out of range or out of order (all
// threads; a barrier).
__device__ __forceinline__ bool bias_bad(const ProcArgs &a, const RowRules &r)
{
    bool bad = false;
    for (int j = r.b0 + static_cast<int>(threadIdx.x); j < r.b1; j += LP_THREADS) {
        const int id = a.bias_ids[j];
        bad |= id < 0 || id >= a.V || (j > r.b0 && a.bias_ids[j - 1] >= id);
    }
    return __syncthreads_or(bad) != 0;
}

// WRITE and GRAD: one CTA per (row, segment); no column depends on another.
template <typename T, typename TO, int OP, bool TOUCH>
__global__ void __launch_bounds__(LP_THREADS) process_map_kernel(const ProcArgs a)
{
    extern __shared__ uint32_t smem[];
    uint32_t *slot = smem, *bitmap = smem + LP_SEG;
    const int row = static_cast<int>(blockIdx.x / static_cast<unsigned>(a.segs));
    const int seg = static_cast<int>(blockIdx.x % static_cast<unsigned>(a.segs));
    const int c0 = seg * a.seg_slices * LG_SLICE;
    const int c1 = min(a.V, c0 + a.seg_slices * LG_SLICE);
    const T *z = static_cast<const T *>(a.z) + row * a.ld;
    TO *out = static_cast<TO *>(a.out) + row * a.ldo;
    const bool vec = row_vec(z), vec_out = row_vec(out);

    RowRules r = row_rules(a, row);
    float g = 1.f, lse = 0.f;
    int target = -1;
    if constexpr (OP == LP_GRAD) {
        g = a.grad[row];
        lse = a.lse[row];
        if (lse == neg_inf())
            lse = -neg_inf();   // nothing is left of the row: every probability is 0
        target = a.targets[row];
    }
    if constexpr (TOUCH)
        r.bad |= bias_bad(a, r);
    if (r.bad || (OP == LP_GRAD && g == 0.f)) {
        float v[8];
        const float fill = r.bad ? quiet_nan() : 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i)
            v[i] = fill;
        for (int col = c0 + static_cast<int>(threadIdx.x) * 8; col < c1; col += LP_THREADS * 8)
            store8<TO>(out, col, c1, vec_out, v);
        if (r.bad && threadIdx.x == 0)
            report_bad_input(a.status);
        return;
    }
    if constexpr (TOUCH)
        fill_table<T, OP>(a, r, z, c0, c1 - c0, slot, bitmap, target, g, lse);

    const float gi = g * r.inv_tau;
    for (int col = c0 + static_cast<int>(threadIdx.x) * 8; col < c1; col += LP_THREADS * 8) {
        Raw8<T> raw;
        load8<T>(raw, z, col, c1, vec);
        float v[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float x = Elem<T>::get(raw.w, i);
            if constexpr (OP == LP_WRITE) {
                v[i] = x * r.inv_tau;
            } else {
                const float p = exp2_approx(fmaf(x, r.inv_tau, -lse) * LG_LOG2E);
                v[i] = -p * gi;
                if (col + i == target)
                    v[i] = x == neg_inf() ? 0.f : (1.f - p) * gi;
            }
        }
        if constexpr (TOUCH) {
            const int k = col - c0;
            const uint32_t bits = reinterpret_cast<const uint8_t *>(bitmap)[k >> 3];
            if (bits) {
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    if (bits >> i & 1)
                        v[i] = __uint_as_float(slot[k + i]);
            }
        }
        if (r.mask) {
            const uint32_t bits = r.mask[col >> 3];
#pragma unroll
            for (int i = 0; i < 8; ++i)
                if (!(bits >> i & 1))
                    v[i] = OP == LP_WRITE ? neg_inf() : 0.f;
        }
        store8<TO>(out, col, c1, vec_out, v);
    }
}

// LOGP: a cluster per row; each rank reduces seg_slices slices, one warp per
// slice, in segments of at most LP_SEG_SLICES where there is a table.  The
// slices' partials go to rank 0's shared memory, which folds them.
template <typename T, bool TOUCH>
__global__ void __launch_bounds__(LP_THREADS) process_logp_kernel(const ProcArgs a)
{
    extern __shared__ uint32_t smem[];
    uint32_t *slot = smem, *bitmap = smem + LP_SEG;
    __shared__ float2 part[LG_MAX_SLICES];
    __shared__ float target_t;
    const int rank = static_cast<int>(cluster_ctarank());
    const int row = static_cast<int>(blockIdx.x / static_cast<unsigned>(a.segs));
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int slices = (a.V + LG_SLICE - 1) / LG_SLICE;
    const int s0 = min(slices, rank * a.seg_slices), s1 = min(slices, s0 + a.seg_slices);
    const T *z = static_cast<const T *>(a.z) + row * a.ld;
    const bool vec = row_vec(z);
    cluster_arrive();   // waited for before the first store into rank 0's shared memory

    RowRules r = row_rules(a, row);
    const int target = a.targets[row];
    if constexpr (TOUCH)
        r.bad |= bias_bad(a, r);
    const float k2 = LG_LOG2E / r.tau;
    const int step = TOUCH ? LP_SEG_SLICES : LG_MAX_SLICES;
    for (int f0 = s0; f0 < s1 && !r.bad; f0 += step) {
        const int f1 = min(s1, f0 + step);
        const int c0 = f0 * LG_SLICE;
        if constexpr (TOUCH) {
            if (f0 != s0)
                __syncthreads();   // the segment before has been read
            fill_table<T, LP_LOGP>(a, r, z, c0, min(a.V, f1 * LG_SLICE) - c0, slot, bitmap, target, 0.f, 0.f);
        }
        for (int s = f0 + warp; s < f1; s += LP_WARPS) {
            Raw8<T> raw[4];
#pragma unroll
            for (int u = 0; u < 4; ++u)
                load8<T>(raw[u], z, s * LG_SLICE + u * 256 + lane * 8, a.V, vec);
            float m = neg_inf(), sum = 0.f;
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                const int col = s * LG_SLICE + u * 256 + lane * 8;
                float t[8];
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    t[i] = Elem<T>::get(raw[u].w, i) * k2;
                if (TOUCH && col < a.V) {
                    const int k = col - c0;
                    const uint32_t bits = reinterpret_cast<const uint8_t *>(bitmap)[k >> 3];
                    if (bits) {
#pragma unroll
                        for (int i = 0; i < 8; ++i)
                            if (bits >> i & 1)
                                t[i] = __uint_as_float(slot[k + i]);
                    }
                }
                if (r.mask && col < a.V) {
                    const uint32_t bits = r.mask[col >> 3];
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        if (!(bits >> i & 1))
                            t[i] = neg_inf();
                }
                if (static_cast<unsigned>(target) - static_cast<unsigned>(col) < 8u) {
                    float v = t[0];
#pragma unroll
                    for (int i = 1; i < 8; ++i)
                        v = target - col == i ? t[i] : v;
                    target_t = v;
                }
                lane_add8(m, sum, t);
            }
            warp_join(m, sum);
            if (lane == 0)
                part[s] = make_float2(m, sum);
        }
    }
    __syncthreads();
    cluster_wait();
    if (rank != 0) {
        const uint32_t part0 = mapa_shared(smem_u32(part), 0);
        for (int s = s0 + static_cast<int>(threadIdx.x); s < s1; s += LP_THREADS)
            st_cluster_f2(part0 + s * 8, part[s].x, part[s].y);
        if (threadIdx.x == 0 && target >= s0 * LG_SLICE && target < s1 * LG_SLICE)
            st_shared_cluster(mapa_shared(smem_u32(&target_t), 0), __float_as_int(target_t));
    }
    __syncwarp();
    cluster_arrive();
    cluster_wait();
    if (rank == 0 && warp == 0) {
        float m = neg_inf(), sum = 0.f;
        if (!r.bad)
            fold_slices(part, slices, lane, m, sum);
        if (lane == 0) {
            const bool in = target >= 0 && target < a.V;
            a.out_lse[row] = r.bad ? quiet_nan() : row_lse(m, sum);
            a.out_logp[row] = r.bad || !in ? quiet_nan() : row_logp(target_t, m, sum);
            if (r.bad)
                report_bad_input(a.status);
        }
    }
}

constexpr int kTableBytes = (LP_SEG + LP_SEG / 32) * 4;

template <typename F> cudaError_t set_smem(F *kernel)
{
    return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kTableBytes);
}

template <typename T, typename TO, int OP> cudaError_t launch_map(ProcArgs a, int num_sms, cudaStream_t s)
{
    const bool touch = a.spans || a.bias_offsets;
    const int slices = lg_slices(a.V);
    // segments of 16 slices; fewer while the rows alone do not give the GPU two CTAs per SM
    int per = std::min(LP_SEG_SLICES, slices);
    while (per > 4 && static_cast<int64_t>(a.N) * ((slices + per - 1) / per) < 2 * num_sms)
        per = (per + 1) / 2;
    a.seg_slices = per;
    a.segs = (slices + per - 1) / per;
    const unsigned grid = static_cast<unsigned>(a.N) * static_cast<unsigned>(a.segs);
    if (touch)
        process_map_kernel<T, TO, OP, true><<<grid, LP_THREADS, kTableBytes, s>>>(a);
    else
        process_map_kernel<T, TO, OP, false><<<grid, LP_THREADS, 0, s>>>(a);
    return cudaGetLastError();
}

template <typename T> cudaError_t launch_logp(ProcArgs a, int num_sms, cudaStream_t s)
{
    const bool touch = a.spans || a.bias_offsets;
    const int slices = lg_slices(a.V);
    int ranks = 1;   // CTAs of a row: more while the rows alone leave SMs idle
    while (ranks < LG_CLUSTER && ranks * 2 <= slices && static_cast<int64_t>(a.N) * ranks < 2 * num_sms)
        ranks *= 2;
    a.segs = ranks;
    a.seg_slices = (slices + ranks - 1) / ranks;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(static_cast<unsigned>(a.N) * static_cast<unsigned>(ranks));
    cfg.blockDim = dim3(LP_THREADS);
    cfg.dynamicSmemBytes = touch ? kTableBytes : 0;
    cfg.stream = s;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = static_cast<unsigned>(ranks);
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
