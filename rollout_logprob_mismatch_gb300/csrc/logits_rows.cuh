// logits_rows.cuh -- device code shared by the operators on a head's logits:
// eight columns of a row at a time (any element type, any alignment), and the
// reduction of a slice of a row to (maximum, sum of exponentials).
//
// Log-sum-exp of a row, in base 2: with t_v = x_v log2(e), a set of columns is
// the pair (M, S), M = max t, S = sum 2^(t - M); two sets join as
// M = max(M1, M2), S = S1 2^(M1 - M) + S2 2^(M2 - M); lse = (M + log2 S) ln 2.
// A set of -inf columns only is (-inf, 0).  NaN and +inf make S NaN.
#pragma once

#include <cstdint>

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "../../include/tim.h"
#include "logits_internal.h"
#include "tim_internal.h"
#include "tim_ptx.cuh"

namespace tim {

constexpr float LG_LOG2E = 1.4426950408889634f;
constexpr float LG_LN2 = 0.6931471805599453f;

__device__ __forceinline__ float neg_inf() { return __int_as_float(static_cast<int>(0xff800000u)); }
__device__ __forceinline__ float quiet_nan() { return __int_as_float(0x7fc00000); }

__device__ __forceinline__ float exp2_approx(float x)   // 2 ulp; 2^-inf = 0, 2^nan = nan
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// ---------------------------------------------------------------- element types
template <typename T> struct Elem;

template <> struct Elem<float> {
    static constexpr int WORDS = 8;   // 32-bit words of 8 elements
    static constexpr uint32_t NEG_INF = 0xff800000u;
    static __device__ __forceinline__ float get(const uint32_t *w, int i) { return __uint_as_float(w[i]); }
    static __device__ __forceinline__ float load(const float *p) { return *p; }
    static __device__ __forceinline__ float from(float x) { return x; }
    static __device__ __forceinline__ uint32_t bits(const float *p) { return __float_as_uint(*p); }
    static __device__ __forceinline__ void put(uint32_t *w, int i, uint32_t b) { w[i] = b; }
};

template <> struct Elem<__nv_bfloat16> {
    static constexpr int WORDS = 4;
    static constexpr uint32_t NEG_INF = 0xff80u;
    static __device__ __forceinline__ float get(const uint32_t *w, int i)
    {
        return __uint_as_float((i & 1) ? (w[i >> 1] & 0xffff0000u) : (w[i >> 1] << 16));
    }
    static __device__ __forceinline__ float load(const __nv_bfloat16 *p) { return __bfloat162float(*p); }
    static __device__ __forceinline__ __nv_bfloat16 from(float x) { return __float2bfloat16_rn(x); }
    static __device__ __forceinline__ uint32_t bits(const __nv_bfloat16 *p) { return __bfloat16_as_ushort(*p); }
    static __device__ __forceinline__ void put(uint32_t *w, int i, uint32_t b) { w[i >> 1] |= b << ((i & 1) * 16); }
};

template <> struct Elem<__half> {
    static constexpr int WORDS = 4;
    static constexpr uint32_t NEG_INF = 0xfc00u;
    static __device__ __forceinline__ float get(const uint32_t *w, int i)
    {
        return __half2float(__ushort_as_half(static_cast<unsigned short>((i & 1) ? (w[i >> 1] >> 16) : w[i >> 1])));
    }
    static __device__ __forceinline__ float load(const __half *p) { return __half2float(*p); }
    static __device__ __forceinline__ __half from(float x) { return __float2half_rn(x); }
    static __device__ __forceinline__ uint32_t bits(const __half *p) { return __half_as_ushort(*p); }
    static __device__ __forceinline__ void put(uint32_t *w, int i, uint32_t b) { w[i >> 1] |= b << ((i & 1) * 16); }
};

// Two floats to the packed word of a 16-bit type.
template <typename T> __device__ __forceinline__ uint32_t pack2(float lo, float hi);
template <> __device__ __forceinline__ uint32_t pack2<__nv_bfloat16>(float lo, float hi)
{
    const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&v);
}
template <> __device__ __forceinline__ uint32_t pack2<__half>(float lo, float hi)
{
    const __half2 v = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&v);
}

// ---------------------------------------------------------------- eight columns
// Columns col .. col + 7 of a row; columns past V read as -inf.  vec: the row
// starts on a 16-byte boundary (col is a multiple of 8).
template <typename T> struct Raw8 {
    uint32_t w[Elem<T>::WORDS];
};

template <typename T> __device__ __forceinline__ bool row_vec(const T *row)
{
    return (reinterpret_cast<uintptr_t>(row) & 15) == 0;
}

template <typename T> __device__ __forceinline__ void load8(Raw8<T> &r, const T *row, int col, int V, bool vec)
{
    if (vec && col + 8 <= V) {
        const uint4 *p = reinterpret_cast<const uint4 *>(row + col);
#pragma unroll
        for (int k = 0; k < Elem<T>::WORDS / 4; ++k) {
            const uint4 v = p[k];
            r.w[4 * k] = v.x;
            r.w[4 * k + 1] = v.y;
            r.w[4 * k + 2] = v.z;
            r.w[4 * k + 3] = v.w;
        }
        return;
    }
#pragma unroll
    for (int k = 0; k < Elem<T>::WORDS; ++k)
        r.w[k] = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i)
        Elem<T>::put(r.w, i, col + i < V ? Elem<T>::bits(row + col + i) : Elem<T>::NEG_INF);
}

template <typename T> __device__ __forceinline__ void store8(T *row, int col, int V, bool vec, const float *v)
{
    if (vec && col + 8 <= V) {
        uint4 *p = reinterpret_cast<uint4 *>(row + col);
        if constexpr (sizeof(T) == 4) {
            p[0] = make_uint4(__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3]));
            p[1] = make_uint4(__float_as_uint(v[4]), __float_as_uint(v[5]), __float_as_uint(v[6]), __float_as_uint(v[7]));
        } else {
            p[0] = make_uint4(pack2<T>(v[0], v[1]), pack2<T>(v[2], v[3]), pack2<T>(v[4], v[5]), pack2<T>(v[6], v[7]));
        }
        return;
    }
#pragma unroll
    for (int i = 0; i < 8; ++i)
        if (col + i < V)
            row[col + i] = Elem<T>::from(v[i]);
}

// ---------------------------------------------------------------- reductions
__device__ __forceinline__ float finite_ref(float m) { return m == neg_inf() ? 0.f : m; }

// Adds t[0..7] (base-2 exponents) to the lane's running (m, s).
__device__ __forceinline__ void lane_add8(float &m, float &s, const float *t)
{
    const float c = fmaxf(fmaxf(fmaxf(t[0], t[1]), fmaxf(t[2], t[3])), fmaxf(fmaxf(t[4], t[5]), fmaxf(t[6], t[7])));
    const float n = fmaxf(m, c), ref = finite_ref(n);
    float e[8];
#pragma unroll
    for (int i = 0; i < 8; ++i)
        e[i] = exp2_approx(t[i] - ref);
    s = s * exp2_approx(m - ref) + (((e[0] + e[1]) + (e[2] + e[3])) + ((e[4] + e[5]) + (e[6] + e[7])));
    m = n;
}

// The warp's (m, s) from its lanes', in every lane; xor order, so the same in each.
__device__ __forceinline__ void warp_join(float &m, float &s)
{
    float n = m;
#pragma unroll
    for (int d = 16; d > 0; d >>= 1)
        n = fmaxf(n, __shfl_xor_sync(0xffffffffu, n, d));
    s *= exp2_approx(m - finite_ref(n));
#pragma unroll
    for (int d = 16; d > 0; d >>= 1)
        s += __shfl_xor_sync(0xffffffffu, s, d);
    m = n;
}

// Joins (n, t) into (m, s).
__device__ __forceinline__ void join(float &m, float &s, float n, float t)
{
    const float k = fmaxf(m, n), ref = finite_ref(k);
    s = s * exp2_approx(m - ref) + t * exp2_approx(n - ref);
    m = k;
}

// Folds n slice partials (one warp; the same value in every lane): lane l takes
// slices l, l + 32, ... in order, then the lanes join.
__device__ __forceinline__ void fold_slices(const float2 *part, int n, int lane, float &m, float &s)
{
    m = neg_inf();
    s = 0.f;
    for (int i = lane; i < n; i += 32) {
        join(m, s, part[i].x, part[i].y);
    }
    warp_join(m, s);
}

// Natural log of a folded row's sum of exponentials: -inf for an empty row, NaN
// where the row held a NaN or +inf.
__device__ __forceinline__ float row_lse(float m, float s)
{
    return s == 0.f ? neg_inf() : (m + log2f(s)) * LG_LN2;
}

// log-probability of a column with base-2 exponent t (from the pair, not from
// the rounded lse: exact to the rounding of a small number near 0).
__device__ __forceinline__ float row_logp(float t, float m, float s)
{
    if (s == 0.f || (t == neg_inf() && s == s))
        return neg_inf();
    return ((t - m) - log2f(s)) * LG_LN2;
}

__device__ __forceinline__ void report_bad_input(int *status)
{
    atomicCAS(status, 0, static_cast<int>(TIM_ERR_BAD_INPUT));
}

__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }

__device__ __forceinline__ void st_cluster_f2(uint32_t addr, float x, float y)
{
    asm volatile("st.shared::cluster.v2.f32 [%0], {%1, %2};" ::"r"(addr), "f"(x), "f"(y) : "memory");
}

} // namespace tim
