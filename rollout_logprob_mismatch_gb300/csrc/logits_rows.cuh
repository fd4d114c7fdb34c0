// logits_rows.cuh -- device code shared by the operators on a head's logits:
// eight columns of a row at a time (any element type, any alignment), and the
// reduction of a slice of a row to (maximum, sum of exponentials).
//
// Log-sum-exp of y = x / tau: a set of columns is the pair (M, S), M = max x,
// S = sum e^((x - M) / tau) = sum 2^((x - M) k2), k2 = log2(e) / tau; two sets join
// as M = max(M1, M2), S = S1 2^((M1 - M) k2) + S2 2^((M2 - M) k2); lse = M / tau +
// log S.  The difference comes before the scale: the largest column's term is
// exactly 1, and a row of the type's lowest values does not overflow.  A set of
// -inf columns only is (-inf, 0).  NaN and +inf make S NaN.
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

__device__ __forceinline__ float neg_inf() { return __int_as_float(static_cast<int>(0xff800000u)); }
__device__ __forceinline__ float quiet_nan() { return __int_as_float(0x7fc00000); }

__device__ __forceinline__ float exp2_approx(float x)   // 2 ulp; 2^-inf = 0, 2^nan = nan
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

__device__ __forceinline__ float fmin_nan(float x, float y)   // NaN if either is
{
    float m;
    asm("min.NaN.f32 %0, %1, %2;" : "=f"(m) : "f"(x), "f"(y));
    return m;
}

// 2^x of a probability from a rounded log-sum-exp: at most 1.  (Where |lse| passes
// some 1e6, as in a row of an additive mask's values, its rounding alone is more than
// the logarithm of any vocabulary, and 2^x without the limit may be 1e28.)
__device__ __forceinline__ float prob2(float x) { return exp2_approx(fmin_nan(x, 0.f)); }

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
// Columns col .. col + 7 of a row (col a multiple of 8, lanes side by side: a
// warp covers 256 columns); columns past V read as -inf.
//
// A row that does not start on a 16-byte boundary (an odd V) is read in aligned
// 16-byte pieces all the same: the pieces around the eight columns, shifted
// together; the overlap with the next lane comes from L1.  Element loads in their
// place took 2.2 times as long (500 rows of 50261 fp16 logits).  Stores hand the
// tail of one lane's columns to the next lane and write aligned pieces.  A row's
// first and last columns go element by element, so no access leaves the row.
template <typename T> struct Raw8 {
    uint32_t w[Elem<T>::WORDS];
};

// Bytes from the 16-byte boundary before the row's start (every chunk's too).
template <typename T> __device__ __forceinline__ uint32_t row_shift(const T *row)
{
    return static_cast<uint32_t>(reinterpret_cast<uintptr_t>(row) & 15);
}

// w[i] of the byte sequence q read from byte `shift` on (shift below 16, a
// multiple of the element size; W + 4 words in q).
template <int W, bool HALVES> __device__ __forceinline__ void shift_words(uint32_t *w, uint32_t *q, uint32_t shift)
{
#pragma unroll
    for (int i = 0; i < W + 2; ++i)
        q[i] = shift & 8 ? q[i + 2] : q[i];
#pragma unroll
    for (int i = 0; i < W + 1; ++i)
        q[i] = shift & 4 ? q[i + 1] : q[i];
#pragma unroll
    for (int i = 0; i < W; ++i)
        w[i] = HALVES && (shift & 2) ? __funnelshift_r(q[i], q[i + 1], 16) : q[i];
}

template <typename T>
__device__ __forceinline__ void load8(Raw8<T> &r, const T *row, int col, int V, uint32_t shift)
{
    constexpr int W = Elem<T>::WORDS;
    if (shift == 0 ? col + 8 <= V : col >= 8 && col + 16 <= V) {
        const uint4 *p = reinterpret_cast<const uint4 *>(reinterpret_cast<const char *>(row + col) - shift);
        if (shift == 0) {
#pragma unroll
            for (int k = 0; k < W / 4; ++k) {
                const uint4 v = p[k];
                r.w[4 * k] = v.x;
                r.w[4 * k + 1] = v.y;
                r.w[4 * k + 2] = v.z;
                r.w[4 * k + 3] = v.w;
            }
        } else {
            uint32_t q[W + 4];
#pragma unroll
            for (int k = 0; k < W / 4 + 1; ++k) {
                const uint4 v = p[k];
                q[4 * k] = v.x;
                q[4 * k + 1] = v.y;
                q[4 * k + 2] = v.z;
                q[4 * k + 3] = v.w;
            }
            shift_words<W, sizeof(T) == 2>(r.w, q, shift);
        }
        return;
    }
#pragma unroll
    for (int k = 0; k < W; ++k)
        r.w[k] = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i)
        Elem<T>::put(r.w, i, col + i < V ? Elem<T>::bits(row + col + i) : Elem<T>::NEG_INF);
}

// The lane's eight values, rounded to T and packed.
template <typename T> __device__ __forceinline__ Raw8<T> pack8(const float *v)
{
    Raw8<T> r;
#pragma unroll
    for (int k = 0; k < Elem<T>::WORDS; ++k) {
        if constexpr (sizeof(T) == 4)
            r.w[k] = __float_as_uint(v[k]);
        else
            r.w[k] = pack2<T>(v[2 * k], v[2 * k + 1]);
    }
    return r;
}

// Element i of the lane's eight to its place.
template <typename T> __device__ __forceinline__ void store1(T *row, int col, const Raw8<T> &r, int i)
{
    if constexpr (sizeof(T) == 4)
        reinterpret_cast<uint32_t *>(row)[col + i] = r.w[i];
    else
        reinterpret_cast<uint16_t *>(row)[col + i] = static_cast<uint16_t>(r.w[i >> 1] >> ((i & 1) * 16));
}

// Stores the lane's eight; the whole warp, col = its lane's column.
template <typename T>
__device__ __forceinline__ void store8(T *row, int col, int V, uint32_t shift, const Raw8<T> &r)
{
    constexpr int W = Elem<T>::WORDS;
    const int lane = threadIdx.x & 31;
    const bool whole = col - lane * 8 + 256 <= V;   // the same in every lane
    if (shift == 0 ? col + 8 <= V : whole) {
        if (shift == 0) {
            uint4 *p = reinterpret_cast<uint4 *>(row + col);
#pragma unroll
            for (int k = 0; k < W / 4; ++k)
                p[k] = make_uint4(r.w[4 * k], r.w[4 * k + 1], r.w[4 * k + 2], r.w[4 * k + 3]);
            return;
        }
        // the 16 bytes before this lane's columns are the lane before's last
        uint32_t q[W + 4], o[W];
#pragma unroll
        for (int k = 0; k < 4; ++k)
            q[k] = __shfl_up_sync(0xffffffffu, r.w[W - 4 + k], 1);
#pragma unroll
        for (int k = 0; k < W; ++k)
            q[4 + k] = r.w[k];
        shift_words<W, sizeof(T) == 2>(o, q, 16 - shift);
        uint4 *p = reinterpret_cast<uint4 *>(reinterpret_cast<char *>(row + col) - shift);
        const int head = static_cast<int>((16 - shift) / sizeof(T));   // own elements in the first piece
        if (lane != 0)
            p[0] = make_uint4(o[0], o[1], o[2], o[3]);
        if constexpr (W == 8)
            p[1] = make_uint4(o[4], o[5], o[6], o[7]);
        if (lane == 0) {
#pragma unroll
            for (int i = 0; i < 8; ++i)
                if (i < head)
                    store1(row, col, r, i);
        }
        if (lane == 31) {
            const int tail = static_cast<int>(shift / sizeof(T));
#pragma unroll
            for (int i = 0; i < 8; ++i)
                if (i >= 8 - tail)
                    store1(row, col, r, i);
        }
        return;
    }
#pragma unroll
    for (int i = 0; i < 8; ++i)
        if (col + i < V)
            store1(row, col, r, i);
}

// N chunks of 256 columns from column b on, into N registers of eight a lane.  Away
// from a row's end, in an aligned row, nothing has to be looked at per load.
template <typename T, int N>
__device__ __forceinline__ void load_chunks(Raw8<T> (&r)[N], const T *row, int b, int V, uint32_t shift)
{
    constexpr int W = Elem<T>::WORDS;
    const int lane = threadIdx.x & 31;
    if (shift == 0 && b + N * 256 <= V) {
        const uint4 *p = reinterpret_cast<const uint4 *>(row + b) + lane * (W / 4);
#pragma unroll
        for (int u = 0; u < N; ++u)
#pragma unroll
            for (int k = 0; k < W / 4; ++k) {
                const uint4 v = p[u * 8 * W + k];
                r[u].w[4 * k] = v.x;
                r[u].w[4 * k + 1] = v.y;
                r[u].w[4 * k + 2] = v.z;
                r[u].w[4 * k + 3] = v.w;
            }
        return;
    }
#pragma unroll
    for (int u = 0; u < N; ++u)
        load8<T>(r[u], row, b + u * 256 + lane * 8, V, shift);
}

// For 16-bit types: the masks of two words whose halves' bits are set in a nibble
// (128 bytes of shared memory; two 8-byte loads and a logic operation a word in
// place of some 28 instructions per eight columns).
struct HalfMasks {
    uint2 of[16];
    __device__ __forceinline__ void fill()   // a barrier before use
    {
        if (threadIdx.x < 16) {
            const uint32_t b = threadIdx.x;
            of[b] = make_uint2((b & 1 ? 0xffffu : 0u) | (b & 2 ? 0xffff0000u : 0u),
                               (b & 4 ? 0xffffu : 0u) | (b & 8 ? 0xffff0000u : 0u));
        }
    }
};

// Columns whose bit in `drop` is set become `fill` (the bits of one element).
template <typename T>
__device__ __forceinline__ void drop8(Raw8<T> &r, uint32_t drop, const HalfMasks &masks, uint32_t fill = Elem<T>::NEG_INF)
{
    if constexpr (sizeof(T) == 4) {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            r.w[i] = drop >> i & 1 ? fill : r.w[i];
    } else {
        const uint32_t two = fill | fill << 16;
        const uint2 lo = masks.of[drop & 15], hi = masks.of[drop >> 4];
        r.w[0] = (r.w[0] & ~lo.x) | (two & lo.x);
        r.w[1] = (r.w[1] & ~lo.y) | (two & lo.y);
        r.w[2] = (r.w[2] & ~hi.x) | (two & hi.x);
        r.w[3] = (r.w[3] & ~hi.y) | (two & hi.y);
    }
}

// ---------------------------------------------------------------- packed pairs of fp32
using Pair = unsigned long long;

__device__ __forceinline__ Pair pair(float lo, float hi)
{
    Pair p;
    asm("mov.b64 %0, {%1, %2};" : "=l"(p) : "f"(lo), "f"(hi));
    return p;
}
__device__ __forceinline__ void unpair(Pair p, float &lo, float &hi)
{
    asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(p));
}
__device__ __forceinline__ Pair add2(Pair a, Pair b)
{
    Pair p;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(p) : "l"(a), "l"(b));
    return p;
}
__device__ __forceinline__ Pair mul2(Pair a, Pair b)
{
    Pair p;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(p) : "l"(a), "l"(b));
    return p;
}
__device__ __forceinline__ Pair fma2(Pair a, Pair b, Pair c)
{
    Pair p;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(p) : "l"(a), "l"(b), "l"(c));
    return p;
}

// x / tau by the rounded reciprocal and one residual step: q = x inv, q + (x - q tau) inv.
// q is off by up to 1.5 units in the last place, the step by that times 2^-24 before its
// own rounding, so x / tau is off by (1/2 + 2^-20) of one.  An infinite or NaN q stays as it is.
__device__ __forceinline__ float quotient(float x, float tau, float inv)
{
    const float q = __fmul_rn(x, inv);
    const float better = __fmaf_rn(__fmaf_rn(-q, tau, x), inv, q);
    return fabsf(q) < INFINITY ? better : q;
}
__device__ __forceinline__ void quotient2(Pair x, Pair minus_tau, Pair inv, float &lo, float &hi)   // two, the same bits
{
    const Pair q = mul2(x, inv);
    float q0, q1;
    unpair(q, q0, q1);
    unpair(fma2(fma2(q, minus_tau, x), inv, q), lo, hi);
    lo = fabsf(q0) < INFINITY ? lo : q0;
    hi = fabsf(q1) < INFINITY ? hi : q1;
}
template <typename T> __device__ __forceinline__ Pair get2(const Raw8<T> &r, int k)   // columns 2k, 2k + 1
{
    return pair(Elem<T>::get(r.w, 2 * k), Elem<T>::get(r.w, 2 * k + 1));
}

// ---------------------------------------------------------------- reductions
// Products are rounded on their own (__fmul_rn) and sums in a fixed form, so that
// no kernel contracts them in its own way: every entry point gives a row the
// same sums.
__device__ __forceinline__ float finite_ref(float m) { return m == neg_inf() ? 0.f : m; }

__device__ __forceinline__ float warp_max(float x)   // NaN lanes do not count
{
    float y;
    asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(y) : "f"(x));
    return y;
}

__device__ __forceinline__ float warp_sum(float x)   // xor order: the same bits in every lane
{
#pragma unroll
    for (int d = 16; d > 0; d >>= 1)
        x += __shfl_xor_sync(0xffffffffu, x, d);
    return x;
}

// The largest of n * 8 raw columns (NaN ones do not count).
template <typename T, int N> __device__ __forceinline__ float raw_max(const Raw8<T> (&raw)[N])
{
    if constexpr (sizeof(T) == 4) {
        float m = neg_inf();
#pragma unroll
        for (int u = 0; u < N; ++u)
#pragma unroll
            for (int k = 0; k < 4; ++k)
                asm("max.f32 %0, %0, %1, %2;"
                    : "+f"(m)
                    : "f"(__uint_as_float(raw[u].w[2 * k])), "f"(__uint_as_float(raw[u].w[2 * k + 1])));
        return m;
    } else {
        uint32_t m = raw[0].w[0];
#pragma unroll
        for (int u = 0; u < N; ++u)
#pragma unroll
            for (int k = 0; k < 4; ++k)
                if constexpr (Elem<T>::NEG_INF == 0xff80u)
                    asm("max.bf16x2 %0, %0, %1;" : "+r"(m) : "r"(raw[u].w[k]));
                else
                    asm("max.f16x2 %0, %0, %1;" : "+r"(m) : "r"(raw[u].w[k]));
        return fmaxf(Elem<T>::get(&m, 0), Elem<T>::get(&m, 1));
    }
}

// (M, S), in every lane, of a warp's columns and of the n values at `more`: the
// largest first (with packed maxima on the raw 16-bit pairs), then the sum.
template <typename T, int N>
__device__ __forceinline__ void warp_sums(const Raw8<T> (&raw)[N], float k2, const uint32_t *more, int n, float &M,
                                          float &S)
{
    const int lane = threadIdx.x & 31;
    const float first = lane < n ? __uint_as_float(more[lane]) : neg_inf();
    float top = fmaxf(raw_max<T, N>(raw), first);
    for (int i = lane + 32; i < n; i += 32)
        top = fmaxf(top, __uint_as_float(more[i]));
    M = warp_max(top);
    const float ref = finite_ref(M);
    const Pair neg = pair(-ref, -ref), kk = pair(k2, k2);
    Pair acc[2] = {pair(0.f, 0.f), pair(0.f, 0.f)};
#pragma unroll
    for (int u = 0; u < N; ++u)
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            float lo, hi;
            unpair(mul2(add2(get2<T>(raw[u], k), neg), kk), lo, hi);
            acc[k & 1] = add2(acc[k & 1], pair(exp2_approx(lo), exp2_approx(hi)));
        }
    float lo, hi;
    unpair(add2(acc[0], acc[1]), lo, hi);
    lo += hi;
    if (n > 0)
        lo += exp2_approx(__fmul_rn(first - ref, k2));
    for (int i = lane + 32; i < n; i += 32)
        lo += exp2_approx(__fmul_rn(__uint_as_float(more[i]) - ref, k2));
    S = warp_sum(lo);
}

// Joins (n, t) into (m, s).
__device__ __forceinline__ void join(float &m, float &s, float n, float t, float k2)
{
    const float k = fmaxf(m, n), ref = finite_ref(k);
    s = __fmaf_rn(s, exp2_approx(__fmul_rn(m - ref, k2)), __fmul_rn(t, exp2_approx(__fmul_rn(n - ref, k2))));
    m = k;
}

// Adds one column to a lane's (m, s).
__device__ __forceinline__ void join_value(float &m, float &s, float x, float k2)
{
    join(m, s, x, x == neg_inf() ? 0.f : 1.f, k2);
}

// The warp's (m, s) from its lanes', in every lane.
__device__ __forceinline__ void warp_join(float &m, float &s, float k2)
{
    const float n = warp_max(m);
    s = warp_sum(__fmul_rn(s, exp2_approx(__fmul_rn(m - finite_ref(n), k2))));
    m = n;
}

// Natural log of a folded row's sum of exponentials: -inf for an empty row, NaN
// where the row held a NaN or +inf.
__device__ __forceinline__ float row_lse(float m, float s, float inv_tau)
{
    return s == 0.f ? neg_inf() : __fmaf_rn(m, inv_tau, logf(s));
}

// log-probability of a column x (from the pair, not from the rounded lse: a
// probability near 1 keeps its digits).
__device__ __forceinline__ float row_logp(float x, float m, float s, float inv_tau)
{
    if (s == 0.f || (x == neg_inf() && s == s))
        return neg_inf();
    return __fmaf_rn(x - m, inv_tau, -logf(s));
}

__device__ __forceinline__ void report_bad_input(int *status)
{
    atomicCAS(status, 0, static_cast<int>(TIM_ERR_BAD_INPUT));
}

// (relaxed: the CTA runs, and what a fence released before it; no store of this
// thread is waited for)
__device__ __forceinline__ void cluster_arrive_relaxed() { asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }

__device__ __forceinline__ void st_cluster_f2(uint32_t addr, float x, float y)
{
    asm volatile("st.shared::cluster.v2.f32 [%0], {%1, %2};" ::"r"(addr), "f"(x), "f"(y) : "memory");
}

} // namespace tim
