// adapters.cuh -- device code shared by the adapters' kernels: bf16 parts of fp32
// values and the warp's 16 x 8 x 16 product.
#pragma once

#include <cfloat>

#include "logits_rows.cuh"

namespace tim {

// D (16 x 8, fp32) += A (16 x 16) B (16 x 8), bf16.  Lane l = 4 g + q holds rows g and
// g + 8 of A (k pairs 2q and 2q + 8), column g of B (the same k pairs), and columns 2q
// and 2q + 1 of D in rows g and g + 8.  The order of k is the caller's as long as A and
// B agree: the kernels here give a lane four (or eight) neighbouring k in place of two
// pairs, so that its operands come in 8- and 16-byte loads.
__device__ __forceinline__ void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1)
{
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// x = p[0] + p[1] + ... up to half a unit of the last part: each part is what the ones
// before leave, rounded to bf16 (2^-8 of it at most, so two parts leave 2^-16 |x| and
// three 2^-24).  A finite x above bf16's largest value has that as its part 0; an infinite
// or NaN x is all in part 0.
template <int PARTS> __device__ __forceinline__ void split_bf16(float x, uint16_t (&p)[PARTS])
{
    const bool finite = fabsf(x) <= FLT_MAX;
#pragma unroll
    for (int i = 0; i < PARTS; ++i) {
        uint16_t b = __bfloat16_as_ushort(__float2bfloat16_rn(x));
        if (i == 0 && finite && (b & 0x7fffu) == 0x7f80u)
            b -= 1;   // rounded to infinity: the largest of its sign
        p[i] = i == 0 || finite ? b : uint16_t(0);
        x -= __uint_as_float(static_cast<uint32_t>(b) << 16);
    }
}

// Eight values as P planes of packed bf16 parts, split_bf16 of each.
template <int P> __device__ __forceinline__ void split8(const float (&x)[8], uint32_t (&o)[P][4])
{
    float most = 0.f;
    if (P > 1) {
#pragma unroll
        for (int k = 0; k < 8; ++k)
            most = fmaxf(most, fabsf(x[k]));
    }
    const bool finite = most <= 3.38953139e38f;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        float lo = x[2 * k], hi = x[2 * k + 1];
#pragma unroll
        for (int i = 0; i < P; ++i) {
            o[i][k] = pack2<__nv_bfloat16>(lo, hi);
            lo -= __uint_as_float(o[i][k] << 16);
            hi -= __uint_as_float(o[i][k] & 0xffff0000u);
        }
    }
    if (P > 1 && !finite) {
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            uint16_t a[P], b[P];
            split_bf16<P>(x[2 * k], a);
            split_bf16<P>(x[2 * k + 1], b);
#pragma unroll
            for (int i = 0; i < P; ++i)
                o[i][k] = a[i] | static_cast<uint32_t>(b[i]) << 16;
        }
    }
}

// A whole warp waits for a barrier's phase; the same answer in every lane (false: some
// lane's wait ran out, or another role's did), so that the warp leaves its loops together.
__device__ __forceinline__ bool warp_wait(uint32_t bar, uint32_t parity, volatile int *abort, uint64_t budget_ns)
{
    return __all_sync(0xffffffffu, mbar_wait_sleep(bar, parity, abort, budget_ns));
}

// Columns c0 .. c1 - 1 of a row of V on their way to shared memory at st (16-byte
// aligned), where they keep their address's low bits: the aligned pieces inside the row
// as one bulk copy, which the caller issues, the elements before and behind them at once
// (no access leaves the row).  Ends with a fence towards the copies.
struct RowCopy {
    const char *src;
    uint32_t off, bytes;   // into st + off
};

template <typename T> __device__ __forceinline__ RowCopy stage_row(const T *row, int c0, int c1, int V, uint8_t *st)
{
    const uintptr_t lo = reinterpret_cast<uintptr_t>(row + c0), hi = reinterpret_cast<uintptr_t>(row + c1);
    const uintptr_t from = lo & ~uintptr_t(15), end = reinterpret_cast<uintptr_t>(row + V);
    uintptr_t x = from, y = (hi + 15) & ~uintptr_t(15);
    if (x < reinterpret_cast<uintptr_t>(row))
        x += 16;
    if (y > end)
        y = end & ~uintptr_t(15);
    for (uintptr_t k = lo; k < min(hi, x); k += sizeof(T))
        *reinterpret_cast<T *>(st + (k - from)) = *reinterpret_cast<const T *>(k);
    for (uintptr_t k = max(lo, max(x, y)); k < hi; k += sizeof(T))
        *reinterpret_cast<T *>(st + (k - from)) = *reinterpret_cast<const T *>(k);
    fence_proxy_async_smem();
    RowCopy c;
    c.src = reinterpret_cast<const char *>(x);
    c.off = static_cast<uint32_t>(x - from);
    c.bytes = y > x ? static_cast<uint32_t>(y - x) : 0u;
    return c;
}

} // namespace tim
