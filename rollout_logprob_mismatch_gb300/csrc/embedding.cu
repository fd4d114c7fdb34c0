// embedding.cu -- lookup of the table's rows with a scale, and the table's gradient
// by sorted tokens (sm_103a).
//
//   out_n = s W[t_n],   dW[v] (+)= s sum over n with t_n = v of g_n
//
// The lookup is a copy: a warp moves pieces of 256 columns.  The gradient first orders
// the tokens by id in one launch: each CTA owns EM_RANGE ids, counts the tokens below
// them, takes its own in order and orders those by counting, so that nothing has to be
// cleared and no atomic decides an order.  Then every row of dW is written once, with
// the sum of its tokens' gradients taken in the tokens' order; rows of many tokens are
// summed in tiles of sorted positions first, so that one frequent id does not hold one
// warp for the whole call.  The order of a row's sum depends on N and its tokens' sorted
// positions alone: the same call gives the same bits.
#include <algorithm>

#include "logits_rows.cuh"
#include "table_internal.h"
#include "tim_internal.h"

namespace tim {
namespace {

// ---------------------------------------------------------------- lookup
// 32768 x 4096 bf16: 86 us, 0.93 of the copy rate counting repeated rows as read once each time.
// Unit u = (token u / pieces, piece u % pieces of 256 columns); a warp takes PER units.
template <typename TW, typename TO, int PER>
__global__ void __launch_bounds__(256) embedding_kernel(const EmbeddingArgs a)
{
    const int lane = threadIdx.x & 31;
    const uint32_t pieces = (static_cast<uint32_t>(a.D) + 255) / 256;
    const uint32_t units = static_cast<uint32_t>(a.N) * pieces;
    const uint32_t u0 = (blockIdx.x * 8u + (threadIdx.x >> 5)) * PER;
    const TW *W = static_cast<const TW *>(a.x);
    TO *out = static_cast<TO *>(a.out);
    pdl_wait();
    pdl_launch_dependents();
    Raw8<TW> r[PER];
    bool live[PER];
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        const uint32_t u = u0 + i;
        live[i] = false;
        if (u >= units)
            continue;
        const int col = static_cast<int>(u % pieces) * 256 + lane * 8;
        const int id = a.tokens[u / pieces];
        live[i] = static_cast<unsigned>(id) < static_cast<unsigned>(a.V);
        if (live[i] && col < a.D) {
            const TW *row = W + static_cast<size_t>(id) * a.D;
            load8<TW>(r[i], row, col, a.D, row_shift(row));
        }
    }
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        const uint32_t u = u0 + i;
        if (u >= units)
            continue;   // the same in every lane
        const int col = static_cast<int>(u % pieces) * 256 + lane * 8;
        TO *row = out + static_cast<size_t>(u / pieces) * a.D;
        float v[8];
#pragma unroll
        for (int k = 0; k < 8; ++k)
            v[k] = live[i] ? Elem<TW>::get(r[i].w, k) * a.scale : 0.f;
        store8<TO>(row, col, a.D, row_shift(row), pack8<TO>(v));
    }
}

// ---------------------------------------------------------------- order by id
// 32768 tokens, 128256 ids: 23 us, the chain of three passes over a CTA's part of the list.
__device__ __forceinline__ int warp_scan(int x)   // inclusive
{
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(0xffffffffu, x, o);
        x += lane >= o ? v : 0;
    }
    return x;
}

__global__ void __launch_bounds__(EM_SORT_THREADS) embedding_sort_kernel(const EmbeddingArgs a)
{
    constexpr int WARPS = EM_SORT_THREADS / 32;
    static_assert(EM_RANGE <= EM_SORT_THREADS, "a thread scans one id's counts");
    extern __shared__ int counts_of[];
    int (&counts)[WARPS][EM_RANGE] = *reinterpret_cast<int (*)[WARPS][EM_RANGE]>(counts_of);   // a warp's tokens of each id, then where its next one goes
    __shared__ int sb[WARPS], so[WARPS], sums[WARPS];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int lo = blockIdx.x * EM_RANGE, hi = min(a.V, lo + EM_RANGE);
    for (int i = tid; i < WARPS * EM_RANGE; i += EM_SORT_THREADS)
        (&counts[0][0])[i] = 0;
    pdl_wait();
    pdl_launch_dependents();
    // ids outside [0, V) have no row.  Each warp has a part of the list, in order.
    const int per = ((a.N + 31) / 32 + WARPS - 1) / WARPS * 32;
    const int n0 = min(a.N, warp * per), n1 = min(a.N, n0 + per);
    int below = 0, own = 0;
#pragma unroll 8
    for (int n = n0 + lane; n < n1; n += 32) {
        const int id = a.tokens[n];
        below += id >= 0 && id < lo;
        own += id >= lo && id < hi;
    }
    below = __reduce_add_sync(0xffffffffu, below);
    own = __reduce_add_sync(0xffffffffu, own);
    if (lane == 0) {
        sb[warp] = below;
        so[warp] = own;
    }
    __syncthreads();
    int base = 0, total = 0, at = 0;
#pragma unroll
    for (int w = 0; w < WARPS; ++w) {
        base += sb[w];
        total += so[w];
        at += w < warp ? so[w] : 0;
    }
    at += base;
    if (own > 0) {
#pragma unroll 8
        for (int n = n0; n < n1; n += 32) {
            const int id = n + lane < n1 ? a.tokens[n + lane] : -1;
            const bool in = id >= lo && id < hi;
            const unsigned all = __ballot_sync(0xffffffffu, in);
            TIM_DCHECK(!in || at + __popc(all) <= base + total, a.status, TIM_CHECK_STORE, n + lane, id);
            if (in)
                a.staged[at + __popc(all & ((1u << lane) - 1u))] = make_int2(id, n + lane);
            at += __popc(all);
        }
    }
    __syncthreads();
    // each warp has a part of the CTA's tokens, whole groups of 32
    const int part = ((total + 31) / 32 + WARPS - 1) / WARPS * 32;
    const int p0 = min(total, warp * part), p1 = min(total, p0 + part);
#pragma unroll 4
    for (int p = p0 + lane; p < p1; p += 32)
        atomicAdd(&counts[warp][a.staged[base + p].x - lo], 1);
    __syncthreads();
    // where each id starts, and where each warp's tokens of it do
    int mine = 0;
    if (tid < EM_RANGE) {
#pragma unroll
        for (int w = 0; w < WARPS; ++w)
            mine += counts[w][tid];
    }
    const int scan = warp_scan(mine);
    if (lane == 31)
        sums[warp] = scan;
    __syncthreads();
    int start = base + scan - mine;
#pragma unroll
    for (int w = 0; w < WARPS; ++w)
        start += w < warp ? sums[w] : 0;
    if (lo + tid < hi)
        a.offsets[lo + tid] = start;
    if (tid < EM_RANGE) {
#pragma unroll
        for (int w = 0; w < WARPS; ++w) {
            const int c = counts[w][tid];
            counts[w][tid] = start;
            start += c;
        }
    }
    if (hi == a.V && tid == 0)
        a.offsets[a.V] = base + total;
    __syncthreads();
    constexpr int GROUPS = 4;   // of 32 tokens, loaded together
    for (int p = p0; p < p1; p += 32 * GROUPS) {
        int2 x[GROUPS];
#pragma unroll
        for (int i = 0; i < GROUPS; ++i)
            x[i] = p + i * 32 + lane < p1 ? a.staged[base + p + i * 32 + lane] : make_int2(-1, 0);
#pragma unroll
        for (int i = 0; i < GROUPS; ++i) {
            const unsigned same = __match_any_sync(0xffffffffu, x[i].x);
            const int rank = __popc(same & ((1u << lane) - 1u));
            int to = 0;
            if (x[i].x >= 0)
                to = counts[warp][x[i].x - lo] + rank;
            __syncwarp();
            if (x[i].x >= 0 && rank == 0)
                counts[warp][x[i].x - lo] += __popc(same);
            __syncwarp();
            TIM_DCHECK(x[i].x < 0 || (to >= base && to < base + total), a.status, TIM_CHECK_STORE, to, x[i].x);
            if (x[i].x >= 0) {
                a.order[to] = x[i].y;
                a.ids[to] = x[i].x;
            }
        }
    }
}

// ---------------------------------------------------------------- sums
// A warp's columns: EM_PIECES pieces of 256 from col0 on, eight of each a lane: side by
// side (VEC: rows that start on 16 bytes), else every 32nd, element by element (a warp's
// accesses then lie together whatever the row's alignment).
constexpr int EM_PIECES = 2;
constexpr int EM_COLS = EM_PIECES * 256;
constexpr int EM_AHEAD = 4;   // tokens whose rows are in flight together

template <typename T, bool VEC> struct Pieces {
    Raw8<T> r[EM_PIECES];
    __device__ __forceinline__ void load(const T *row, int col0, int D)
    {
        const int lane = threadIdx.x & 31;
#pragma unroll
        for (int i = 0; i < EM_PIECES; ++i) {
            if constexpr (VEC) {
                const int col = col0 + i * 256 + lane * 8;
                if (col < D) {   // D is a multiple of 8
                    const uint4 *p = reinterpret_cast<const uint4 *>(row + col);
#pragma unroll
                    for (int k = 0; k < Elem<T>::WORDS / 4; ++k) {
                        const uint4 v = p[k];
                        r[i].w[4 * k] = v.x;
                        r[i].w[4 * k + 1] = v.y;
                        r[i].w[4 * k + 2] = v.z;
                        r[i].w[4 * k + 3] = v.w;
                    }
                }
            } else {
#pragma unroll
                for (int k = 0; k < Elem<T>::WORDS; ++k)
                    r[i].w[k] = 0;
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                    const int col = col0 + i * 256 + k * 32 + lane;
                    if (col < D)
                        Elem<T>::put(r[i].w, k, Elem<T>::bits(row + col));
                }
            }
        }
    }
    __device__ __forceinline__ void add_to(float (&acc)[EM_PIECES][8]) const
    {
#pragma unroll
        for (int i = 0; i < EM_PIECES; ++i)
#pragma unroll
            for (int k = 0; k < 8; ++k)
                acc[i][k] += Elem<T>::get(r[i].w, k);
    }
};

// dst = acc * scale (+ dst)
template <bool VEC>
__device__ __forceinline__ void put_row(float *dst, const float (&acc)[EM_PIECES][8], int col0, int D, float scale, bool add)
{
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int i = 0; i < EM_PIECES; ++i) {
        if constexpr (VEC) {
            const int col = col0 + i * 256 + lane * 8;
            if (col < D) {
                float4 *p = reinterpret_cast<float4 *>(dst + col);
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    float4 v = make_float4(__fmul_rn(acc[i][4 * k], scale), __fmul_rn(acc[i][4 * k + 1], scale), __fmul_rn(acc[i][4 * k + 2], scale),
                                           __fmul_rn(acc[i][4 * k + 3], scale));
                    if (add) {
                        const float4 y = p[k];
                        v.x += y.x;
                        v.y += y.y;
                        v.z += y.z;
                        v.w += y.w;
                    }
                    p[k] = v;
                }
            }
        } else {
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                const int col = col0 + i * 256 + k * 32 + lane;
                if (col < D)
                    dst[col] = add ? __fmul_rn(acc[i][k], scale) + dst[col] : acc[i][k] * scale;
            }
        }
    }
}

// acc += the rows of sorted positions b .. e - 1, in order.
template <typename T, bool VEC>
__device__ __forceinline__ void sum_positions(float (&acc)[EM_PIECES][8], const EmbeddingArgs &a, int b, int e, int col0)
{
    const T *x = static_cast<const T *>(a.x);
    const int lane = threadIdx.x & 31;
    for (int p0 = b; p0 < e; p0 += 32) {
        const int mine = p0 + lane < e ? a.order[p0 + lane] : 0;
        TIM_DCHECK(static_cast<unsigned>(mine) < static_cast<unsigned>(a.N), a.status, TIM_CHECK_UNIT, p0 + lane, mine);
        const int count = min(32, e - p0);
        for (int j = 0; j < count; j += EM_AHEAD) {
            Pieces<T, VEC> r[EM_AHEAD];
#pragma unroll
            for (int i = 0; i < EM_AHEAD; ++i)
                if (j + i < count)
                    r[i].load(x + static_cast<size_t>(__shfl_sync(0xffffffffu, mine, j + i)) * a.D, col0, a.D);
#pragma unroll
            for (int i = 0; i < EM_AHEAD; ++i)
                if (j + i < count)
                    r[i].add_to(acc);
        }
    }
}

// Two kinds of CTAs.  The first tile_ctas: tiles of a.tile sorted positions, a warp EM_COLS
// columns of one: the part of a tile that belongs to an id of more than a.many tokens is
// summed into partial[tile][0] where the id goes on from the tile before, into
// partial[tile][1] where it begins in the tile.  The others: zeros for the rows of dW that
// no token has, EM_IDS rows a warp (nothing but stores, and a read of the offsets).
// 128256 x 4096, 32768 bf16 tokens: 258 us, 1.74 GB, the copy rate.
template <typename T, bool VEC>
__global__ void __launch_bounds__(256, 2) embedding_tiles_kernel(const EmbeddingArgs a, int tile_ctas, int column_blocks)
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    pdl_wait();
    pdl_launch_dependents();
    if (blockIdx.x >= tile_ctas) {
        const int id0 = (static_cast<int>(blockIdx.x - tile_ctas) * 8 + warp) * EM_IDS;
        if (id0 >= a.V)
            return;
        const int at = lane <= EM_IDS ? a.offsets[min(a.V, id0 + lane)] : 0;
        for (int i = 0; i < EM_IDS && id0 + i < a.V; ++i) {
            if (__shfl_sync(0xffffffffu, at, i) != __shfl_sync(0xffffffffu, at, i + 1))
                continue;
            float *row = a.dW + static_cast<size_t>(id0 + i) * a.D;
            // up to a 16-byte boundary, whole 16 bytes, the rest
            const int head = VEC ? 0 : min(a.D, static_cast<int>((16 - (reinterpret_cast<uintptr_t>(row) & 15)) / 4 & 3));
            const int whole = head + (a.D - head) / 4 * 4;
            if (lane < head)
                row[lane] = 0.f;
#pragma unroll 4
            for (int c = head + lane * 4; c < whole; c += 128)
                *reinterpret_cast<float4 *>(row + c) = make_float4(0.f, 0.f, 0.f, 0.f);
            if (whole + lane < a.D)
                row[whole + lane] = 0.f;
        }
        return;
    }
    const int unit = static_cast<int>(blockIdx.x) * 8 + warp;
    const int tile = unit / column_blocks, col0 = unit % column_blocks * EM_COLS;
    const int total = a.offsets[a.V];
    if (tile >= (total + a.tile - 1) / a.tile)
        return;
    const int p0 = tile * a.tile, p1 = min(total, p0 + a.tile);
#pragma unroll 1
    for (int k = 0; k < 2; ++k) {   // an id of more than a tile's tokens is the tile's first or its last
        const int id = a.ids[k == 0 ? p0 : p1 - 1];
        const int b = a.offsets[id], e = a.offsets[id + 1];
        TIM_DCHECK(static_cast<unsigned>(id) < static_cast<unsigned>(a.V) && b >= 0 && b < e && e <= total, a.status, TIM_CHECK_UNIT,
                   tile, id);
        if (e - b <= a.many || (b >= p0) != (k == 1))
            continue;
        float acc[EM_PIECES][8] = {};
        sum_positions<T, VEC>(acc, a, max(p0, b), min(p1, e), col0);
        put_row<VEC>(a.partial + (static_cast<size_t>(tile) * 2 + k) * a.D, acc, col0, a.D, 1.f, false);
    }
}

// Rows that have tokens, EM_COLS columns a warp: unit (EM_FIRST positions, columns); the
// warp takes the ids whose first sorted position is among them.  32768 x 4096 bf16: 140 us, 0.52 GB
// (rows of 1 KB a warp in the tokens' order, four in flight: 46 % of DRAM's nominal peak).
constexpr int EM_FIRST = 8;

template <typename T, bool VEC> __global__ void __launch_bounds__(256, 2) embedding_rows_kernel(const EmbeddingArgs a, int column_blocks)
{
    const int64_t unit = static_cast<int64_t>(blockIdx.x) * 8 + (threadIdx.x >> 5);
    const int u0 = static_cast<int>(unit / column_blocks) * EM_FIRST, col0 = static_cast<int>(unit % column_blocks) * EM_COLS;
    const int lane = threadIdx.x & 31;
    pdl_wait();
    pdl_launch_dependents();
    const int total = a.offsets[a.V];
    if (u0 >= total)
        return;
    int my_id = 0, my_b = -1, my_e = 0;
    if (lane < EM_FIRST && u0 + lane < total) {
        my_id = a.ids[u0 + lane];
        my_b = a.offsets[my_id];
        my_e = a.offsets[my_id + 1];
        TIM_DCHECK(static_cast<unsigned>(my_id) < static_cast<unsigned>(a.V) && my_b <= u0 + lane && u0 + lane < my_e && my_e <= total,
                   a.status, TIM_CHECK_STORE, u0 + lane, my_id);
    }
    for (unsigned first = __ballot_sync(0xffffffffu, my_b == u0 + lane); first; first &= first - 1) {
        const int from = __ffs(first) - 1;
        const int id = __shfl_sync(0xffffffffu, my_id, from);
        const int b = u0 + from, e = __shfl_sync(0xffffffffu, my_e, from);
        float acc[EM_PIECES][8] = {};
        if (e - b > a.many) {
            // the first tile's partial is in slot 1 (the id begins in it), the others' in slot 0
            const int t1 = (e + a.tile - 1) / a.tile;
            for (int t = b / a.tile; t < t1; t += EM_AHEAD) {
                Pieces<float, VEC> r[EM_AHEAD];
#pragma unroll
                for (int i = 0; i < EM_AHEAD; ++i)
                    if (t + i < t1)
                        r[i].load(a.partial + (static_cast<size_t>(t + i) * 2 + ((t + i) * a.tile <= b)) * a.D, col0, a.D);
#pragma unroll
                for (int i = 0; i < EM_AHEAD; ++i)
                    if (t + i < t1)
                        r[i].add_to(acc);
            }
        } else {
            sum_positions<T, VEC>(acc, a, b, e, col0);
        }
        put_row<VEC>(a.dW + static_cast<size_t>(id) * a.D, acc, col0, a.D, a.scale, a.accumulate);
    }
}

template <typename F, typename... Rest>
cudaError_t launch(F kernel, int64_t ctas, int threads, int smem, cudaStream_t s, const EmbeddingArgs &a, Rest... rest)
{
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1] = {pdl_attribute()};
    cfg.gridDim = dim3(static_cast<unsigned>(ctas), 1, 1);
    cfg.blockDim = dim3(threads, 1, 1);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, a, rest...);
}

template <typename TW, typename TO> cudaError_t lookup(const EmbeddingArgs &a, cudaStream_t s)
{
    const int64_t units = static_cast<int64_t>(a.N) * ((a.D + 255) / 256);
    if (units <= 4096)   // few tokens: one piece a warp
        return launch(embedding_kernel<TW, TO, 1>, (units + 7) / 8, 256, 0, s, a);
    return launch(embedding_kernel<TW, TO, 4>, (units + 31) / 32, 256, 0, s, a);
}

template <typename TW> cudaError_t lookup_to(const EmbeddingArgs &a, int out_dtype, cudaStream_t s)
{
    if (out_dtype == TIM_F32)
        return lookup<TW, float>(a, s);
    if (out_dtype == TIM_BF16)
        return lookup<TW, __nv_bfloat16>(a, s);
    return lookup<TW, __half>(a, s);
}

template <typename T, bool VEC> cudaError_t sum(const EmbeddingArgs &a, cudaStream_t s)
{
    const int blocks = (a.D + EM_COLS - 1) / EM_COLS;
    const int64_t tiles = a.N > a.many ? (a.N + a.tile - 1) / a.tile : 0;
    const int64_t tile_ctas = (tiles * blocks + 7) / 8;
    const int64_t zero_ctas = a.accumulate ? 0 : (a.V + 8 * EM_IDS - 1) / (8 * EM_IDS);
    if (tile_ctas + zero_ctas > 0) {
        const cudaError_t e = launch(embedding_tiles_kernel<T, VEC>, tile_ctas + zero_ctas, 256, 0, s, a,
                                     static_cast<int>(tile_ctas), blocks);
        if (e != cudaSuccess)
            return e;
    }
    return launch(embedding_rows_kernel<T, VEC>, (static_cast<int64_t>((a.N + EM_FIRST - 1) / EM_FIRST) * blocks + 7) / 8, 256, 0,
                  s, a, blocks);
}

template <typename T> cudaError_t sum(const EmbeddingArgs &a, cudaStream_t s)
{
    const bool vec = a.D % 8 == 0 && (reinterpret_cast<uintptr_t>(a.x) & 15) == 0 && (reinterpret_cast<uintptr_t>(a.dW) & 15) == 0;
    return vec ? sum<T, true>(a, s) : sum<T, false>(a, s);
}

} // namespace

cudaError_t embedding_launch(const EmbeddingArgs &a, int dtype, int out_dtype, cudaStream_t s)
{
    if (dtype == TIM_F32)
        return lookup_to<float>(a, out_dtype, s);
    if (dtype == TIM_BF16)
        return lookup_to<__nv_bfloat16>(a, out_dtype, s);
    return lookup_to<__half>(a, out_dtype, s);
}

constexpr int SORT_SMEM = EM_SORT_THREADS / 32 * EM_RANGE * static_cast<int>(sizeof(int));

cudaError_t embedding_prepare_device()
{
    return cudaFuncSetAttribute(embedding_sort_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, SORT_SMEM);
}

cudaError_t embedding_sort_launch(const EmbeddingArgs &a, cudaStream_t s)
{
    return launch(embedding_sort_kernel, (a.V + EM_RANGE - 1) / EM_RANGE, EM_SORT_THREADS, SORT_SMEM, s, a);
}

cudaError_t embedding_sum_launch(const EmbeddingArgs &a, int dtype, cudaStream_t s)
{
    if (dtype == TIM_F32)
        return sum<float>(a, s);
    if (dtype == TIM_BF16)
        return sum<__nv_bfloat16>(a, s);
    return sum<__half>(a, s);
}

} // namespace tim
