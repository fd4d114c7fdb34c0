// adapters.cu -- low-rank adapters of many requests beside the shared head (sm_103a).
//
// y_n = z_n + s_a B_a (A_a h_n), a = the adapter of row n: z are the shared head's
// logits, A_a [R, D] and B_a [V, R] the adapter's factors.  Two launches:
//   shrink  orders the rows by adapter (a CTA counts the ids below its own and takes
//           its own in order: no counter to clear, no atomics, the same order every
//           time) and writes t_n = s_a A_a h_n in bf16 parts;
//   map     y = z + t B^T, one pass over the logits.
// A row's products are formed with its own adapter's factors only: where a tile of 16
// rows meets several adapters, the tile is multiplied with each and every row keeps its
// own (masking t to zero instead would let an infinite or NaN factor of one tenant
// reach another's rows).
#include <algorithm>

#include "adapters.cuh"
#include "table_internal.h"

namespace tim {
namespace {

// ---------------------------------------------------------------- shrink
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

// CTA (a, c): the rows of adapter a, chunks c, c + gridDim.y, ... of a.chunk of them.
// a = n: the rows under no adapter (only ordered).  The 16 warps take a chunk's tiles of
// 16 rows and share k among those of a tile, then add up through shared memory in order.
template <int RP, int PARTS>
__global__ void __launch_bounds__(AD_SHRINK_THREADS) adapters_shrink_kernel(const AdapterArgs a)
{
    constexpr int WARPS = AD_SHRINK_THREADS / 32;
    constexpr int NC = RP < 32 ? RP : 32;      // rank columns at a time
    constexpr int AHEAD = 4;                   // steps of 32 k whose loads are in flight together
    __shared__ int32_t mine[AD_CHUNK];
    __shared__ float sums[WARPS][16][NC + 1];
    __shared__ int sb[WARPS], so[WARPS];
    const int ad = blockIdx.x, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int g = lane >> 2, q = lane & 3;
    pdl_wait();
    pdl_launch_dependents();

    // each warp has a part of the list, in order
    const int per = ((a.N + 31) / 32 + WARPS - 1) / WARPS * 32;
    const int r0 = min(a.N, warp * per), r1 = min(a.N, r0 + per);
    int below = 0, own = 0;
#pragma unroll 8
    for (int r = r0 + lane; r < r1; r += 32) {
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
    int base = 0, count = 0, before = 0;
#pragma unroll
    for (int w = 0; w < WARPS; ++w) {
        base += sb[w];
        count += so[w];
        before += w < warp ? so[w] : 0;
    }
    if (blockIdx.y == 0) {
        if (tid == 0) {
            a.plan.offsets[ad] = base;
            if (ad == a.n)
                a.plan.offsets[ad + 1] = a.N;
        }
        if (own > 0)
            own_rows(a, ad, r0, r1, base + before, [&](int r, int p) {
                a.plan.perm[p] = r;
                a.plan.adapter[p] = ad;
            });
    }
    if (ad == a.n)
        return;
    const float scale = a.scale ? a.scale[ad] : 1.f;
    const uint16_t *A = a.A + static_cast<size_t>(ad) * a.R * a.D;
    const int kchunks = (a.D + 31) / 32;
    const uint4 zero = make_uint4(0u, 0u, 0u, 0u);

    for (int c = blockIdx.y; c * a.chunk < count; c += gridDim.y) {
        const int c0 = c * a.chunk, rows = min(a.chunk, count - c0);
        __syncthreads();   // the chunk before has been read
        if (own > 0 && before < c0 + rows && before + own > c0)
            own_rows(a, ad, r0, r1, before, [&](int r, int p) {
                if (p >= c0 && p < c0 + rows)
                    mine[p - c0] = r;
            });
        __syncthreads();
        const int tiles = a.chunk / 16;             // 1, 2 or 4
        const int m0 = (warp % tiles) * 16, kw = warp / tiles, ks = WARPS / tiles;
        const bool on0 = m0 + g < rows, on1 = m0 + g + 8 < rows;
        const uint16_t *h0 = a.h + static_cast<size_t>(on0 ? mine[m0 + g] : 0) * a.D;
        const uint16_t *h1 = a.h + static_cast<size_t>(on1 ? mine[m0 + g + 8] : 0) * a.D;
        for (int n0 = 0; n0 < RP; n0 += NC) {
            float acc[NC / 8][4] = {};
            if (m0 < rows && n0 < a.R) {
                for (int kc0 = kw; kc0 < kchunks; kc0 += ks * AHEAD) {
                    uint4 x0[AHEAD], x1[AHEAD], w[AHEAD][NC / 8];
#pragma unroll
                    for (int i = 0; i < AHEAD; ++i) {
                        const int k = (kc0 + i * ks) * 32 + q * 8;   // D is a multiple of 8: the eight are in or out together
                        const bool on = k < a.D;
                        x0[i] = on && on0 ? __ldg(reinterpret_cast<const uint4 *>(h0 + k)) : zero;
                        x1[i] = on && on1 ? __ldg(reinterpret_cast<const uint4 *>(h1 + k)) : zero;
#pragma unroll
                        for (int j = 0; j < NC / 8; ++j) {
                            const int r = n0 + j * 8 + g;
                            w[i][j] = on && r < a.R
                                          ? __ldg(reinterpret_cast<const uint4 *>(A + static_cast<size_t>(r) * a.D + k))
                                          : zero;
                        }
                    }
#pragma unroll
                    for (int i = 0; i < AHEAD; ++i)
#pragma unroll
                        for (int j = 0; j < NC / 8; ++j) {
                            mma16816(acc[j], {x0[i].x, x1[i].x, x0[i].y, x1[i].y}, w[i][j].x, w[i][j].y);
                            mma16816(acc[j], {x0[i].z, x1[i].z, x0[i].w, x1[i].w}, w[i][j].z, w[i][j].w);
                        }
                }
            }
            if (n0 > 0)
                __syncthreads();   // the ranks before have been added up
#pragma unroll
            for (int j = 0; j < NC / 8; ++j) {
                sums[warp][g][j * 8 + 2 * q] = acc[j][0];
                sums[warp][g][j * 8 + 2 * q + 1] = acc[j][1];
                sums[warp][g + 8][j * 8 + 2 * q] = acc[j][2];
                sums[warp][g + 8][j * 8 + 2 * q + 1] = acc[j][3];
            }
            __syncthreads();
            for (int i = tid; i < rows * NC; i += AD_SHRINK_THREADS) {
                const int m = i / NC, r = i % NC;
                float u = 0.f;
                for (int w = m / 16; w < WARPS; w += tiles)
                    u += sums[w][m % 16][r];
                uint16_t p[PARTS];
                split_bf16<PARTS>(u * scale, p);
                uint16_t *t = a.plan.t + (static_cast<size_t>(base) + c0 + m) * a.plan.t_pitch + n0 + r;
#pragma unroll
                for (int k = 0; k < PARTS; ++k)
                    t[k * RP] = p[k];
            }
        }
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
    static constexpr int STEPS = RP / 16;                // products along the rank
};

template <int WORDS> __device__ __forceinline__ void load_words(uint32_t *w, const uint16_t *p, bool on)
{
    if constexpr (WORDS == 2) {
        const uint2 v = on ? __ldg(reinterpret_cast<const uint2 *>(p)) : make_uint2(0u, 0u);
        w[0] = v.x;
        w[1] = v.y;
    } else {
        const uint4 v = on ? __ldg(reinterpret_cast<const uint4 *>(p)) : make_uint4(0u, 0u, 0u, 0u);
        w[0] = v.x;
        w[1] = v.y;
        w[2] = v.z;
        w[3] = v.w;
    }
}

// A warp's CB blocks of 32 columns: product j (of four) of a block has as its column n
// the logits' column 8 (n / 2) + 2 j + n % 2, so that lane q's eight results are eight
// neighbours.
template <int RP, int CB> struct Factor {
    uint32_t w[CB][4][Ranks<RP>::GROUPS][Ranks<RP>::WORDS];
    __device__ __forceinline__ void load(const uint16_t *B, int v0, int V, int R)
    {
        using K = Ranks<RP>;
        const int lane = threadIdx.x & 31, g = lane >> 2, q = lane & 3;
#pragma unroll
        for (int c = 0; c < CB; ++c)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int v = v0 + c * 32 + 8 * (g >> 1) + 2 * j + (g & 1);
                const uint16_t *row = B + static_cast<size_t>(min(v, V - 1)) * R;
#pragma unroll
                for (int k = 0; k < K::GROUPS; ++k) {
                    const int r = k * 32 + q * K::STEP;
                    load_words<K::WORDS>(w[c][j][k], row + (r < R ? r : 0), v < V && r < R);
                }
            }
    }
};

// A CTA: row_chunk positions, 256 CB columns, eight warps of 32 CB columns (the CTAs
// side by side in the grid share their rows).  A tile is 16 positions; the next tile's logits are in flight while a tile is
// multiplied, and an adapter's factor stays in registers while the adapter is the same.
template <typename T, int RP, int PARTS, int CB, bool AL>
__global__ void __launch_bounds__(AD_MAP_THREADS) adapters_map_kernel(const AdapterArgs a)
{
    using K = Ranks<RP>;
    __shared__ int32_t s_row[AD_MAP_ROWS], s_ad[AD_MAP_ROWS + 1];
    const int lane = threadIdx.x & 31, g = lane >> 2, q = lane & 3;
    const int slabs = (a.V + 256 * CB - 1) / (256 * CB);
    const int v0 = (blockIdx.x % slabs * 8 + (threadIdx.x >> 5)) * 32 * CB;
    const int p0 = blockIdx.x / slabs * a.row_chunk;
    pdl_wait();
    pdl_launch_dependents();
    const int live = a.in_place ? a.plan.offsets[a.n] : a.N;   // rows under no adapter come last
    const int rows = min(live - p0, a.row_chunk);
    if (rows <= 0)
        return;
    for (int i = threadIdx.x; i < rows; i += AD_MAP_THREADS) {
        s_row[i] = a.plan.perm[p0 + i];
        s_ad[i] = a.plan.adapter[p0 + i];
    }
    if (threadIdx.x == 0)
        s_ad[rows] = -1;
    __syncthreads();
    if (v0 >= a.V)
        return;
    const T *z = static_cast<const T *>(a.z);
    T *out = static_cast<T *>(a.out);

    auto load = [&](Raw8<T> (&x)[2][CB], int p) {
#pragma unroll
        for (int half = 0; half < 2; ++half) {
            const int i = p + g + half * 8;
            if (i < rows) {
                const T *row = z + static_cast<size_t>(s_row[i]) * a.ld;
#pragma unroll
                for (int c = 0; c < CB; ++c) {
                    const int col = v0 + c * 32 + q * 8;
                    if (col < a.V)
                        load8<T>(x[half][c], row, col, a.V, AL ? 0u : row_shift(row));
                }
            }
        }
    };
    int ad = s_ad[0];
    Factor<RP, CB> f;
    if (ad < a.n)
        f.load(a.B + static_cast<size_t>(ad) * a.V * a.R, v0, a.V, a.R);
    Raw8<T> x[2][CB];
    load(x, 0);
    for (int p = 0; p < rows; p += 16) {
        Raw8<T> y[2][CB];
#pragma unroll
        for (int c = 0; c < CB; ++c) {
            y[0][c] = x[0][c];
            y[1][c] = x[1][c];
        }
        if (p + 16 < rows)
            load(x, p + 16);
        const int e = min(p + 16, rows);
        const bool on0 = p + g < e, on1 = p + g + 8 < e;
        uint32_t t[PARTS][K::GROUPS][2][K::WORDS];   // rows g and g + 8 of t
        const uint16_t *t0 = a.plan.t + static_cast<size_t>(p0 + p + g) * (PARTS * RP);
        const bool has0 = on0 && s_ad[p + g] < a.n, has1 = on1 && s_ad[p + g + 8] < a.n;
#pragma unroll
        for (int i = 0; i < PARTS; ++i)
#pragma unroll
            for (int k = 0; k < K::GROUPS; ++k) {
                const int r = i * RP + k * 32 + q * K::STEP;
                load_words<K::WORDS>(t[i][k][0], t0 + r, has0);
                load_words<K::WORDS>(t[i][k][1], t0 + 8 * (PARTS * RP) + r, has1);
            }
        float keep[CB][4][4] = {};
        for (int s = p; s < e;) {
            // the positions of this tile under the adapter at hand: s .. m - 1
            int m = e;
            if (s_ad[e - 1] != ad)
                for (m = s + 1; s_ad[m] == ad;)
                    ++m;
            if (ad < a.n) {
                float acc[CB][4][4] = {};
#pragma unroll
                for (int i = 0; i < PARTS; ++i)
#pragma unroll
                    for (int k = 0; k < K::STEPS; ++k) {
                        const int grp = RP == 16 ? 0 : k / 2, w = RP == 16 ? 0 : (k % 2) * 2;
#pragma unroll
                        for (int c = 0; c < CB; ++c)
#pragma unroll
                            for (int j = 0; j < 4; ++j)
                                mma16816(acc[c][j],
                                         {t[i][grp][0][w], t[i][grp][1][w], t[i][grp][0][w + 1], t[i][grp][1][w + 1]},
                                         f.w[c][j][grp][w], f.w[c][j][grp][w + 1]);
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
            if (s_ad[m] >= 0 && s_ad[m] != ad) {   // (-1 behind the last position)
                ad = s_ad[m];
                if (ad < a.n)
                    f.load(a.B + static_cast<size_t>(ad) * a.V * a.R, v0, a.V, a.R);
            }
        }
#pragma unroll
        for (int half = 0; half < 2; ++half) {
            const bool on = half ? on1 : on0, has = half ? has1 : has0;
            T *row = out + static_cast<size_t>(on ? s_row[p + g + half * 8] : 0) * a.ldo;
            const bool any = !AL && __any_sync(0xffffffffu, row_shift(row) != 0);
#pragma unroll
            for (int c = 0; c < CB; ++c) {
                float v[8];
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    v[i] = Elem<T>::get(y[half][c].w, i) + keep[c][i >> 1][2 * half + (i & 1)];
                Raw8<T> w = pack8<T>(v);
                if (!has)
                    w = y[half][c];   // a row under no adapter keeps its bits
                const int col = v0 + c * 32 + q * 8;
                store_quad<T>(row, col, a.V, w, on && col < a.V, any);
            }
        }
    }
}

template <typename F> cudaError_t launch(F kernel, dim3 grid, int threads, const AdapterArgs &a, cudaStream_t s)
{
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1] = {pdl_attribute()};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads, 1, 1);
    cfg.stream = s;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, a);
}

template <int PARTS> cudaError_t shrink(const AdapterArgs &a, dim3 grid, cudaStream_t s)
{
    switch (ad_rank_pad(a.R)) {
    case 16: return launch(adapters_shrink_kernel<16, PARTS>, grid, AD_SHRINK_THREADS, a, s);
    case 32: return launch(adapters_shrink_kernel<32, PARTS>, grid, AD_SHRINK_THREADS, a, s);
    case 64: return launch(adapters_shrink_kernel<64, PARTS>, grid, AD_SHRINK_THREADS, a, s);
    default: return launch(adapters_shrink_kernel<128, PARTS>, grid, AD_SHRINK_THREADS, a, s);
    }
}

// Column blocks of a warp: 128 bytes of a row where the factor's registers allow it.
template <typename T, int RP> constexpr int map_blocks() { return sizeof(T) == 2 && RP <= 32 ? 2 : 1; }

template <typename T, int PARTS, int RP> cudaError_t map(AdapterArgs a, int num_sms, cudaStream_t s)
{
    constexpr int CB = map_blocks<T, RP>();
    const int slabs = (a.V + 256 * CB - 1) / (256 * CB);
    // few rows: a tile a CTA, so that the adapters' factors come in parallel
    int64_t rows = AD_MAP_ROWS;
    while (rows > 16 && slabs * ((a.N + rows - 1) / rows) < int64_t(8) * num_sms)
        rows /= 2;
    a.row_chunk = static_cast<int32_t>(rows);
    const dim3 grid(static_cast<unsigned>(slabs * ((a.N + rows - 1) / rows)));
    auto aligned = [](const void *p, int64_t ld, int64_t N) {
        return (reinterpret_cast<uintptr_t>(p) & 15) == 0 && (N == 1 || ld * sizeof(T) % 16 == 0);
    };
    if (aligned(a.z, a.ld, a.N) && aligned(a.out, a.ldo, a.N))
        return launch(adapters_map_kernel<T, RP, PARTS, CB, true>, grid, AD_MAP_THREADS, a, s);
    return launch(adapters_map_kernel<T, RP, PARTS, CB, false>, grid, AD_MAP_THREADS, a, s);
}

template <typename T, int PARTS> cudaError_t map(const AdapterArgs &a, int num_sms, cudaStream_t s)
{
    switch (ad_rank_pad(a.R)) {
    case 16: return map<T, PARTS, 16>(a, num_sms, s);
    case 32: return map<T, PARTS, 32>(a, num_sms, s);
    case 64: return map<T, PARTS, 64>(a, num_sms, s);
    default: return map<T, PARTS, 128>(a, num_sms, s);
    }
}

} // namespace

cudaError_t adapters_shrink_launch(AdapterArgs a, int parts, int num_sms, cudaStream_t s)
{
    // a CTA of 16 rows at a time while that does not give every SM more than two
    a.chunk = 16;
    while (a.chunk < AD_CHUNK && a.N > 2 * num_sms * a.chunk)
        a.chunk *= 2;
    // about two CTAs an SM in all: each reads the whole list of ids
    const int chunks = (a.N + a.chunk - 1) / a.chunk;
    const int ys = std::max(1, std::min(chunks, (2 * num_sms + a.n) / (a.n + 1)));
    const dim3 grid(static_cast<unsigned>(a.n + 1), static_cast<unsigned>(ys), 1);
    return parts == 3 ? shrink<3>(a, grid, s) : shrink<2>(a, grid, s);
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
