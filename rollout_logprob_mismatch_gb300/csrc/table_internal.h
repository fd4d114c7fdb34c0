// table_internal.h -- launch shapes and arguments of the operators beside the
// head's table: low-rank adapters on its logits, embedding lookup and gradient.
// Not part of the ABI.
#pragma once

#include <cstdint>

#include <cuda.h>
#include <cuda_runtime.h>

#include "../../include/tim.h"

namespace tim {

// Device memory from the library's stream-ordered pool; a tim_status code.
int workspace_alloc(void **p, size_t bytes, cudaStream_t s);
cudaError_t workspace_free(void *p, cudaStream_t s);

// Tensor map of bf16 elements: dims and box innermost first, strides in bytes of the
// outer dims, swizzle span in bytes; out-of-range elements read as zero.  A tim_status code.
int encode_bf16_map(CUtensorMap *m, const void *base, int rank, const uint64_t *dims, const uint64_t *strides,
                    const uint32_t *box, int span);

inline size_t ws_round(size_t x) { return (x + 255) / 256 * 256; }

// ---------------------------------------------------------------- adapters
constexpr int AD_MAX_RANK = 128;
constexpr int AD_MAX_ADAPTERS = 65535;
// Rows up to which they are ordered and projected in one launch, and the map's CTAs have few
// tiles and more factors.  128256 x 4096 bf16 of rank 16: 64 rows of 32 adapters 54 us, 89 with the
// other form of both, 256 rows of 128 145 (181).  Above it the one launch would still win at 512
// and 1000 rows (of 128 adapters 180 us for 201, 233 for 248), and the map's form for few rows wins or
// loses with the adapters a tile meets (1000 rows, rank 32 of 64: 281 for 312; rank 16 of 4: 136 for 128).
constexpr int AD_FEW_ROWS = 256;
constexpr int AD_MAP_THREADS = 288;  // eight warps of products, one of copies
constexpr int AD_MAP_ROWS = 256;     // positions of a CTA of the map, at most
constexpr int AD_MAP_SMEM = 224 * 1024;   // beside the lists of its rows

// Ranks are padded to 16, 32, 64 or 128 inside the kernels (zeros).
inline int ad_rank_pad(int64_t R) { return R <= 16 ? 16 : R <= 32 ? 32 : R <= 64 ? 64 : 128; }

// The batch's rows ordered by adapter (stable), and t = scale A h of each in bf16
// parts: t = part 0 + part 1 (+ part 2), each the rest rounded to nearest.
struct AdapterPlan {
    int32_t *offsets;   // [n + 2]: positions of adapter a are offsets[a] .. offsets[a + 1]; n = no adapter
    int32_t *perm;      // [N]: row of each position
    int32_t *adapter;   // [N]: adapter of each position, n = none
    uint16_t *t;        // bf16 [N + t_pad n][t_pitch]: [parts][RP] and padding; position p of adapter a in row p + t_pad a
    int32_t t_pitch;
    int32_t t_pad;      // 0, or AG_PAD: the rows behind an adapter's last, up to a multiple of 16 of them in all, are zeros
};

struct AdapterArgs {
    const uint16_t *h;        // [N, D] bf16
    const uint16_t *A;        // [n, R, D]
    const uint16_t *B;        // [n, V, R]
    const float *scale;       // [n] or null
    const int32_t *rows;      // [N]
    int32_t N, V, D, R, n;
    AdapterPlan plan;
    const void *z;            // [N, V], rows ld apart
    int64_t ld;
    void *out;
    int64_t ldo;
    int32_t in_place;
    int32_t row_chunk;        // map: positions of a CTA, a multiple of 16
    int32_t stages, factors;  // map: tiles and factors that a CTA has room for
    uint64_t wait_budget_ns;
    int *status;
};

// Orders the rows and projects them.  parts: 2 or 3.
cudaError_t adapters_shrink_launch(const AdapterArgs &a, int parts, int num_sms, cudaStream_t s);
// out = z + t B^T
cudaError_t adapters_expand_launch(AdapterArgs a, int dtype, int num_sms, cudaStream_t s);
cudaError_t adapters_prepare_device();   // shared-memory sizes

// The gradient: slabs of the vocabulary, tiles of 128 columns and 128 rows of bf16, or of
// 64 rows in two planes of bf16 parts (fp16), 32 rows in three (fp32).
constexpr int AG_BLOCK = 128;
constexpr int ag_planes(int dtype) { return dtype == TIM_BF16 ? 1 : dtype == TIM_F16 ? 2 : 3; }
constexpr int ag_step(int dtype) { return 128 >> (ag_planes(dtype) - 1); }   // rows of a tile
constexpr int AG_PAD = 16;           // t has room for so many rows of zeros behind each adapter's
constexpr int AG_SMEM = 227 * 1024;
constexpr int64_t AG_PARTIAL_BYTES = int64_t(1) << 30;   // du's partial sums at most, per part of the batch

// Tiles of a slab: as many as dB's sums have TMEM for, beside two of du (512 columns).
constexpr int ag_blocks(int RP) { return RP == 16 ? 8 : RP == 32 ? 7 : 4; }

// Products that go to one sum of dB in TMEM at most.  The tensor cores cut, rather than
// round, what they add up, so a sum loses in proportion to its length (1.8e-8 of dB's norm a
// product); after these many it is added in fp32 to what is in memory.  Errors of dB at 8200
// rows an adapter and more: 5.0e-7 with 32, 7.5e-7 to 1.0e-6 with 48
// (rank 64 of 4096 x 128256 bf16 618 us, 688 with 32), 1.0e-6 with 64.
constexpr int AG_CHAIN = 48;

// Products of 16 rows of dy with all parts of t (part p of one with part j of the other where p + j < 3).
constexpr int ag_products(int planes) { return planes == 1 ? 3 : planes == 2 ? 5 : 6; }

struct AdapterGradArgs {
    const uint16_t *h, *A, *B;
    const float *scale;
    AdapterPlan plan;
    const void *dy;           // [N, V], rows ld apart
    int64_t ld;
    int32_t N, V, D, R, n;
    int32_t RT;               // the rank padded (16, 32, 64, 128)
    int32_t aligned;          // every row of dy starts on 16 bytes
    int32_t cols, slabs;      // columns of a slab, slabs
    int32_t merged;           // t's first two parts are one operand
    int32_t chains, low;      // sums of dB in TMEM that take steps of rows in turn; one more for the low products, or 0
    int32_t link;             // rows of an adapter that go to them before they are written
    int32_t du_parts;         // parts of a sum of du: slabs times planes
    int32_t row_part;         // positions of a launch
    int32_t p0, p1, r0;       // the launch's positions and first rank
    int32_t row_chunk;        // dh: positions of a CTA
    float *partial;           // [du_parts][min(RT, 64) / 4][p1 - p0 + 16][4]
    uint16_t *du;             // [N][3][RT] bf16 parts of scale B^T dy
    float *dh, *dA, *dB;
    int32_t accumulate, accumulate_dh;
    uint64_t wait_budget_ns;
    int *status;
};

// maps: B, t
cudaError_t adapters_grad_launch(const CUtensorMap (&maps)[2], AdapterGradArgs a, int dtype, int num_sms, cudaStream_t s);
cudaError_t adapters_grad_prepare_device();

// ---------------------------------------------------------------- embedding
constexpr int EM_RANGE = 512;        // ids that one CTA of the sort orders
constexpr int EM_SORT_THREADS = 1024;
constexpr int EM_TILE = 32;          // sorted positions of a partial sum of a long row, at least
constexpr int EM_LONG = 64;          // tokens of an id above which its row is summed in tiles, at least
constexpr int EM_IDS = 4;            // rows of the table that a warp looks at for zeros

struct EmbeddingArgs {
    const int32_t *tokens;    // [N]
    int32_t N, V, D;
    float scale;
    const void *x;            // lookup: the table [V, D]; gradient: the rows' [N, D]
    void *out;                // lookup: [N, D]
    float *dW;                // gradient: [V, D]
    int32_t accumulate;
    int32_t *offsets;         // [V + 1] sorted positions of each id
    int32_t *order;           // [N] tokens ordered by id (stable)
    int32_t *ids;             // [N] id of each sorted position
    int2 *staged;             // [N] scratch of the sort
    int32_t tile, many;       // positions of a tile; tokens of an id above which it is summed in tiles (>= tile)
    float *partial;           // [ceil(N / tile)][2][D]
    int *status;
};

cudaError_t embedding_launch(const EmbeddingArgs &a, int dtype, int out_dtype, cudaStream_t s);
cudaError_t embedding_prepare_device();   // shared-memory size of the sort
cudaError_t embedding_sort_launch(const EmbeddingArgs &a, cudaStream_t s);
cudaError_t embedding_sum_launch(const EmbeddingArgs &a, int dtype, cudaStream_t s);

} // namespace tim
