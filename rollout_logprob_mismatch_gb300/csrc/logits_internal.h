// logits_internal.h -- launch shapes and arguments of the operators on a head's
// logits (processing, processed log-probability, distillation).  Not part of
// the ABI.
#pragma once

#include <cstdint>

#include <cuda_runtime.h>

namespace tim {

// A row of logits is cut into slices of 1024 columns.  One warp reduces a
// slice, lane by lane in column order, and the slices' partials are folded in
// slice order; nothing else enters a row's sums, so a row has the same bits
// whatever the batch and however many CTAs share it.
constexpr int LG_SLICE = 1024;
constexpr int64_t LG_MAX_V = int64_t(1) << 20;
constexpr int LG_MAX_SLICES = static_cast<int>(LG_MAX_V / LG_SLICE);
constexpr int LG_CLUSTER = 8;                      // CTAs that share a row, at most

inline int lg_slices(int64_t V) { return static_cast<int>((V + LG_SLICE - 1) / LG_SLICE); }

// ---------------------------------------------------------------- processing
constexpr int LP_MAP_THREADS = 256, LP_MAP_CTAS = 6;     // WRITE, GRAD; CTAs of an SM the registers are held to
constexpr int LP_SHORT = 12, LP_LONG = 4096;       // slices up to which, a row's tokens above which all of them build the table
constexpr int LP_WARPS = 8;                        // warps of a CTA at most
constexpr int LP_MAP_SLICES = 64;                  // slices of a segment at most
constexpr int LP_MAP_CAP = 3008, LP_LOGP_CAP = 1536;     // touched columns a table holds (at least LG_SLICE; 3072 measures as 3008)
constexpr int LP_HEAVY = 1536, LP_HEAVY_CAP = 5120;      // tokens of history a row, on average; the table then
constexpr int LP_TABLE = 1 << 18;                  // columns a table covers
static_assert(LP_MAP_SLICES * LG_SLICE <= 65536, "a segment's columns are counted in 16 bits");

enum { LP_WRITE = 0, LP_LOGP = 1, LP_GRAD = 2 };

struct ProcArgs {
    const void *z;             // [N, V], rows ld apart
    int64_t ld;
    int32_t N, V;
    const float *temperature, *repetition, *presence, *frequency;   // [N] or null
    const int32_t *history;    // token ids, history_len of them
    const int32_t *spans;      // [N][3]: begin, first generated token, end
    int32_t history_len;
    const int32_t *bias_offsets, *bias_ids;
    const float *bias_values;
    int32_t num_bias;
    const uint32_t *allowed;   // [num_allowed][allowed_ld] bits
    const int32_t *allowed_rows;
    int64_t allowed_ld;
    int32_t num_allowed;
    const int32_t *targets;    // LOGP, GRAD
    const float *grad, *lse;   // GRAD
    void *out;                 // WRITE: processed logits; GRAD: gradient
    int64_t ldo;
    int32_t in_place;          // out is z
    float *out_logp, *out_lse; // LOGP
    int32_t seg_slices;        // WRITE, GRAD: slices of a CTA; LOGP: of a cluster rank
    int32_t segs;              // CTAs of a row
    int32_t table_columns;     // columns the shared-memory table has room for
    int32_t table_cap;         // touched ones among them
    int *status;
};

// dtype and out_dtype: TIM_F32 / TIM_BF16 / TIM_F16
cudaError_t logits_process_launch(ProcArgs a, int op, int dtype, int out_dtype, int num_sms, cudaStream_t s);

// ---------------------------------------------------------------- distillation
constexpr int LD_THREADS = 256;
constexpr int LD_FEW = 12;                         // slices of a CTA up to which half the threads run
constexpr int LD_MAX_K = 1024;
constexpr int LD_SMEM = 224 * 1024;                // shared memory a CTA may take

enum { LD_FORWARD = 0, LD_BACKWARD = 1, LD_STEP = 2 };

struct DistillArgs {
    const void *z;
    int64_t ld;
    int32_t N, V, K;
    const int32_t *ids;        // [N, K]
    const float *teacher;      // [N, K]
    const float *teacher_lse;  // [N] or null: renormalised over the K
    float temperature;
    const float *grad;         // [N]: BACKWARD, STEP
    const float *lse, *lse_tail;              // BACKWARD
    float *loss, *out_lse, *out_lse_tail;     // FORWARD, STEP
    void *dz;                  // BACKWARD, STEP
    int64_t ldo;
    int32_t per;               // slices of a cluster rank
    int32_t ranks;             // CTAs of a row
    uint64_t wait_budget_ns;   // STEP: wait for the row's copy
    int *status;
};

cudaError_t distill_topk_launch(DistillArgs a, int op, int dtype, int num_sms, cudaStream_t s);

// shared-memory sizes of the kernels above
cudaError_t logits_process_prepare_device();
cudaError_t distill_topk_prepare_device();

} // namespace tim
