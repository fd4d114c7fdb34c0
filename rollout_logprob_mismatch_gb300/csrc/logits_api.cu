// logits_api.cu -- the C entry points of the operators on a head's logits:
// argument checks and launches (no workspace: a row's CTAs meet in shared memory).
#include <cmath>

#include "../../include/tim.h"
#include "logits_internal.h"
#include "tim_internal.h"

namespace {

using tim::fail_message;

bool aligned(const void *p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

uintptr_t elem_bytes(int dtype) { return dtype == TIM_F32 ? 4 : 2; }

int invalid(const char *msg) { return fail_message(TIM_ERR_INVALID_ARG, "%s", msg); }

// Rows that reach past 2^56 elements are in no address space (and their extent in
// bytes might not fit 64 bits).
bool too_far(int64_t N, int64_t stride) { return N > 0 && stride > (int64_t(1) << 56) / N; }

// Checks the logits' sizes; 1 = nothing to do (N = 0).
int check_logits(const void *logits, int dtype, int64_t N, int64_t V, int64_t stride)
{
    if (dtype != TIM_F32 && dtype != TIM_BF16 && dtype != TIM_F16)
        return invalid("dtype must be TIM_F32, TIM_BF16 or TIM_F16");
    if (N < 0 || N >= (int64_t(1) << 31))
        return fail_message(TIM_ERR_INVALID_ARG, "N = %lld out of range [0, 2^31)", static_cast<long long>(N));
    if (V <= 0 || V > tim::LG_MAX_V)
        return fail_message(TIM_ERR_INVALID_ARG, "V = %lld out of range (0, %lld]", static_cast<long long>(V),
                            static_cast<long long>(tim::LG_MAX_V));
    if (stride < V || stride > (int64_t(1) << 40))
        return invalid("the rows' stride must be at least V");
    if (N * tim::lg_slices(V) >= (int64_t(1) << 31))
        return invalid("N x V too large for one call");
    if (too_far(N, stride))
        return invalid("the rows reach past the address space");
    if (N == 0)
        return 1;
    if (!logits)
        return invalid("logits is null");
    if (!aligned(logits, elem_bytes(dtype)))
        return invalid("logits must be aligned to its elements");
    return TIM_OK;
}

// Do N rows of `size` bytes each, `step` bytes apart, share a byte with rows of `size2`
// bytes, `step2` apart?  Exact for equal steps (two parts of one buffer's rows, side by
// side); else the whole ranges are compared.
bool share_bytes(uintptr_t a, uintptr_t step, uintptr_t size, uintptr_t b, uintptr_t step2, uintptr_t size2, int64_t N)
{
    const uintptr_t last = static_cast<uintptr_t>(N - 1);
    if (a + last * step + size <= b || b + last * step2 + size2 <= a)
        return false;
    if (N == 1 || step != step2)
        return true;
    const uintptr_t at = b >= a ? (b - a) % step : (step - (a - b) % step) % step;   // a row of b within a row of a
    return at < size || at + size2 > step;
}

// An output of the logits' shape: not null, aligned, and either apart from the
// logits or exactly over them.
int check_out(const void *logits, int dtype, int64_t N, int64_t V, int64_t stride, const void *out, int out_dtype,
              int64_t out_stride)
{
    if (!out)
        return invalid("the output is null");
    if (out_stride < V || out_stride > (int64_t(1) << 40))
        return invalid("the output rows' stride must be at least V");
    if (too_far(N, out_stride))
        return invalid("the output's rows reach past the address space");
    if (!aligned(out, elem_bytes(out_dtype)))
        return invalid("the output must be aligned to its elements");
    if (out == logits && out_dtype == dtype && (out_stride == stride || N == 1))
        return TIM_OK;
    const uintptr_t es = elem_bytes(dtype), eo = elem_bytes(out_dtype);
    if (share_bytes(reinterpret_cast<uintptr_t>(logits), stride * es, V * es, reinterpret_cast<uintptr_t>(out),
                    out_stride * eo, V * eo, N))
        return invalid("the output overlaps the logits without being the logits");
    return TIM_OK;
}

int set_rules(tim::ProcArgs &a, const tim_logits_rules *r, int64_t N, int64_t V)
{
    if (!r)
        return TIM_OK;
    if (r->num_history < 0 || r->num_bias < 0 || r->num_allowed < 0)
        return invalid("num_history, num_bias and num_allowed must be >= 0");
    if (r->num_history >= 1 << 30 || r->num_bias >= 1 << 30)
        return invalid("num_history and num_bias must be below 2^30");
    if (r->history_spans && r->num_history > 0 && !r->history)
        return invalid("history_spans without history");
    if (r->bias_offsets && r->num_bias > 0 && (!r->bias_ids || !r->bias_values))
        return invalid("bias_offsets without bias_ids and bias_values");
    if (r->allowed && r->allowed_stride < (V + 31) / 32)
        return invalid("allowed_stride must be at least ceil(V / 32) words");
    if (r->allowed && !r->allowed_rows && r->num_allowed < N)
        return invalid("allowed has fewer rows than the logits, and there is no allowed_rows");
    if (r->allowed_rows && !r->allowed)
        return invalid("allowed_rows without allowed");
    if (!aligned(r->temperature, 4) || !aligned(r->repetition, 4) || !aligned(r->presence, 4) ||
        !aligned(r->frequency, 4) || !aligned(r->history, 4) || !aligned(r->history_spans, 4) ||
        !aligned(r->bias_offsets, 4) || !aligned(r->bias_ids, 4) || !aligned(r->bias_values, 4) ||
        !aligned(r->allowed, 4) || !aligned(r->allowed_rows, 4))
        return invalid("the rules' arrays must be 4-byte aligned");
    a.temperature = r->temperature;
    a.repetition = r->repetition;
    a.presence = r->presence;
    a.frequency = r->frequency;
    a.history = r->history;
    a.spans = r->history_spans;
    a.history_len = r->num_history;
    a.bias_offsets = r->bias_offsets;
    a.bias_ids = r->bias_ids;
    a.bias_values = r->bias_values;
    a.num_bias = r->num_bias;
    a.allowed = r->allowed;
    a.allowed_rows = r->allowed_rows;
    a.allowed_ld = r->allowed_stride;
    a.num_allowed = r->num_allowed;
    return TIM_OK;
}

int finish(cudaError_t e, const char *what)
{
    if (e != cudaSuccess)
        return fail_message(TIM_ERR_CUDA, "%s: %s", what, cudaGetErrorString(e));
    return tim::record_error(TIM_OK, "");
}

int process(tim::ProcArgs a, int op, const void *logits, int dtype, int64_t N, int64_t V, int64_t stride,
            const tim_logits_rules *rules, int out_dtype, tim_stream_t stream)
{
    int rc = set_rules(a, rules, N, V);
    if (rc != TIM_OK)
        return rc;
    int sms = 0;
    if ((rc = tim::use_device(&a.status, &sms)) != TIM_OK)
        return rc;
    a.z = logits;
    a.ld = stride;
    a.N = static_cast<int32_t>(N);
    a.V = static_cast<int32_t>(V);
    a.in_place = a.out == logits;
    return finish(tim::logits_process_launch(a, op, dtype, out_dtype, sms, reinterpret_cast<cudaStream_t>(stream)),
                  "launch");
}

int distill(tim::DistillArgs a, int op, const void *logits, int dtype, int64_t N, int64_t V, int64_t stride,
            const int32_t *ids, const float *teacher, const float *teacher_lse, int64_t K, float temperature,
            tim_stream_t stream)
{
    if (!ids || !teacher)
        return invalid("teacher_ids and teacher_logits are required");
    if (!aligned(ids, 4) || !aligned(teacher, 4) || !aligned(teacher_lse, 4) || !aligned(a.grad, 4) ||
        !aligned(a.lse, 4) || !aligned(a.lse_tail, 4) || !aligned(a.loss, 4) || !aligned(a.out_lse, 4) ||
        !aligned(a.out_lse_tail, 4))
        return invalid("teacher and row arrays must be 4-byte aligned");
    int sms = 0;
    const int rc = tim::use_device(&a.status, &sms);
    if (rc != TIM_OK)
        return rc;
    a.z = logits;
    a.ld = stride;
    a.N = static_cast<int32_t>(N);
    a.V = static_cast<int32_t>(V);
    a.K = static_cast<int32_t>(K);
    a.ids = ids;
    a.teacher = teacher;
    a.teacher_lse = teacher_lse;
    a.temperature = temperature;
    a.wait_budget_ns = tim::pipeline_wait_budget_ns();
    return finish(tim::distill_topk_launch(a, op, dtype, sms, reinterpret_cast<cudaStream_t>(stream)), "launch");
}

// K and the temperature are checked for an empty batch too.
int check_distill(int64_t K, float temperature)
{
    if (K < 1 || K > TIM_DISTILL_MAX_K)
        return fail_message(TIM_ERR_INVALID_ARG, "K = %lld out of range [1, %d]", static_cast<long long>(K),
                            TIM_DISTILL_MAX_K);
    if (!(temperature > 0.f) || !std::isfinite(temperature) || !std::isfinite(1.f / temperature))
        return invalid("temperature must be positive and finite");
    return TIM_OK;
}

static_assert(TIM_DISTILL_MAX_K == tim::LD_MAX_K, "the header's limit");

} // namespace

extern "C" {

int tim_process_logits(const void *logits, int dtype, int64_t N, int64_t V, int64_t stride,
                       const tim_logits_rules *rules, void *out, int out_dtype, int64_t out_stride,
                       tim_stream_t stream)
{
    int rc = check_logits(logits, dtype, N, V, stride);
    if (rc < 0)
        return rc;
    if (out_dtype != dtype && out_dtype != TIM_F32)
        return invalid("out_dtype must be dtype or TIM_F32");
    if (rc == 1)
        return tim::record_error(TIM_OK, "");
    if ((rc = check_out(logits, dtype, N, V, stride, out, out_dtype, out_stride)) != TIM_OK)
        return rc;
    tim::ProcArgs a{};
    a.out = out;
    a.ldo = out_stride;
    return process(a, tim::LP_WRITE, logits, dtype, N, V, stride, rules, out_dtype, stream);
}

int tim_processed_logprob(const void *logits, int dtype, int64_t N, int64_t V, int64_t stride,
                          const tim_logits_rules *rules, const int32_t *targets, float *out_logp, float *out_lse,
                          tim_stream_t stream)
{
    const int rc = check_logits(logits, dtype, N, V, stride);
    if (rc < 0)
        return rc;
    if (rc == 1)
        return tim::record_error(TIM_OK, "");
    if (!targets || !out_logp || !out_lse)
        return invalid("null pointer argument");
    if (!aligned(targets, 4) || !aligned(out_logp, 4) || !aligned(out_lse, 4))
        return invalid("targets / outputs must be 4-byte aligned");
    tim::ProcArgs a{};
    a.targets = targets;
    a.out_logp = out_logp;
    a.out_lse = out_lse;
    return process(a, tim::LP_LOGP, logits, dtype, N, V, stride, rules, dtype, stream);
}

int tim_processed_logprob_backward(const void *logits, int dtype, int64_t N, int64_t V, int64_t stride,
                                   const tim_logits_rules *rules, const int32_t *targets, const float *grad_logp,
                                   const float *lse, void *dlogits, int64_t dlogits_stride, tim_stream_t stream)
{
    int rc = check_logits(logits, dtype, N, V, stride);
    if (rc < 0)
        return rc;
    if (rc == 1)
        return tim::record_error(TIM_OK, "");
    if (!targets || !grad_logp || !lse)
        return invalid("null pointer argument");
    if (!aligned(targets, 4) || !aligned(grad_logp, 4) || !aligned(lse, 4))
        return invalid("targets / grad_logp / lse must be 4-byte aligned");
    if ((rc = check_out(logits, dtype, N, V, stride, dlogits, dtype, dlogits_stride)) != TIM_OK)
        return rc;
    tim::ProcArgs a{};
    a.targets = targets;
    a.grad = grad_logp;
    a.lse = lse;
    a.out = dlogits;
    a.ldo = dlogits_stride;
    return process(a, tim::LP_GRAD, logits, dtype, N, V, stride, rules, dtype, stream);
}

int tim_distill_topk(const void *logits, int dtype, int64_t N, int64_t V, int64_t stride, const int32_t *teacher_ids,
                     const float *teacher_logits, const float *teacher_lse, int64_t K, float temperature,
                     float *loss, float *lse, float *lse_tail, tim_stream_t stream)
{
    const int rc = check_logits(logits, dtype, N, V, stride);
    if (rc < 0)
        return rc;
    if (check_distill(K, temperature) != TIM_OK)
        return TIM_ERR_INVALID_ARG;
    if (rc == 1)
        return tim::record_error(TIM_OK, "");
    if (!loss || !lse || (teacher_lse && !lse_tail))
        return invalid("loss, lse and (with teacher_lse) lse_tail are required");
    tim::DistillArgs a{};
    a.loss = loss;
    a.out_lse = lse;
    a.out_lse_tail = lse_tail;
    return distill(a, tim::LD_FORWARD, logits, dtype, N, V, stride, teacher_ids, teacher_logits, teacher_lse, K,
                   temperature, stream);
}

int tim_distill_topk_backward(const void *logits, int dtype, int64_t N, int64_t V, int64_t stride,
                              const int32_t *teacher_ids, const float *teacher_logits, const float *teacher_lse,
                              int64_t K, float temperature, const float *grad_loss, const float *lse,
                              const float *lse_tail, void *dlogits, int64_t dlogits_stride, tim_stream_t stream)
{
    int rc = check_logits(logits, dtype, N, V, stride);
    if (rc < 0)
        return rc;
    if (check_distill(K, temperature) != TIM_OK)
        return TIM_ERR_INVALID_ARG;
    if (rc == 1)
        return tim::record_error(TIM_OK, "");
    if (!grad_loss || !lse || (teacher_lse && !lse_tail))
        return invalid("grad_loss, lse and (with teacher_lse) lse_tail are required");
    if ((rc = check_out(logits, dtype, N, V, stride, dlogits, dtype, dlogits_stride)) != TIM_OK)
        return rc;
    tim::DistillArgs a{};
    a.grad = grad_loss;
    a.lse = lse;
    a.lse_tail = lse_tail;
    a.dz = dlogits;
    a.ldo = dlogits_stride;
    return distill(a, tim::LD_BACKWARD, logits, dtype, N, V, stride, teacher_ids, teacher_logits, teacher_lse, K,
                   temperature, stream);
}

int tim_distill_topk_step(const void *logits, int dtype, int64_t N, int64_t V, int64_t stride,
                          const int32_t *teacher_ids, const float *teacher_logits, const float *teacher_lse,
                          int64_t K, float temperature, const float *grad_loss, float *loss, float *lse,
                          float *lse_tail, void *dlogits, int64_t dlogits_stride, tim_stream_t stream)
{
    int rc = check_logits(logits, dtype, N, V, stride);
    if (rc < 0)
        return rc;
    if (check_distill(K, temperature) != TIM_OK)
        return TIM_ERR_INVALID_ARG;
    if (rc == 1)
        return tim::record_error(TIM_OK, "");
    if (!grad_loss || !loss || !lse || (teacher_lse && !lse_tail))
        return invalid("grad_loss, loss, lse and (with teacher_lse) lse_tail are required");
    if ((rc = check_out(logits, dtype, N, V, stride, dlogits, dtype, dlogits_stride)) != TIM_OK)
        return rc;
    tim::DistillArgs a{};
    a.grad = grad_loss;
    a.loss = loss;
    a.out_lse = lse;
    a.out_lse_tail = lse_tail;
    a.dz = dlogits;
    a.ldo = dlogits_stride;
    return distill(a, tim::LD_STEP, logits, dtype, N, V, stride, teacher_ids, teacher_logits, teacher_lse, K,
                   temperature, stream);
}

} // extern "C"
