// table_api.cu -- the C entry points of the operators beside the head's table:
// low-rank adapters on its logits, embedding lookup, and their gradients.
#include <algorithm>
#include <cmath>

#include "../../include/tim.h"
#include "logits_internal.h"
#include "table_internal.h"
#include "tim_internal.h"

namespace {

using tim::fail_message;

bool aligned(const void *p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

uintptr_t elem_bytes(int dtype) { return dtype == TIM_F32 ? 4 : 2; }

int invalid(const char *msg) { return fail_message(TIM_ERR_INVALID_ARG, "%s", msg); }

bool is_dtype(int d) { return d == TIM_F32 || d == TIM_BF16 || d == TIM_F16; }

int finish(cudaError_t e, cudaError_t freed, const char *what)
{
    if (e == cudaSuccess)
        e = freed;
    if (e != cudaSuccess)
        return fail_message(TIM_ERR_CUDA, "%s: %s", what, cudaGetErrorString(e));
    return tim::record_error(TIM_OK, "");
}

// Do two ranges of bytes share one?
bool overlap(const void *a, int64_t na, const void *b, int64_t nb)
{
    const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
    return na > 0 && nb > 0 && x < y + static_cast<uintptr_t>(nb) && y < x + static_cast<uintptr_t>(na);
}

// Sizes, adapters and rows; N = 0 and no adapters are legal.
int check_adapters(int64_t N, int64_t D, const void *h, const tim_adapters *ad, const int32_t *rows)
{
    if (N >= int64_t(1) << 30)
        return fail_message(TIM_ERR_INVALID_ARG, "N = %lld out of range [0, 2^30)", static_cast<long long>(N));
    if (D <= 0 || D % 8 != 0 || D > 65536)
        return fail_message(TIM_ERR_INVALID_ARG, "D = %lld must be positive, a multiple of 8 and <= 65536",
                            static_cast<long long>(D));
    if (!ad)
        return invalid("adapters is null");
    if (ad->rank < 8 || ad->rank > tim::AD_MAX_RANK || ad->rank % 8 != 0)
        return fail_message(TIM_ERR_INVALID_ARG, "rank = %d must be a multiple of 8 in [8, %d]", ad->rank,
                            tim::AD_MAX_RANK);
    if (ad->num_adapters < 0 || ad->num_adapters > tim::AD_MAX_ADAPTERS)
        return fail_message(TIM_ERR_INVALID_ARG, "num_adapters = %d out of range [0, %d]", ad->num_adapters,
                            tim::AD_MAX_ADAPTERS);
    if (ad->num_adapters > 0 && (!ad->A || !ad->B))
        return invalid("A and B are required");
    if (!aligned(ad->A, 16) || !aligned(ad->B, 16) || !aligned(ad->scale, 4))
        return invalid("A and B must be 16-byte aligned, scale 4-byte aligned");
    if (N > 0 && (!h || !rows))
        return invalid("h and rows are required");
    if (!aligned(h, 16) || !aligned(rows, 4))
        return invalid("h must be 16-byte aligned, rows 4-byte aligned");
    return TIM_OK;
}

// Does an output share a byte with h, the adapters or the rows?
bool over_adapters(const void *out, int64_t bytes, int64_t N, int64_t V, int64_t D, const void *h, const tim_adapters *ad,
                   const int32_t *rows)
{
    const int64_t n = ad->num_adapters, R = ad->rank;
    return overlap(out, bytes, h, 2 * N * D) || overlap(out, bytes, ad->A, 2 * n * R * D) ||
           overlap(out, bytes, ad->B, 2 * n * V * R) || overlap(out, bytes, rows, 4 * N) ||
           overlap(out, bytes, ad->scale, ad->scale ? 4 * n : 0);
}

int check_table(int64_t N, int64_t V, int64_t D, int dtype, const int32_t *tokens)
{
    if (!is_dtype(dtype))
        return invalid("dtype must be TIM_F32, TIM_BF16 or TIM_F16");
    if (N < 0 || N >= int64_t(1) << 30)
        return fail_message(TIM_ERR_INVALID_ARG, "N = %lld out of range [0, 2^30)", static_cast<long long>(N));
    if (V <= 0 || V > tim::LG_MAX_V)
        return fail_message(TIM_ERR_INVALID_ARG, "V = %lld out of range (0, %lld]", static_cast<long long>(V),
                            static_cast<long long>(tim::LG_MAX_V));
    if (D <= 0 || D > 65536)
        return fail_message(TIM_ERR_INVALID_ARG, "D = %lld out of range (0, 65536]", static_cast<long long>(D));
    if (N * ((D + 255) / 256) >= int64_t(1) << 31)
        return invalid("N x D too large for one call");
    if (N > 0 && !tokens)
        return invalid("tokens is null");
    if (!aligned(tokens, 4))
        return invalid("tokens must be 4-byte aligned");
    return TIM_OK;
}

} // namespace

extern "C" {

int tim_adapter_logits(const void *logits, int dtype, int64_t N, int64_t V, int64_t stride, const void *h, int64_t D,
                       const tim_adapters *adapters, const int32_t *rows, void *out, int64_t out_stride,
                       tim_stream_t stream)
{
    int rc = tim::check_logits(logits, dtype, N, V, stride);
    if (rc < 0)
        return rc;
    const bool empty = rc == 1;
    if ((rc = check_adapters(N, D, h, adapters, rows)) != TIM_OK)
        return rc;
    if (empty)
        return tim::record_error(TIM_OK, "");
    if ((rc = tim::check_logits_out(logits, dtype, N, V, stride, out, dtype, out_stride)) != TIM_OK)
        return rc;
    if (over_adapters(out, ((N - 1) * out_stride + V) * static_cast<int64_t>(elem_bytes(dtype)), N, V, D, h, adapters, rows))
        return invalid("the output overlaps an input");
    tim::AdapterArgs a{};
    a.in_place = out == logits;
    if (a.in_place && adapters->num_adapters == 0)
        return tim::record_error(TIM_OK, "");
    int *status = nullptr, sms = 0;
    if ((rc = tim::use_device(&status, &sms)) != TIM_OK)
        return rc;
    a.h = static_cast<const uint16_t *>(h);
    a.A = static_cast<const uint16_t *>(adapters->A);
    a.B = static_cast<const uint16_t *>(adapters->B);
    a.scale = adapters->scale;
    a.rows = rows;
    a.N = static_cast<int32_t>(N);
    a.V = static_cast<int32_t>(V);
    a.D = static_cast<int32_t>(D);
    a.R = adapters->rank;
    a.n = adapters->num_adapters;
    a.z = logits;
    a.ld = stride;
    a.out = out;
    a.ldo = out_stride;
    // t in parts.  Two leave 2^-16 of it at most: below a bf16 output's own rounding (2^-8) and an fp16's
    // (2^-11).  512 x 32000 of rank 16: 0.03 % of bf16 outputs and 0.22 % of fp16 ones are not the correctly
    // rounded ones (0.003 and 0.02 % with t and sums in fp32); where z is about -t B an fp16 output has only
    // some six bits of what is left.  A third part of fp16's takes 8192 x 151936, rank 16, from 899 us to 1107 at best.
    const int parts = dtype == TIM_F32 ? 3 : 2;
    const size_t b_off = tim::ws_round(sizeof(int32_t) * (static_cast<size_t>(a.n) + 2));
    const size_t b_n = tim::ws_round(sizeof(int32_t) * static_cast<size_t>(N));
    a.plan.t_pitch = parts * tim::ad_rank_pad(a.R) + 8;
    a.wait_budget_ns = tim::pipeline_wait_budget_ns();
    a.status = status;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    void *ws = nullptr;
    if ((rc = tim::workspace_alloc(&ws, b_off + 2 * b_n + static_cast<size_t>(N) * a.plan.t_pitch * 2, s)) != TIM_OK)
        return rc;
    char *w = static_cast<char *>(ws);
    a.plan.offsets = reinterpret_cast<int32_t *>(w);
    a.plan.perm = reinterpret_cast<int32_t *>(w + b_off);
    a.plan.adapter = reinterpret_cast<int32_t *>(w + b_off + b_n);
    a.plan.t = reinterpret_cast<uint16_t *>(w + b_off + 2 * b_n);
    cudaError_t e = tim::adapters_shrink_launch(a, parts, sms, s);
    if (e == cudaSuccess)
        e = tim::adapters_expand_launch(a, dtype, sms, s);
    return finish(e, tim::workspace_free(ws, s), "adapter_logits launch");
}

int tim_adapter_logits_backward(const void *dlogits, int dtype, int64_t N, int64_t V, int64_t stride, const void *h,
                                int64_t D, const tim_adapters *adapters, const int32_t *rows, float *dh, float *dA,
                                float *dB, int accumulate_dh, int accumulate_adapters, tim_stream_t stream)
{
    int rc = tim::check_logits(dlogits, dtype, N, V, stride);
    if (rc < 0)
        return rc;
    if ((rc = check_adapters(N, D, h, adapters, rows)) != TIM_OK)
        return rc;
    const int64_t n = adapters->num_adapters, R = adapters->rank;
    if ((N > 0 && !dh) || (n > 0 && (!dA || !dB)))
        return invalid("dh, dA and dB are required");
    if (!aligned(dh, 16) || !aligned(dA, 16) || !aligned(dB, 16))
        return invalid("dh, dA and dB must be 16-byte aligned");
    const int64_t bytes[3] = {4 * N * D, 4 * n * R * D, 4 * n * V * R};
    const void *outs[3] = {dh, dA, dB};
    const int64_t span = N > 0 ? ((N - 1) * stride + V) * static_cast<int64_t>(elem_bytes(dtype)) : 0;
    for (int i = 0; i < 3; ++i) {
        if (overlap(outs[i], bytes[i], dlogits, span) || over_adapters(outs[i], bytes[i], N, V, D, h, adapters, rows))
            return invalid("an output overlaps an input");
        for (int j = 0; j < i; ++j)
            if (overlap(outs[i], bytes[i], outs[j], bytes[j]))
                return invalid("two outputs overlap");
    }
    if (N == 0 && n == 0)
        return tim::record_error(TIM_OK, "");
    int *status = nullptr, sms = 0;
    if ((rc = tim::use_device(&status, &sms)) != TIM_OK)
        return rc;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    if (N == 0 || n == 0) {   // no products: zeros where nothing is added to
        cudaError_t e = cudaSuccess;
        if (N == 0 && !accumulate_adapters) {
            e = cudaMemsetAsync(dA, 0, static_cast<size_t>(bytes[1]), s);
            if (e == cudaSuccess)
                e = cudaMemsetAsync(dB, 0, static_cast<size_t>(bytes[2]), s);
        }
        if (N > 0 && !accumulate_dh)
            e = cudaMemsetAsync(dh, 0, static_cast<size_t>(bytes[0]), s);
        return finish(e, cudaSuccess, "adapter_logits_backward");
    }
    tim::AdapterArgs f{};
    f.h = static_cast<const uint16_t *>(h);
    f.A = static_cast<const uint16_t *>(adapters->A);
    f.scale = adapters->scale;
    f.rows = rows;
    f.N = static_cast<int32_t>(N);
    f.V = static_cast<int32_t>(V);
    f.D = static_cast<int32_t>(D);
    f.R = adapters->rank;
    f.n = adapters->num_adapters;
    f.status = status;
    tim::AdapterGradArgs a{};
    a.h = f.h;
    a.A = f.A;
    a.B = static_cast<const uint16_t *>(adapters->B);
    a.scale = f.scale;
    a.dy = dlogits;
    a.ld = stride;
    a.N = f.N;
    a.V = f.V;
    a.D = f.D;
    a.R = f.R;
    a.n = f.n;
    a.RT = tim::ad_rank_pad(R);
    a.aligned = aligned(dlogits, 16) && (N == 1 || stride * static_cast<int64_t>(elem_bytes(dtype)) % 16 == 0);
    const int RP = std::min(a.RT, 64);
    // a slab an SM while TMEM has room for its dB, else as many waves of them as it takes
    const int64_t blocks = (V + tim::AG_BLOCK - 1) / tim::AG_BLOCK, most = tim::ag_blocks(RP);
    const int64_t waves = (blocks + most * sms - 1) / (most * sms);
    const int64_t per_slab = (blocks + waves * sms - 1) / (waves * sms);
    a.cols = static_cast<int32_t>(per_slab * tim::AG_BLOCK);
    a.slabs = static_cast<int32_t>((blocks + per_slab - 1) / per_slab);
    a.merged = RP <= 32 && 2 * RP + per_slab * 2 * RP <= 512;
    // dB's sums: as many (up to four) as TMEM has room for beside du, for two adapters where that leaves two
    const int64_t columns = per_slab * (a.merged ? 2 : 1) * RP, fit = (512 - 2 * RP) / columns, sums = fit >= 4 ? fit / 2 : fit;
    a.low = !a.merged && sums >= 2;   // merged: the low products have columns of their own already
    a.chains = static_cast<int32_t>(std::min<int64_t>(sums - a.low, 4));
    const int products = tim::ag_step(dtype) / 16 * (a.merged || a.low ? 1 : tim::ag_products(tim::ag_planes(dtype)));
    a.link = a.chains * tim::ag_step(dtype) * (tim::AG_CHAIN / products);
    a.du_parts = a.slabs * tim::ag_planes(dtype);
    const int64_t per_row = int64_t(4) * a.du_parts * RP;
    a.row_part = static_cast<int32_t>(std::min<int64_t>(
        N, std::max<int64_t>(tim::AG_PARTIAL_BYTES / per_row / 128, 1) * 128));
    a.dh = dh;
    a.dA = dA;
    a.dB = dB;
    a.accumulate = accumulate_adapters != 0;
    a.accumulate_dh = accumulate_dh != 0;
    a.wait_budget_ns = tim::pipeline_wait_budget_ns();
    a.status = status;
    const size_t b_off = tim::ws_round(sizeof(int32_t) * (static_cast<size_t>(n) + 2));
    const size_t b_n = tim::ws_round(sizeof(int32_t) * static_cast<size_t>(N));
    const size_t t_rows = static_cast<size_t>(N) + static_cast<size_t>(n) * tim::AG_PAD;
    const size_t b_t = tim::ws_round(t_rows * 3 * a.RT * 2);
    const size_t b_du = tim::ws_round(static_cast<size_t>(N) * 3 * a.RT * 2);
    const size_t b_part = static_cast<size_t>(per_row) * (a.row_part + 16);
    void *ws = nullptr;
    if ((rc = tim::workspace_alloc(&ws, b_off + 2 * b_n + b_t + b_du + b_part, s)) != TIM_OK)
        return rc;
    char *w = static_cast<char *>(ws);
    f.plan.offsets = reinterpret_cast<int32_t *>(w);
    f.plan.perm = reinterpret_cast<int32_t *>(w + b_off);
    f.plan.adapter = reinterpret_cast<int32_t *>(w + b_off + b_n);
    w += b_off + 2 * b_n;
    f.plan.t = reinterpret_cast<uint16_t *>(w);
    f.plan.t_pitch = 3 * a.RT;
    f.plan.t_pad = tim::AG_PAD;
    a.plan = f.plan;
    a.du = reinterpret_cast<uint16_t *>(w + b_t);
    a.partial = reinterpret_cast<float *>(w + b_t + b_du);
    CUtensorMap maps[2];
    const uint64_t d_b[3] = {static_cast<uint64_t>(R), static_cast<uint64_t>(V), static_cast<uint64_t>(n)};
    const uint64_t s_b[2] = {static_cast<uint64_t>(R) * 2, static_cast<uint64_t>(V * R) * 2};
    const uint64_t d_t[2] = {static_cast<uint64_t>(3 * a.RT), t_rows}, s_t[1] = {static_cast<uint64_t>(3 * a.RT) * 2};
    const uint32_t box_b[3] = {static_cast<uint32_t>(RP), tim::AG_BLOCK, 1}, box_t[2] = {
        static_cast<uint32_t>(a.merged ? 2 * RP : RP), static_cast<uint32_t>(tim::ag_step(dtype))};
    if ((rc = tim::encode_bf16_map(&maps[0], a.B, 3, d_b, s_b, box_b, 2 * RP)) != TIM_OK ||
        (rc = tim::encode_bf16_map(&maps[1], f.plan.t, 2, d_t, s_t, box_t, a.merged ? 4 * RP : 2 * RP)) != TIM_OK) {
        tim::workspace_free(ws, s);
        return rc;
    }
    cudaError_t e = tim::adapters_shrink_launch(f, 3, sms, s);
    if (e == cudaSuccess)
        e = tim::adapters_grad_launch(maps, a, dtype, sms, s);
    return finish(e, tim::workspace_free(ws, s), "adapter_logits_backward launch");
}

int tim_embedding(const int32_t *tokens, int64_t N, const void *W, int dtype, int64_t V, int64_t D, float scale,
                  void *out, int out_dtype, tim_stream_t stream)
{
    int rc = check_table(N, V, D, dtype, tokens);
    if (rc != TIM_OK)
        return rc;
    if (!is_dtype(out_dtype))
        return invalid("out_dtype must be TIM_F32, TIM_BF16 or TIM_F16");
    if (!std::isfinite(scale))
        return invalid("scale must be finite");
    if (N == 0)
        return tim::record_error(TIM_OK, "");
    if (!W || !out)
        return invalid("null pointer argument");
    if (!aligned(W, elem_bytes(dtype)) || !aligned(out, elem_bytes(out_dtype)))
        return invalid("W and out must be aligned to their elements");
    const int64_t wb = V * D * static_cast<int64_t>(elem_bytes(dtype)), ob = N * D * static_cast<int64_t>(elem_bytes(out_dtype));
    if (overlap(W, wb, out, ob) || overlap(tokens, 4 * N, out, ob))
        return invalid("the output overlaps an input");
    int *status = nullptr, sms = 0;
    if ((rc = tim::use_device(&status, &sms)) != TIM_OK)
        return rc;
    tim::EmbeddingArgs a{};
    a.tokens = tokens;
    a.N = static_cast<int32_t>(N);
    a.V = static_cast<int32_t>(V);
    a.D = static_cast<int32_t>(D);
    a.scale = scale;
    a.status = status;
    a.x = W;
    a.out = out;
    return finish(tim::embedding_launch(a, dtype, out_dtype, reinterpret_cast<cudaStream_t>(stream)), cudaSuccess,
                  "embedding launch");
}

int tim_embedding_backward(const int32_t *tokens, int64_t N, const void *grad, int dtype, int64_t V, int64_t D,
                           float scale, float *dW, int accumulate_dW, tim_stream_t stream)
{
    int rc = check_table(N, V, D, dtype, tokens);
    if (rc != TIM_OK)
        return rc;
    if (!std::isfinite(scale))
        return invalid("scale must be finite");
    if (!dW || (N > 0 && !grad))
        return invalid("null pointer argument");
    if (!aligned(grad, elem_bytes(dtype)) || !aligned(dW, 4))
        return invalid("grad and dW must be aligned to their elements");
    const int64_t gb = N * D * static_cast<int64_t>(elem_bytes(dtype)), wb = 4 * V * D;
    if (overlap(grad, gb, dW, wb) || overlap(tokens, 4 * N, dW, wb))
        return invalid("dW overlaps an input");
    if (N == 0 && accumulate_dW)
        return tim::record_error(TIM_OK, "");
    int *status = nullptr, sms = 0;
    if ((rc = tim::use_device(&status, &sms)) != TIM_OK)
        return rc;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    if (N == 0)
        return finish(cudaMemsetAsync(dW, 0, static_cast<size_t>(wb), s), cudaSuccess, "cudaMemsetAsync(dW)");
    tim::EmbeddingArgs a{};
    a.tokens = tokens;
    a.N = static_cast<int32_t>(N);
    a.V = static_cast<int32_t>(V);
    a.D = static_cast<int32_t>(D);
    a.scale = scale;
    a.status = status;
    a.x = grad;
    a.dW = dW;
    a.accumulate = accumulate_dW != 0;
    const size_t b_off = tim::ws_round(sizeof(int32_t) * (static_cast<size_t>(V) + 1));
    const size_t b_n = tim::ws_round(sizeof(int32_t) * static_cast<size_t>(N));
    // a tile, and the joining of an id's tiles, is one warp's work: some sqrt(N) / 4 positions,
    // so that neither is long.  65536 equal tokens of 4096 bf16: 1064 us in tiles of 32, 758 of 64, 613
    // of 128; 32768 tokens of ordinary frequencies 425 in tiles of 32, 429 of 64, 437 of 128
    a.tile = tim::EM_TILE;
    while (int64_t(16) * a.tile * a.tile < N)
        a.tile *= 2;
    a.many = std::max(tim::EM_LONG, a.tile);
    const size_t tiles = N > a.many ? (static_cast<size_t>(N) + a.tile - 1) / a.tile : 0;
    const size_t b_part = tiles * 2 * static_cast<size_t>(D) * sizeof(float);
    void *ws = nullptr;
    if ((rc = tim::workspace_alloc(&ws, b_off + 4 * b_n + b_part, s)) != TIM_OK)
        return rc;
    char *w = static_cast<char *>(ws);
    a.offsets = reinterpret_cast<int32_t *>(w);
    a.order = reinterpret_cast<int32_t *>(w + b_off);
    a.ids = reinterpret_cast<int32_t *>(w + b_off + b_n);
    a.staged = reinterpret_cast<int2 *>(w + b_off + 2 * b_n);
    a.partial = reinterpret_cast<float *>(w + b_off + 4 * b_n);
    cudaError_t e = tim::embedding_sort_launch(a, s);
    if (e == cudaSuccess)
        e = tim::embedding_sum_launch(a, dtype, s);
    return finish(e, tim::workspace_free(ws, s), "embedding_backward launch");
}

} // extern "C"
