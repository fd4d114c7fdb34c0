// distill_topk.cu -- distillation of a head's logits from a teacher's top
// logits: the loss, its gradient, and both in one call.
//
// Row i lists ids k with the teacher's logits t_k.  With p = softmax(z / tau):
//   without the teacher's lse  q = softmax over the listed ids of t / tau,
//                              L = sum_k q_k (log q_k - log p_k),
//                              dL/dz_v = (p_v - q_v) / tau;
//   with it                    q_k = e^(t_k / tau - lse_T), the rest q_o = 1 - sum q_k is
//                              one more outcome, whose student probability is that of
//                              the ids not listed, p_o = 1 - sum p_k:
//                              L = sum_k q_k (log q_k - log p_k) + q_o (log q_o - log p_o),
//                              dL/dz_v = (p_v - q_v) / tau for the listed ids and
//                              p_v (1 - q_o / p_o) / tau = (p_o - q_o) r_v / tau for the
//                              others, r_v = p_v / p_o (computed as a softmax of its own).
// (q_v is 0 for ids that are not listed; an id listed twice adds up.)  log p_o is the
// log-sum-exp over the columns whose bit is not set in a bitmap of the listed
// ids, never 1 - sum p_k, which loses all its digits when p_o is small.
//
// What bounds it: the row streams through once for the sums and once for the
// gradient; the listed ids cost K gathers and K stores.  The gradient pass writes
// every column as if it were not listed; after a barrier the listed ones, all of
// which the same CTA owns, are written over.  In a step the row comes from memory
// once: a cluster holds it in its CTAs' shared memory (one bulk copy each, of at most
// 52 KB while fewer than eight CTAs share the row, up to LD_SMEM then) between the
// passes, and the CTAs exchange the slices' partials.
//
// Measured on a GB300 against the bytes each has to move at 6760 GB/s:
//   loss      8192 x 151936 bf16, K = 64   390 us of 369 us: memory; 495 us with a tail:
//             issue slots; 1024 x 129280 fp32 81 us of 78 us
//   gradient  4096 x 128256 bf16, K = 64   308 to 312 us of 311 us: memory; 1024 x 129280
//             fp32 165 us of 157 us
//   step      4096 x 151936 bf16, K = 64   511 us of 369 us (507 us with a tail), 1024 x
//             129280 fp32 with a tail, K = 128, 222 us of 157 us: a CTA's life of 10 us (row
//             2.5 us, sums 2 us, the other CTAs 2 us, gradient 2 us), of which five (39 KB of
//             row each) or three (64 KB) fit an SM
#include <algorithm>
#include <cstddef>

#include "logits_rows.cuh"

namespace tim {
namespace {

// What a row's teacher contributes besides its own q_k.
struct TeacherRow {
    float max;    // largest t_k (0 for a tail: not used)
    float lse;    // log sum e^((t_k - max) / tau), or the given one
    float rest;   // q_o (0 without a tail)
    int any;      // the row lists something (without a tail: of a probability above 0)
};

// Shared memory of a CTA: the header, the slices' partials, the student's z at the
// listed ids, the bitmap of the rank's columns, the table drop8 takes (16-bit types
// with a tail), the rank's part of the row.
struct Head {
    uint64_t bar, parts;   // the row's copy; the partials and the teacher's statistics
    int dup, abort, pad[2];
    TeacherRow teacher;
    float m, s, mr, sr;   // all columns; those that are not listed
};

struct Layout {
    uint32_t part, x, bits, masks, row, bytes;
};

template <typename T> __host__ __device__ inline Layout layout(int slices, int per, int K, bool sums, bool bits, bool tail, bool hold)
{
    Layout l;
    l.part = sizeof(Head);
    l.x = l.part + (sums ? static_cast<uint32_t>(slices) * 16 : 0);
    l.bits = l.x + (sums ? static_cast<uint32_t>(K + 3) / 4 * 16 : 0);
    l.masks = l.bits + (bits ? static_cast<uint32_t>(per) * (LG_SLICE / 8) : 0);
    l.row = l.masks + (sums && tail && sizeof(T) == 2 ? static_cast<uint32_t>(sizeof(HalfMasks)) : 0);
    l.bytes = l.row + (hold ? static_cast<uint32_t>(per) * LG_SLICE * static_cast<uint32_t>(sizeof(T)) + 16 : 0);
    return l;
}

// log q of a listed id from t / tau = hi + lo and the teacher's log-sum-exp:
// hi - lse is exact when they are close, so large probabilities keep their digits.
__device__ __forceinline__ float teacher_logq(float t, float tau, float lse)
{
    const float hi = t / tau;
    const float lo = isfinite(hi) ? fmaf(-hi, tau, t) / tau : 0.f;
    return (hi - lse) + lo;
}

// log q_k of a listed id.
template <bool TAIL> __device__ __forceinline__ float listed_logq(float t, float tau, const TeacherRow &w)
{
    return w.any ? teacher_logq(TAIL ? t : t - w.max, tau, w.lse) : neg_inf();
}

__device__ __forceinline__ float q_of(float logq) { return logq == neg_inf() ? 0.f : expf(logq); }

// The q_o that counts.  Where the student gives the rest nothing (p_o, or the largest of
// the rest relative to the row's largest, is 0 in fp32: a list that holds every id, a
// grammar both are under), what the rounding of the teacher's lse and of sum q_k can
// leave of 1 - sum q_k is 0: four roundings of the lse, 64 of the sum.  log p_o = -inf
// would make an infinite loss of it.
__device__ __forceinline__ float counted_rest(const TeacherRow &w, float p_o)
{
    const float noise = fminf(0.5f, 0x1p-22f * (16.f + fabsf(w.lse)));
    return p_o == 0.f && w.rest <= noise ? 0.f : w.rest;
}

__device__ __forceinline__ bool in_use(int id, int V) { return id >= 0 && id < V; }

// One warp; the same in every lane.  Also the student's logits at the listed ids,
// for the loss (listed_x, where it is given).
template <typename T, bool TAIL>
__device__ __forceinline__ TeacherRow teacher_row(const DistillArgs &a, int row, int lane, const T *z, float *listed_x)
{
    const int32_t *ids = a.ids + static_cast<int64_t>(row) * a.K;
    const float *t = a.teacher + static_cast<int64_t>(row) * a.K;
    TeacherRow w{0.f, 0.f, 0.f, 0};
    bool any = false;
    float top = neg_inf();
    for (int k = lane; k < a.K; k += 32)
        if (in_use(ids[k], a.V)) {
            any = true;
            top = fmaxf(top, t[k]);
            if (listed_x)
                listed_x[k] = Elem<T>::load(z + ids[k]);
        }
    w.any = __any_sync(0xffffffffu, any);
    float s = 0.f;
    if constexpr (TAIL) {
        w.lse = a.teacher_lse[row];
        for (int k = lane; k < a.K; k += 32)
            if (in_use(ids[k], a.V))
                s += q_of(listed_logq<true>(t[k], a.temperature, w));
        s = warp_sum(s);
        w.rest = s <= 1.f ? 1.f - s : (s > 1.f ? 0.f : s);   // NaN stays
    } else {
        w.max = finite_ref(warp_max(top));
        for (int k = lane; k < a.K; k += 32)
            if (in_use(ids[k], a.V))
                s += expf((t[k] - w.max) / a.temperature);
        s = warp_sum(s);
        w.lse = logf(s);
        w.any = w.any && s != 0.f;
    }
    return w;
}

// The rank's columns z[c0 .. c1) into shared memory at dst + shift bytes: one bulk
// copy of the whole 16-byte pieces, the up to seven elements before and after
// them by plain loads (so nothing outside the row is read).  All threads; the
// plain stores are visible after the next barrier of the CTA.
template <int NT, typename T>
__device__ __forceinline__ void fetch_row(const T *z, int c0, int c1, uint32_t shift, uint8_t *dst, uint32_t bar)
{
    const uintptr_t a0 = reinterpret_cast<uintptr_t>(z + c0), a1 = reinterpret_cast<uintptr_t>(z + c1);
    const uintptr_t base = a0 - shift;                       // the 16-byte boundary that dst stands for
    uintptr_t lo = (a0 + 15) & ~uintptr_t(15), hi = a1 & ~uintptr_t(15);
    if (hi <= lo)
        lo = hi = a1;                                        // shorter than a piece
    if (threadIdx.x == 0) {
        const uint32_t bytes = static_cast<uint32_t>(hi - lo);
        mbar_arrive_expect_tx(bar, bytes);
        if (bytes > 0)
            bulk_load(smem_u32(dst) + static_cast<uint32_t>(lo - base), reinterpret_cast<const void *>(lo), bytes, bar,
                      l2_policy_evict_first());
    }
    const int head = static_cast<int>((lo - a0) / sizeof(T)), tail = static_cast<int>((a1 - hi) / sizeof(T));
    T *s = reinterpret_cast<T *>(dst + shift);
    for (int i = threadIdx.x; i < head + tail; i += NT) {
        const int col = i < head ? i : (c1 - c0) - (head + tail) + i;
        s[col] = z[c0 + col];
    }
}

// HOLD: the rank's part of the row stays in shared memory between the two passes
// of a step.
template <typename T, int OP, bool TAIL, bool HOLD, int NT>
__global__ void __launch_bounds__(NT) distill_kernel(const DistillArgs a)
{
    constexpr int WARPS = NT / 32;
    constexpr bool SUMS = OP != LD_BACKWARD, GRAD = OP != LD_FORWARD, BITS = TAIL || GRAD;
    extern __shared__ __align__(16) uint8_t smem[];
    const int slices = (a.V + LG_SLICE - 1) / LG_SLICE;
    const Layout lay = layout<T>(slices, a.per, a.K, SUMS, BITS, TAIL, HOLD);
    Head &hd = *reinterpret_cast<Head *>(smem);
    float4 *part = reinterpret_cast<float4 *>(smem + lay.part);
    float *listed_x = reinterpret_cast<float *>(smem + lay.x);
    uint32_t *bitmap = reinterpret_cast<uint32_t *>(smem + lay.bits);   // columns of this rank
    HalfMasks &masks = *reinterpret_cast<HalfMasks *>(smem + lay.masks);
    const int rank = static_cast<int>(blockIdx.x % static_cast<unsigned>(a.ranks));
    const int row = static_cast<int>(blockIdx.x / static_cast<unsigned>(a.ranks));
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int s0 = min(slices, rank * a.per), s1 = min(slices, s0 + a.per);
    const int c0 = min(a.V, s0 * LG_SLICE), c1 = min(a.V, s1 * LG_SLICE);
    const T *z = static_cast<const T *>(a.z) + row * a.ld;
    T *dz = GRAD ? static_cast<T *>(a.dz) + row * a.ldo : nullptr;
    const uint32_t shift = row_shift(z), shift_out = GRAD ? row_shift(dz) : 0u;
    const int32_t *ids = a.ids + static_cast<int64_t>(row) * a.K;
    const float *teacher = a.teacher + static_cast<int64_t>(row) * a.K;
    const float tau = a.temperature, inv_tau = 1.f / tau, k2 = LG_LOG2E * inv_tau;
    float g = 0.f;
    if constexpr (GRAD)
        g = a.grad[row];
    TIM_DCHECK(!GRAD || threadIdx.x != 0 || rank != 0 || (isfinite(g) && (SUMS || a.lse[row] < INFINITY)), a.status,
               TIM_CHECK_BACKWARD_INPUT, row, __float_as_uint(g));
    const int takers = GRAD ? a.ranks : 1;   // ranks that fold the row's partials
    // the columns as the passes read them: from memory, or from this CTA's copy
    const T *src = HOLD ? reinterpret_cast<const T *>(smem + lay.row + shift) : z;
    const int off = HOLD ? c0 : 0;
    if (threadIdx.x == 0) {
        hd.dup = 0;
        hd.abort = 0;
        if constexpr (SUMS) {
            mbar_init(smem_u32(&hd.bar), 1);
            mbar_init(smem_u32(&hd.parts), 1);
            fence_mbar_init();
            if (a.ranks > 1 && rank < takers)
                mbar_arrive_expect_tx(smem_u32(&hd.parts), static_cast<uint32_t>(slices) * 16 + 16);
        }
    }
    if constexpr (HOLD) {
        // rank 0's last warp passes no other barrier before it waits for the row:
        // barrier 3 brings it the abort word as it was set above
        if (rank == 0 && warp == 0)
            named_arrive(3, 64);
        fetch_row<NT>(z, c0, c1, shift, smem + lay.row, smem_u32(&hd.bar));
    }
    if (SUMS && a.ranks > 1)
        cluster_arrive_relaxed();   // waited for before the first store into another CTA's shared memory

    auto zero_row = [&] {
        const float v[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
        for (int b = c0 + warp * 256; b < c1; b += WARPS * 256)
            store8<T>(dz, b + lane * 8, c1, shift_out, pack8<T>(v));
    };
    if constexpr (!SUMS) {
        if (g == 0.f) {
            zero_row();
            return;
        }
    }

    // the thread's first listed id and its teacher's logit, ahead of their use
    const int id0 = static_cast<int>(threadIdx.x) < a.K ? ids[threadIdx.x] : -1;
    const float t0 = static_cast<int>(threadIdx.x) < a.K ? teacher[threadIdx.x] : 0.f;
    // In a call with sums rank 0's last warp takes no columns: it finds the teacher's
    // statistics while the row comes in and hands them to every rank.  (As one more
    // task of a warp with columns they were what all the ranks waited for, some
    // 2 us of a CTA's 11.)
    const bool teacher_warp = SUMS && rank == 0 && warp == WARPS - 1;
    const int workers = SUMS && rank == 0 ? WARPS - 1 : WARPS;
    auto mark = [&] {   // this rank's listed ids in the bitmap
        for (int k = threadIdx.x; k < a.K; k += workers * 32) {
            const int id = ids[k];
            if (id >= c0 && id < c1) {
                const uint32_t bit = 1u << ((id - c0) & 31);
                if (atomicOr(bitmap + ((id - c0) >> 5), bit) & bit)
                    hd.dup = 1;
            }
        }
    };
    if constexpr (BITS) {
        for (int j = threadIdx.x; j < (c1 - c0 + 31) / 32; j += NT)
            bitmap[j] = 0;
    }
    if constexpr (TAIL || !SUMS) {
        if constexpr (SUMS && TAIL && sizeof(T) == 2)
            masks.fill();
        if (teacher_warp) {   // does not wait for the bitmap
            named_arrive(1, NT);
            named_arrive(2, NT);
        } else {
            named_sync(1, NT);
            mark();
            named_sync(2, NT);
        }
    } else if constexpr (HOLD) {   // the row's first and last elements, stored plainly
        if (teacher_warp)
            named_arrive(1, NT);
        else
            named_sync(1, NT);
    }
    // No rank writes a gradient before it has the statistics, so the gathers of z are
    // over by then.
    TeacherRow tr{0.f, 0.f, 0.f, 0};
    if constexpr (HOLD)
        if (teacher_warp)
            named_sync(3, 64);
    if (teacher_warp || (!SUMS && warp == WARPS - 1)) {
        tr = teacher_row<T, TAIL>(a, row, lane, z, SUMS ? listed_x : nullptr);
        if (lane == 0 && (!SUMS || a.ranks == 1))
            hd.teacher = tr;
    }
    if constexpr (!SUMS)
        __syncthreads();

    if constexpr (SUMS) {
        // The sums: of the columns that are not listed (all of them without a tail)
        // and of the listed ones, slice by slice.  Each partial goes to every CTA that
        // folds the row as it comes up: a store that counts its bytes on the other
        // CTA's barrier, so no CTA waits for another's stores.
        uint32_t peer = 0;   // shared memory of rank `lane`
        if (a.ranks > 1) {
            cluster_wait();   // every CTA's barriers exist
            if (lane < takers)
                peer = mapa_shared(smem_u32(smem), static_cast<uint32_t>(lane));
            if (teacher_warp && lane < takers)
                st_async_f4(peer + static_cast<uint32_t>(offsetof(Head, teacher)), tr.max, tr.lse, tr.rest,
                            __int_as_float(tr.any), peer + static_cast<uint32_t>(offsetof(Head, parts)));
        } else {
            __syncthreads();
        }
        bool late = false;
        if constexpr (HOLD) {
            late = !mbar_wait_sleep(smem_u32(&hd.bar), 0, &hd.abort, a.wait_budget_ns);
            if (late) {
                atomicCAS(a.status, 0, static_cast<int>(TIM_ERR_TIMEOUT));
                drain_wait(smem_u32(&hd.bar), 0);
            }
        }
        for (int sl = teacher_warp ? s1 : s0 + warp; sl < s1; sl += workers) {
            Raw8<T> raw[4];
            load_chunks<T, 4>(raw, src, sl * LG_SLICE - off, c1 - off, shift);
            float lm, ls, km = neg_inf(), ks = 0.f;
            if constexpr (TAIL) {   // the listed ones out of the stream, one by one
#pragma unroll
                for (int u = 0; u < 4; ++u) {
                    const int col = sl * LG_SLICE + u * 256 + lane * 8;
                    const uint32_t bits =
                        col < c1 ? reinterpret_cast<const uint8_t *>(bitmap)[(col - c0) >> 3] : 0u;
                    if (bits) {
#pragma unroll
                        for (int i = 0; i < 8; ++i)
                            if (bits >> i & 1)
                                join_value(km, ks, Elem<T>::get(raw[u].w, i), k2);
                        drop8(raw[u], bits, masks);
                    }
                }
                if (__any_sync(0xffffffffu, ks != 0.f))
                    warp_join(km, ks, k2);
            }
            warp_sums<T, 4>(raw, k2, nullptr, 0, lm, ls);
            if (late)
                ls = quiet_nan();
            if (a.ranks == 1) {
                if (lane == 0)
                    part[sl] = make_float4(lm, ls, km, ks);
            } else if (lane < takers) {
                st_async_f4(peer + lay.part + static_cast<uint32_t>(sl) * 16, lm, ls, km, ks,
                            peer + static_cast<uint32_t>(offsetof(Head, parts)));
            }
        }
        if (a.ranks == 1 || (GRAD && !TAIL) || (!GRAD && rank == 0))
            __syncthreads();   // partials and listed logits, the cleared bitmap
        if (!GRAD && (rank != 0 || warp != 0))
            return;
        if constexpr (GRAD && !TAIL)
            if (!teacher_warp)
                mark();   // (while the other CTAs' partials come in)
        bool lost = false;
        if (a.ranks > 1 && warp == 0) {
            lost = !mbar_wait_cluster(smem_u32(&hd.parts), 0, &hd.abort, a.wait_budget_ns);
            if (lost) {
                atomicCAS(a.status, 0, static_cast<int>(TIM_ERR_TIMEOUT));
                drain_wait(smem_u32(&hd.parts), 0);
            }
        }
        if (warp == 0) {   // fold in slice order: lane l takes slices l, l + 32, ...
            float mr = neg_inf(), sr = 0.f, km = neg_inf(), ks = 0.f;
            for (int j = lane; j < slices; j += 32) {
                const float4 p = part[j];
                join(mr, sr, p.x, p.y, k2);
                if constexpr (TAIL)
                    join(km, ks, p.z, p.w, k2);
            }
            warp_join(mr, sr, k2);
            float m = mr, s = sr;
            if constexpr (TAIL) {
                warp_join(km, ks, k2);
                join(m, s, km, ks, k2);
            }
            if (lane == 0) {
                hd.m = m;
                hd.s = lost ? quiet_nan() : s;
                hd.mr = mr;
                hd.sr = sr;
            }
            __syncwarp();
        }
        if constexpr (GRAD)
            __syncthreads();
    }

    auto write_loss = [&] {   // one warp of rank 0
        const TeacherRow tr = hd.teacher;
        const float m = hd.m, s = hd.s, mr = hd.mr, sr = hd.sr;
        float loss = 0.f;
        for (int k = lane; k < a.K; k += 32)
            if (in_use(ids[k], a.V)) {
                const float lq = listed_logq<TAIL>(teacher[k], tau, tr), q = q_of(lq);
                if (q != 0.f)   // NaN goes on
                    loss = __fmaf_rn(q, lq - row_logp(listed_x[k], m, s, inv_tau), loss);
            }
        loss = warp_sum(loss);
        if constexpr (TAIL) {
            const float rest = counted_rest(tr, sr == 0.f ? 0.f : exp2_approx((mr - m) * k2));
            if (rest != 0.f)
                loss = __fmaf_rn(rest,
                                 logf(rest) - (sr == 0.f ? neg_inf() : __fmaf_rn(mr - m, inv_tau, logf(sr) - logf(s))), loss);
        }
        if (lane == 0) {
            a.loss[row] = loss;
            a.out_lse[row] = row_lse(m, s, inv_tau);
            if (TAIL)
                a.out_lse_tail[row] = row_lse(mr, sr, inv_tau);
        }
    };
    if constexpr (!GRAD) {
        write_loss();
        return;
    }

    if constexpr (GRAD) {
        // (a row whose list carries nothing has the constant loss 0)
        if ((SUMS && g == 0.f) || (!TAIL && !hd.teacher.any)) {
            zero_row();
            if (SUMS && rank == 0 && warp == WARPS - 1)
                write_loss();
            return;
        }
        // p_v = 2^((z_v first - ref) second) scale: the row's maximum and 1 / sum in a
        // step, the forward's lse in a backward call.  The ids that are not listed have
        // (p_o - q_o) r_v, r_v = 2^((z_v first - rest_ref) second) rest_scale <= 1 the
        // student's distribution over them alone: p_v (1 - q_o / p_o) without a quotient
        // that overflows when p_o is small.
        const TeacherRow w = hd.teacher;
        const float gi = g / tau;
        const float first = SUMS ? 1.f : inv_tau, second = SUMS ? k2 : LG_LOG2E;
        float ref, scale = 1.f, rest_ref, others;   // others: what multiplies 2^(..) of the ids that are not listed
        if constexpr (SUMS) {
            ref = rest_ref = finite_ref(hd.m);
            scale = hd.s == 0.f ? 0.f : 1.f / hd.s;
            others = scale;
            if constexpr (TAIL) {
                rest_ref = finite_ref(hd.mr);
                const float p_o = hd.sr * exp2_approx((hd.mr - ref) * k2) * scale;
                others = hd.sr == 0.f ? 0.f : (p_o - counted_rest(w, p_o)) / hd.sr;
            }
        } else {
            ref = a.lse[row];
            const float lse = ref;
            if (ref == neg_inf())
                ref = -neg_inf();
            rest_ref = ref;
            others = 1.f;
            if constexpr (TAIL) {
                rest_ref = a.lse_tail[row];
                const float p_o = prob2((rest_ref - lse) * LG_LOG2E);
                others = rest_ref == neg_inf() ? 0.f : p_o - counted_rest(w, p_o);
                if (rest_ref == neg_inf())
                    rest_ref = -neg_inf();
            }
        }
        // the listed ids' values first: z may be written over in place
        constexpr int KPT = (LD_MAX_K + NT - 1) / NT;
        float own[KPT];
#pragma unroll
        for (int n = 0; n < KPT; ++n) {
            const int k = static_cast<int>(threadIdx.x) + n * NT;
            own[n] = 0.f;
            if (n * NT >= a.K)
                continue;
            const int id = k >= a.K ? -1 : n == 0 ? id0 : ids[k];
            if (id >= c0 && id < c1) {
                float q = 0.f;
                if (hd.dup) {   // ids listed more than once add up, in the list's order: K steps for each id of this CTA
                    for (int j = 0; j < a.K; ++j)
                        q += ids[j] == id ? q_of(listed_logq<TAIL>(teacher[j], tau, w)) : 0.f;
                } else {
                    q = q_of(listed_logq<TAIL>(n == 0 ? t0 : teacher[k], tau, w));
                }
                const float e = fmaf(Elem<T>::load(src + id - off), first, -ref) * second;
                const float p = SUMS ? exp2_approx(e) * scale : prob2(e);
                own[n] = (p - q) * gi;
            }
        }
        if constexpr (!HOLD)
            __syncthreads();
        const float wgi = others * gi;
        const Pair first2 = pair(first, first), ref2 = pair(-rest_ref, -rest_ref), second2 = pair(second, second),
                   w2 = pair(wgi, wgi);
        for (int b = c0 + warp * 512; b < c1; b += WARPS * 512) {
            Raw8<T> raw[2];
            load_chunks<T, 2>(raw, src, b - off, c1 - off, shift);
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                float v[8];
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    float lo, hi;
                    unpair(mul2(fma2(get2<T>(raw[u], k), first2, ref2), second2), lo, hi);
                    const Pair p = SUMS ? pair(exp2_approx(lo), exp2_approx(hi)) : pair(prob2(lo), prob2(hi));
                    unpair(mul2(p, w2), v[2 * k], v[2 * k + 1]);
                }
                store8<T>(dz, b + u * 256 + lane * 8, c1, shift_out, pack8<T>(v));
            }
        }
        __syncthreads();
#pragma unroll
        for (int n = 0; n < KPT; ++n) {
            const int k = static_cast<int>(threadIdx.x) + n * NT;
            if (n * NT >= a.K)
                break;
            const int id = k >= a.K ? -1 : n == 0 ? id0 : ids[k];
            if (id >= c0 && id < c1)
                dz[id] = Elem<T>::from(own[n]);
        }
        if (SUMS && rank == 0 && warp == WARPS - 1)
            write_loss();
    }
}

template <typename T, int OP, bool TAIL, bool HOLD, int NT>
cudaError_t launch_kernel(const DistillArgs &a, const Layout &l, cudaStream_t s)
{
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(static_cast<unsigned>(a.N) * static_cast<unsigned>(a.ranks));
    cfg.blockDim = dim3(NT);
    cfg.dynamicSmemBytes = l.bytes;
    cfg.stream = s;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = static_cast<unsigned>(a.ranks);
    at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = OP != LD_BACKWARD && a.ranks > 1 ? 1 : 0;   // (the backward's CTAs do not meet)
    return cudaLaunchKernelEx(&cfg, distill_kernel<T, OP, TAIL, HOLD, NT>, a);
}

template <typename T, int OP, bool TAIL> cudaError_t launch(DistillArgs a, int num_sms, cudaStream_t s)
{
    const int slices = lg_slices(a.V);
    // CTAs of a row: more while the rows alone leave SMs idle, and in the single passes
    // while parts stay long, so that the last of the CTAs end together (forward of 1941
    // rows of 116416 bf16 91 us against 105 us)
    int ranks = 1;
    const int64_t rows = a.N;
    while (ranks < LG_CLUSTER && ((ranks * 2 <= slices && rows * ranks < 4 * num_sms) ||
                                  (OP != LD_STEP && ranks * 32 <= slices && rows * ranks < 16 * num_sms)))
        ranks *= 2;
    if (OP == LD_STEP)   // a rank's part of the row: at most 52 KB where eight ranks allow it, so that four or five CTAs fit an SM
        while (ranks < LG_CLUSTER && static_cast<size_t>((slices + ranks - 1) / ranks) * LG_SLICE * sizeof(T) > 52 * 1024)
            ranks *= 2;
    a.per = (slices + ranks - 1) / ranks;
    a.ranks = (slices + a.per - 1) / a.per;
    constexpr bool SUMS = OP != LD_BACKWARD, BITS = TAIL || OP != LD_FORWARD;
    // short parts: half the threads, twice the CTAs (step of 4096 rows of 8192 fp16 with a
    // tail 52 us against 65 us)
    const bool few = a.per <= LD_FEW;
    if constexpr (OP == LD_STEP) {
        const Layout l = layout<T>(slices, a.per, a.K, SUMS, BITS, TAIL, true);
        if (l.bytes <= LD_SMEM)
            return few ? launch_kernel<T, OP, TAIL, true, LD_THREADS / 2>(a, l, s)
                       : launch_kernel<T, OP, TAIL, true, LD_THREADS>(a, l, s);
        return launch_kernel<T, OP, TAIL, false, LD_THREADS>(a, layout<T>(slices, a.per, a.K, SUMS, BITS, TAIL, false), s);
    } else {
        const Layout l = layout<T>(slices, a.per, a.K, SUMS, BITS, TAIL, false);
        return few ? launch_kernel<T, OP, TAIL, false, LD_THREADS / 2>(a, l, s)
                   : launch_kernel<T, OP, TAIL, false, LD_THREADS>(a, l, s);
    }
}

template <typename T> cudaError_t launch_op(const DistillArgs &a, int op, int num_sms, cudaStream_t s)
{
    const bool tail = a.teacher_lse != nullptr;
    if (op == LD_FORWARD)
        return tail ? launch<T, LD_FORWARD, true>(a, num_sms, s) : launch<T, LD_FORWARD, false>(a, num_sms, s);
    if (op == LD_BACKWARD)
        return tail ? launch<T, LD_BACKWARD, true>(a, num_sms, s) : launch<T, LD_BACKWARD, false>(a, num_sms, s);
    return tail ? launch<T, LD_STEP, true>(a, num_sms, s) : launch<T, LD_STEP, false>(a, num_sms, s);
}

template <typename T, int OP, bool TAIL, bool HOLD> cudaError_t set_smem()
{
    cudaError_t e = cudaFuncSetAttribute(distill_kernel<T, OP, TAIL, HOLD, LD_THREADS>,
                                         cudaFuncAttributeMaxDynamicSharedMemorySize, LD_SMEM);
    if (HOLD && e == cudaSuccess)
        e = cudaFuncSetAttribute(distill_kernel<T, OP, TAIL, HOLD, LD_THREADS / 2>,
                                 cudaFuncAttributeMaxDynamicSharedMemorySize, LD_SMEM);
    return e;
}

template <typename T, bool TAIL> cudaError_t prepare_tail()
{
    for (cudaError_t e : {set_smem<T, LD_FORWARD, TAIL, false>(), set_smem<T, LD_BACKWARD, TAIL, false>(),
                          set_smem<T, LD_STEP, TAIL, false>(), set_smem<T, LD_STEP, TAIL, true>()})
        if (e != cudaSuccess)
            return e;
    return cudaSuccess;
}

template <typename T> cudaError_t prepare()
{
    const cudaError_t e = prepare_tail<T, false>();
    return e != cudaSuccess ? e : prepare_tail<T, true>();
}

} // namespace

cudaError_t distill_topk_launch(DistillArgs a, int op, int dtype, int num_sms, cudaStream_t s)
{
    if (dtype == TIM_F32)
        return launch_op<float>(a, op, num_sms, s);
    if (dtype == TIM_BF16)
        return launch_op<__nv_bfloat16>(a, op, num_sms, s);
    return launch_op<__half>(a, op, num_sms, s);
}

cudaError_t distill_topk_prepare_device()
{
    for (cudaError_t e : {prepare<float>(), prepare<__nv_bfloat16>(), prepare<__half>()})
        if (e != cudaSuccess)
            return e;
    return cudaSuccess;
}

} // namespace tim
