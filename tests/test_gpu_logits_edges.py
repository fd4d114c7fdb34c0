"""Edges of the operators on a head's logits: rows whose probabilities, masks or
lists leave nothing on one side, values at the types' limits, long segments in
place, outputs on other streams."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import logits_ref as ref  # noqa: E402
import rollout_logprob_mismatch_gb300 as tim  # noqa: E402
from test_gpu_logits import assert_close, dev, draw_logits, draw_teacher, rules  # noqa: E402


# ----------------------------------------------------------------------------- the step's waits
@pytest.mark.parametrize("tail", [False, True])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_step_on_clusters_records_no_timeout(dtype, tail):
    """A step whose row is held by a cluster, on shared memory that the call before
    left full of ones and NaN: no wait takes what it finds there for an abort."""
    N, V, K = 40, 40001, 50
    z, _ = draw_logits(N, V, dtype, 6)
    ids, t, tlse = draw_teacher(N, V, K, 6, tail=tail)
    args = (z, dev(ids), dev(t), dev(np.ones(N, np.float32)))
    tl = None if tlse is None else dev(tlse)
    first = tim.distill_topk_step(*args, teacher_lse=tl)
    dirty = torch.full((600, V), float("nan"), dtype=z.dtype, device="cuda")
    many = (args[1].repeat(15, 1), args[2].repeat(15, 1), args[3].repeat(15))
    for _ in range(20):
        tim.distill_topk_step(dirty, *many, teacher_lse=None if tl is None else tl.repeat(15))
        again = tim.distill_topk_step(*args, teacher_lse=tl)
        for k in ("loss", "lse", "dlogits"):
            assert torch.equal(again[k], first[k]), k
    tim.check()


# ----------------------------------------------------------------------------- distillation in fp64
U = 2.0 ** -24
HALF = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8, "f16": 2.0 ** -11}


def lse_of(x):
    """log sum e^x whose gradient keeps log(size) at values that swallow it, in fp64 too."""
    m = x.max().detach()
    return m + torch.logsumexp(x - m, 0) if bool(torch.isfinite(m)) else torch.logsumexp(x, 0)


def distill64(z, ids, t, tlse, tau, g=None):
    """(loss [N], its gradient [N, V] by automatic differentiation, lse, lse_tail) in
    fp64, from the loss's definition; q_o counts as 0 where p_o is 0 in fp32 and
    the rounding of tlse explains it; a row whose list carries nothing has loss 0."""
    N, V = z.shape
    x = torch.from_numpy(z / tau).double().requires_grad_(True)
    loss, lse, lt = [], np.empty(N), np.empty(N)
    for i in range(N):
        on = (ids[i] >= 0) & (ids[i] < V)
        cols = torch.from_numpy(ids[i][on].astype(np.int64))
        tt = torch.from_numpy(t[i][on].astype(np.float64) / tau)
        listed = torch.zeros(V, dtype=torch.bool)
        listed[cols] = True
        L = lse_of(x[i])
        rest = x[i][~listed]
        R = lse_of(rest) if rest.numel() else torch.tensor(-np.inf)
        lse[i], lt[i] = float(L.detach()), float(R.detach())
        if tlse is None:
            logq = tt - torch.logsumexp(tt, 0) if (tt > -np.inf).any() else torch.full_like(tt, -np.inf)
        else:
            logq = tt - float(tlse[i])
        q = torch.exp(logq)
        some = q > 0
        total = torch.sum(q[some] * (logq[some] - (x[i][cols[some]] - L))) if some.any() else x[i, 0] * 0
        if tlse is not None:
            qo = max(0.0, 1.0 - float(q.sum()))
            if lt[i] - lse[i] < -126 * np.log(2.0) and qo <= 2.0 ** -22 * (16 + abs(float(tlse[i]))):
                qo = 0.0
            if qo > 0:
                total = total + qo * (np.log(qo) - (R - L))
        loss.append(total)
    loss = torch.stack(loss)
    grad = None
    if g is not None:
        (grad,) = torch.autograd.grad((loss * torch.from_numpy(g).double()).sum(), x)
        grad = grad.numpy() / tau
    return loss.detach().numpy(), grad, lse, lt


def far_tolerance(z, ids, t, tlse, tau, g, dtype, lse, lt, from_lse):
    """What the gradient may be off by.  Listed ids: p and q as in logits_ref.  The
    others are p_o r - q_o r, r = e^(y - lse_tail) <= 1 the student's distribution over
    them: r's exponent carries 8 u of its terms (their spread in a step, the terms
    themselves where lse_tail is given in fp32), p_o = e^(lse_tail - lse) and q_o their own."""
    N, V = z.shape
    tol = np.empty((N, V))
    y = z / tau
    for i in range(N):
        on = (ids[i] >= 0) & (ids[i] < V)
        logq = t[i][on].astype(np.float64) / tau - float(tlse[i])
        q = np.exp(logq)
        qo = max(0.0, 1.0 - q.sum())
        T = np.abs(logq).max() + abs(float(tlse[i]))
        listed = np.zeros(V, bool)
        listed[ids[i][on]] = True
        qv = np.zeros(V)
        np.add.at(qv, ids[i][on], q)
        p = np.exp(y[i] - lse[i])
        near = U * (8 * (np.abs(y[i][listed]).max() + abs(lse[i])) + 96)
        po = np.exp(lt[i] - lse[i])
        top = y[i][~listed].max()
        r = np.exp(y[i] - top, where=~listed, out=np.zeros(V))
        r /= r.sum()
        spread = np.abs(y[i]) + abs(lt[i]) if from_lse else np.abs(y[i] - top)
        with np.errstate(over="ignore"):
            dr = np.minimum(1.0, r * np.expm1(np.minimum(700.0, U * (8 * spread + 96))))
            dpo = min(1.0, po * np.expm1(min(700.0, U * (8 * (abs(lt[i]) + abs(lse[i])) + 96))))
        qerr = q.sum() * U * (8 * T + 32) + 8 * U
        rest = (po + qo) * dr + (r + dr) * (dpo + qerr)
        tol[i] = np.where(listed, p * near + qv * U * (8 * T + 32) + 2 * U * (p + qv), rest)
    return tol * np.abs(g)[:, None] / tau


# ----------------------------------------------------------------------------- a small p_o
@pytest.mark.parametrize("tau", [1.0, 0.125])
@pytest.mark.parametrize("dtype,gap", [("f32", 20.0), ("f32", 100.0), ("f32", 1e4), ("f32", None), ("bf16", 100.0),
                                       ("bf16", None), ("f16", 1e4), ("f16", None)])
@pytest.mark.parametrize("V", [300, 5001, 40001])
def test_tail_gradient_of_students_that_all_but_rule_out_the_rest(V, dtype, gap, tau):
    """Unlisted logits far below the listed ones (gap None: the type's lowest value, as
    an additive mask writes it): p_o is small or 0 in fp32, and the others' gradient
    g (p_v - q_o e^(z_v / tau - lse_tail)) / tau stays finite and right, with a teacher
    that has a rest and one that has none."""
    N, K = 4, 12
    rng = np.random.default_rng(V)
    z, _ = draw_logits(N, V, dtype, V + 1, std=1.0)
    ids = np.stack([rng.choice(V, K, replace=False) for _ in range(N)]).astype(np.int32)
    on = torch.zeros(N, V, dtype=torch.bool, device="cuda").scatter_(1, dev(ids).long(), True)
    if gap is None:
        z = torch.where(on, z, torch.full_like(z, torch.finfo(z.dtype).min))
    else:
        z = torch.where(on, z, z - gap)
    z64 = z.double().cpu().numpy()
    t = rng.normal(0, 1, (N, K)).astype(np.float32)
    mass = np.log(np.exp(t.astype(np.float64) / tau).sum(1))
    rest = np.array([0.25, 1e-3, 0.0, 0.0])
    tlse = (mass - np.log1p(-rest) - np.array([0, 0, 1e-3, 1e-3])).astype(np.float32)   # rows 2, 3: sum q above 1
    g = np.array([1.0, -0.5, 2.0, 1.0], np.float32)
    with np.errstate(over="ignore", invalid="ignore"):
        loss, grad, lse, lt = distill64(z64, ids, t, tlse, tau, g)
        # a step knows sum q_k only as 1 where no rest is left: its listed term is p_v - q_v
        sumq = np.exp(t.astype(np.float64) / tau - tlse.astype(np.float64)[:, None]).sum(1)
        over = np.maximum(sumq - 1.0, 0.0)
        p = np.exp(z64 / tau - lse[:, None])
        grad = grad - (g * over / tau)[:, None] * p
        tol = far_tolerance(z64, ids, t, tlse, tau, g, dtype, lse, lt, False)
    least = 2.0 ** -25 if dtype == "f16" else 2.0 ** -126        # half of fp16's smallest step
    tol = tol + HALF[dtype] * np.abs(grad) + least
    args, tl = (dev(ids), dev(t)), dev(tlse)
    s = tim.distill_topk_step(z, *args, dev(g), teacher_lse=tl, temperature=tau)
    f = tim.distill_topk(z, *args, teacher_lse=tl, temperature=tau)
    b = tim.distill_topk_backward(z, *args, dev(g), f["lse"], f["lse_tail"], teacher_lse=tl, temperature=tau)
    tim.check()
    d = s["dlogits"].double().cpu().numpy()
    assert np.isfinite(d).all(), "step"
    assert (np.abs(d - grad) <= tol).all(), ("step", (np.abs(d - grad) - tol).max())
    with np.errstate(over="ignore", invalid="ignore"):
        tol = far_tolerance(z64, ids, t, tlse, tau, g, dtype, lse, lt, True)
    tol = tol + HALF[dtype] * np.abs(grad) + least
    d = b.double().cpu().numpy()
    assert np.isfinite(d).all(), "backward"
    assert (np.abs(d - grad) <= tol).all(), ("backward", (np.abs(d - grad) - tol).max())
    assert torch.equal(s["loss"], f["loss"])
    if np.abs(lt).max() < 3e38:                       # (else z / tau itself passes fp32's range)
        q = np.exp(t.astype(np.float64) / tau - tlse.astype(np.float64)[:, None])
        T = np.abs(t / tau).max() + 2 * np.abs(tlse).max()
        Y = np.abs(z64[on.cpu().numpy()]).max() / tau
        qo = np.maximum(0.0, 1.0 - q.sum(1))
        d = np.log(np.maximum(qo, 2.0 ** -24)) - (lt - lse)
        qerr = (q.sum(1) * U * (8 * T + 32) + 8 * U) * (qo > 0)
        ltol = U * (8 * (T + Y) + 200) * (30 + np.abs(loss)) + qerr * (np.abs(d) + 1)
        assert (np.abs(s["loss"].double().cpu().numpy() - loss) <= ltol).all()


# ----------------------------------------------------------------------------- lists that carry nothing
@pytest.mark.parametrize("V,K", [(7, 3), (3000, 40), (40001, 64)])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_rows_whose_listed_logits_are_all_minus_infinity(V, K, dtype):
    """Valid ids with the teacher's logits all -inf (a list padded with an id and -inf)
    and no teacher_lse: the loss is 0 whatever the student says, and so is its gradient,
    also where the student has an infinity or a NaN."""
    N = 5
    z, _ = draw_logits(N, V, dtype, V)
    rng = np.random.default_rng(V)
    ids = np.stack([rng.choice(V, K, replace=False) for _ in range(N)]).astype(np.int32)
    t = rng.normal(0, 1, (N, K)).astype(np.float32)
    t[1] = -np.inf
    ids[2], t[2] = 0, -np.inf            # padding alone: id 0 and -inf, K times
    t[3, 1:] = -np.inf                   # one that carries all
    t[4], ids[4, :] = -np.inf, -1        # an empty list
    z[1, 0] = float("nan")
    z[4, 1] = float("inf")
    g = np.ones(N, np.float32)
    use = [0, 3]
    z64 = z.double().cpu().numpy()
    loss, grad, lse, _ = distill64(z64[use], ids[use], t[use], None, 1.0, g[use])
    args = (dev(ids), dev(t))
    s = tim.distill_topk_step(z, *args, dev(g))
    f = tim.distill_topk(z, *args)
    b = tim.distill_topk_backward(z, *args, dev(g), f["lse"])
    z2, z3 = z.clone(), z.clone()
    tim.distill_topk_step(z2, *args, dev(g), dlogits=z2)
    tim.distill_topk_backward(z3, *args, dev(g), f["lse"], dlogits=z3)
    tim.check()
    for name, d in (("step", s["dlogits"]), ("backward", b), ("step in place", z2), ("backward in place", z3)):
        assert bool((d[[1, 2, 4]] == 0).all()), name
        got = d[use].double().cpu().numpy()
        tol = U * (16 * np.abs(z64[use]).max() + 200) + HALF[dtype] * np.abs(grad) + 2.0 ** -126
        assert (np.abs(got - grad) <= tol).all(), name
    assert bool((s["loss"][[1, 2, 4]] == 0).all()) and torch.equal(s["loss"], f["loss"])
    assert (np.abs(s["loss"][use].double().cpu().numpy() - loss) <= U * (16 * np.abs(z64[use]).max() + 200) + U * 16 * (1 + np.abs(loss))).all()


# ----------------------------------------------------------------------------- nothing unlisted is left
@pytest.mark.parametrize("kind,low", [("covering", -np.inf), ("same grammar", -np.inf), ("same grammar, wide", -np.inf),
                                      ("same grammar", -1e4), ("same grammar", -3.4028234663852886e38)])
def test_no_infinite_loss_from_the_rounding_of_teacher_lse(kind, low):
    """A list that holds every id the student gives anything: 1 - sum q_k is what the
    rounding of teacher_lse leaves, some 1e-7, and no outcome.  A q_o that the rounding
    does not explain, on ids the student rules out, makes the loss +inf as it should."""
    N = 400
    V, K = {"covering": (24, 24), "same grammar": (2000, 24), "same grammar, wide": (151936, 300)}[kind]
    z, _ = draw_logits(N, V, "f32", 5)
    rng = np.random.default_rng(K)
    ids = np.stack([rng.choice(V, K, replace=False) for _ in range(N)]).astype(np.int32)
    on = torch.zeros(N, V, dtype=torch.bool, device="cuda").scatter_(1, dev(ids).long(), True)
    z = z.masked_fill(~on, low)
    t = rng.normal(0, 3, (N, K)).astype(np.float32)
    exact = np.log(np.exp(t.astype(np.float64)).sum(1))
    tlse = exact.astype(np.float32)
    tlse[:8] = (exact[:8] + 0.01).astype(np.float32)     # one percent on what the student rules out
    g = np.ones(N, np.float32)
    zl = z.gather(1, dev(ids).long()).double().cpu().numpy()
    where = np.tile(np.arange(K, dtype=np.int32), (N, 1))
    loss, grad, lse, _ = distill64(zl, where, t, tlse, 1.0, g)      # the listed columns are the whole row
    assert (loss[:8] == np.inf).all() and np.isfinite(loss[8:]).all()
    far = np.inf if low == -np.inf else 0.009 * -low      # what the first rows' one percent costs, at least
    tl = dev(tlse)
    s = tim.distill_topk_step(z, dev(ids), dev(t), dev(g), teacher_lse=tl)
    f = tim.distill_topk(z, dev(ids), dev(t), teacher_lse=tl)
    tim.check()
    assert torch.equal(s["loss"], f["loss"]) and bool((s["lse_tail"] < low + 8).all() or low < -1e30)
    b = tim.distill_topk_backward(z, dev(ids), dev(t), dev(g), f["lse"], f["lse_tail"], teacher_lse=tl)
    tim.check()
    got = s["loss"].double().cpu().numpy()
    assert (got[:8] >= far).all()
    assert np.isfinite(got[8:]).all(), int((~np.isfinite(got[8:])).sum())
    logq = t.astype(np.float64) - tlse.astype(np.float64)[:, None]
    weighed = (np.exp(logq) * np.abs(logq - (zl - lse[:, None]))).sum(1)
    tol = U * (8 * (np.abs(zl).max() + np.abs(t).max() + 2 * np.abs(tlse).max()) + 200) * (2 + weighed[8:])
    assert (np.abs(got[8:] - loss[8:]) <= tol).all()
    # p_v - q_v: the fp64 gradient scales p by sum q_k, which the rounding of tlse keeps near 1
    dtol = U * (16 * (np.abs(zl).max() + np.abs(tlse).max()) + 200)
    for d in (s["dlogits"], b):
        at = d.gather(1, dev(ids).long()).double().cpu().numpy()
        assert (np.abs(at - grad)[8:] <= dtol).all()
        assert bool((d.masked_fill(on, 0)[8:] == 0).all()) and bool(torch.isfinite(d).all())


# ----------------------------------------------------------------------------- probabilities from a rounded lse
@pytest.mark.parametrize("tau", [0.7, 1.0, 1.3, 3.0])
@pytest.mark.parametrize("dtype,low", [("f32", -1e9), ("f32", None), ("bf16", -1e9), ("bf16", None), ("f16", None)])
def test_gradients_of_rows_at_the_lowest_values_stay_bounded(dtype, low, tau):
    """Rows whose every logit is an additive mask's value: lse's rounding in fp32 is
    larger than log V, so e^(y - lse) says little there, but it is a probability: a
    gradient is at most |g| times its slope."""
    N, V = 5, 3001
    low = torch.finfo({"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}[dtype]).min if low is None else low
    z, _ = draw_logits(N, V, dtype, 2)
    z[1:] = low
    z[2, 7] = low / 2
    z[4, 9] = float("nan")
    hist = np.array([3, 4, 5, 5], np.int32)
    r = tim.LogitsRules(temperature=dev(np.full(N, tau, np.float32)), repetition=dev(np.full(N, 1.0, np.float32)),
                        history=dev(hist), history_spans=dev(np.tile([0, 1, 4], (N, 1)).astype(np.int32)))
    for R in (r, tim.LogitsRules(temperature=r.temperature)):
        for target in (5, 100):
            a = dev(np.full(N, target, np.int32))
            lp, lse = tim.processed_logprob(z, R, a)
            g = np.linspace(1, 2, N).astype(np.float32)
            d = tim.processed_logprob_backward(z, R, a, dev(g), lse).double().cpu().numpy()
            limit = g / tau * (1 + 2 * HALF[dtype])
            assert np.isfinite(d[:4]).all() and (np.abs(d[:4]).max(1) <= limit[:4]).all(), np.abs(d[:4]).max(1)
            # (a column whose y is -inf has gradient 0, in a row that holds a NaN too)
            some = torch.isfinite(tim.process_logits(z, R, out_dtype=torch.float32)[4]).cpu().numpy()
            assert np.isnan(d[4][some]).all() and torch.isnan(lse[4])
    ids = np.tile(np.array([1, 2, 3, 4, 5, 6, 7, 8], np.int32), (N, 1))
    t = np.random.default_rng(1).normal(0, 1, ids.shape).astype(np.float32)
    tlse = (np.log(np.exp(t.astype(np.float64) / tau).sum(1)) + 0.1).astype(np.float32)
    for tl in (None, dev(tlse)):
        f = tim.distill_topk(z, dev(ids), dev(t), teacher_lse=tl, temperature=tau)
        b = tim.distill_topk_backward(z, dev(ids), dev(t), dev(g), f["lse"], f["lse_tail"], teacher_lse=tl, temperature=tau)
        d = b.double().cpu().numpy()
        assert np.isfinite(d[:4]).all() and (np.abs(d[:4]).max(1) <= limit[:4]).all(), np.abs(d[:4]).max(1)
        assert np.isnan(d[4]).all()
    tim.check()


# ----------------------------------------------------------------------------- one quotient for all columns
@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
def test_processed_logits_are_one_rounding_from_the_quotient(dtype):
    """Without penalties y = z / temperature is off by half a unit in the last place of
    fp32 (and 2^-20 of one: the quotient's correction), and a column that is in the
    history with neutral parameters has the bits of one that is not."""
    N, V = 64, 4099
    z, z64 = draw_logits(N, V, dtype, 12, std=4.0)
    rng = np.random.default_rng(8)
    tau = rng.uniform(0.3, 2.5, N).astype(np.float32)
    z[:, 0], z[:, 1], z[:, 2], z[:, 3] = float("inf"), -float("inf"), 0.0, torch.finfo(z.dtype).min
    z64 = z.double().cpu().numpy()
    one = dev(np.ones(N, np.float32))
    R = tim.LogitsRules(temperature=dev(tau))
    y = tim.process_logits(z, R, out_dtype=torch.float32)
    hist = dev(np.arange(0, V, 2, dtype=np.int32))
    spans = dev(np.tile([0, hist.shape[0] // 2, hist.shape[0]], (N, 1)).astype(np.int32))
    neutral = tim.LogitsRules(temperature=dev(tau), repetition=one, presence=one * 0, frequency=one * 0, history=hist,
                              history_spans=spans)
    assert torch.equal(tim.process_logits(z, neutral, out_dtype=torch.float32), y)
    if dtype != "f32":
        assert torch.equal(tim.process_logits(z, neutral), tim.process_logits(z, R))
    tim.check()
    want = z64 / tau[:, None].astype(np.float64)
    got = y.double().cpu().numpy()
    inside = np.abs(want) < 3.4e38
    with np.errstate(over="ignore"):
        want32 = want.astype(np.float32)
    ulp = np.spacing(np.abs(want32)).astype(np.float64)
    off = np.abs(np.where(inside, got, 0.0) - np.where(inside, want, 0.0))
    assert (off[inside] <= 0.5 * (1 + 2.0 ** -19) * ulp[inside]).all(), (off[inside] / ulp[inside]).max()
    assert (got[:, 0] == np.inf).all() and (got[:, 1] == -np.inf).all()
    past = np.abs(want) > 3.41e38
    assert (got[past] == want32[past]).all()


# ----------------------------------------------------------------------------- interleaved rows
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_outputs_between_the_rows_of_the_logits(dtype):
    """Logits and output as the halves of one [N, 2, V] buffer: no element is shared, so
    the call runs; halves that share a column are refused."""
    N, V = 9, 1003
    DT = {"f32": torch.float32, "bf16": torch.bfloat16}[dtype]
    buf = torch.zeros(N, 2, V, dtype=DT, device="cuda")
    z, _ = draw_logits(N, V, dtype, 3)
    buf[:, 0] = z
    R = tim.LogitsRules(temperature=dev(np.full(N, 0.8, np.float32)))
    t = dev(np.arange(N, dtype=np.int32))
    g = dev(np.ones(N, np.float32))
    want = tim.process_logits(z, R)
    tim.process_logits(buf[:, 0], R, out=buf[:, 1])
    assert torch.equal(buf[:, 1], want) and torch.equal(buf[:, 0], z)
    lse = tim.processed_logprob(z, R, t)[1]
    tim.processed_logprob_backward(buf[:, 0], R, t, g, lse, dlogits=buf[:, 1])
    assert torch.equal(buf[:, 1], tim.processed_logprob_backward(z, R, t, g, lse)) and torch.equal(buf[:, 0], z)
    buf[:, 1] = z
    tim.process_logits(buf[:, 1], R, out=buf[:, 0])      # the output before the logits
    assert torch.equal(buf[:, 0], want) and torch.equal(buf[:, 1], z)
    flat = torch.zeros(N, 2 * V, dtype=DT, device="cuda")
    for a, b in ((flat[:, :V], flat[:, V - 1:2 * V - 1]), (flat[:, V:], flat[:, 1:V + 1]),
                 (flat[1:, :V], flat.view(-1)[V:V + (N - 1) * 2 * V].view(N - 1, 2 * V)[:, 1:V + 1])):
        with pytest.raises(tim.TimError):
            tim.process_logits(a, R if a.shape[0] == N else None, out=b)
    tim.check()


# ----------------------------------------------------------------------------- outputs on other streams
def test_outputs_of_another_stream_are_not_handed_to_the_current_one():
    """Every output a call allocates for another stream comes from that stream's memory:
    after it is dropped an allocation of its size on the current stream is another
    block.  A block of the current stream is handed out again at once (the control that
    makes this test able to fail)."""
    side = torch.cuda.Stream()

    def handed_out(holder):
        """The output in `holder` dropped: is its block what the current stream gets next?"""
        x = holder.pop()
        shape, dtype, at = x.shape, x.dtype, x.data_ptr()
        held = [torch.empty(shape, dtype=dtype, device="cuda") for _ in range(20)]   # whatever else is free
        del x
        new = torch.empty(shape, dtype=dtype, device="cuda")
        del held
        return new.data_ptr() == at

    def check(N, V, calls):
        # (every output is above 10 MB: a block of its own)
        z = torch.randn(N, V, device="cuda")
        t = torch.zeros(N, dtype=torch.int32, device="cuda")
        f = torch.ones(N, device="cuda")
        lse = torch.logsumexp(z, 1)
        args = (z, t.view(N, 1), f.view(N, 1))
        torch.cuda.synchronize()
        for call in calls:
            holder = [call(z, t, f, lse, args, None)]
            torch.cuda.synchronize()
            assert handed_out(holder), "the control: a block of the current stream"
            holder = [call(z, t, f, lse, args, side)]
            side.synchronize()
            assert not handed_out(holder)

    check(3 << 20, 2, [lambda z, t, f, lse, a, s: tim.processed_logprob(z, None, t, stream=s)[0],
                       lambda z, t, f, lse, a, s: tim.processed_logprob(z, None, t, stream=s)[1],
                       lambda z, t, f, lse, a, s: tim.distill_topk(*a, stream=s)["loss"],
                       lambda z, t, f, lse, a, s: tim.distill_topk(*a, stream=s)["lse"],
                       lambda z, t, f, lse, a, s: tim.distill_topk(*a, teacher_lse=lse, stream=s)["lse_tail"]])
    check(64, 151936, [lambda z, t, f, lse, a, s: tim.process_logits(z, None, stream=s),
                       lambda z, t, f, lse, a, s: tim.processed_logprob_backward(z, None, t, f, lse, stream=s),
                       lambda z, t, f, lse, a, s: tim.distill_topk_backward(*a, f, lse, stream=s),
                       lambda z, t, f, lse, a, s: tim.distill_topk_step(*a, f, stream=s)["dlogits"]])
    tim.check()


# ----------------------------------------------------------------------------- long segments
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_long_segments_in_place_and_not(dtype):
    """A batch large enough that a CTA has some fifty slices of a row: rows whose table
    half of the CTA builds, whose table is full under half and under all of it, and
    rows without history, out of place, in place, and each against fp64."""
    N, V = 300, 151936
    z, z64 = draw_logits(N, V, dtype, 41)
    rng = np.random.default_rng(17)
    # tokens of rows: none, few, 4000 distinct ones in the row's first third, 9000 anywhere,
    # 9000 in the first third, 5000 of few ids
    parts = [np.zeros(0), rng.integers(0, V, 60), rng.permutation(40000)[:4000], rng.integers(0, V, 9000),
             rng.permutation(45000)[:9000], rng.integers(0, V, 200)[rng.integers(0, 200, 5000)]]
    start = np.concatenate([[0], np.cumsum([p.size for p in parts])])
    kind = np.arange(N) % len(parts)
    spans = np.stack([start[kind], start[kind] + (start[kind + 1] - start[kind]) // 3, start[kind + 1]], 1)
    r = {"history": np.concatenate(parts).astype(np.int32), "history_spans": spans.astype(np.int32),
         "repetition": rng.choice([1.0, 1.2, 0.9], N).astype(np.float32), "presence": np.full(N, 0.3, np.float32),
         "frequency": np.full(N, 0.1, np.float32), "temperature": rng.uniform(0.6, 1.4, N).astype(np.float32),
         "bias_offsets": (np.arange(N + 1) * 5).astype(np.int32), "bias_values": rng.normal(0, 2, 5 * N).astype(np.float32),
         "bias_ids": np.concatenate([np.sort(rng.choice(V, 5, replace=False)) for _ in range(N)]).astype(np.int32),
         "allowed": rng.integers(-2 ** 31, 2 ** 31, (2, (V + 31) // 32)).astype(np.int32),
         "allowed_rows": rng.integers(-1, 2, N).astype(np.int32)}
    R = rules(r)
    rows = np.r_[0:6, 150:156, N - 6:N]
    sub = {k: (v[rows] if k in ("history_spans", "repetition", "presence", "frequency", "temperature", "allowed_rows") else v)
           for k, v in r.items()}
    sub["bias_offsets"] = (np.arange(rows.size + 1) * 5).astype(np.int32)
    sub["bias_ids"] = r["bias_ids"].reshape(N, 5)[rows].reshape(-1)
    sub["bias_values"] = r["bias_values"].reshape(N, 5)[rows].reshape(-1)
    y = tim.process_logits(z, R)
    want, tol = ref.process_ref(z64[rows], sub, dtype)
    assert_close(y[rows], want, tol, "process")
    z2 = z.clone()
    assert torch.equal(tim.process_logits(z2, R, out=z2), y), "process in place"
    t = rng.integers(0, V, N).astype(np.int32)
    t[::2] = r["history"][spans[::2, 1] % r["history"].size]
    lp, lse = tim.processed_logprob(z, R, dev(t))
    wlp, wlse, ltol = ref.logprob_ref(z64[rows], sub, t[rows])
    assert_close(lp[rows], wlp, ltol, "logp")
    assert_close(lse[rows], wlse, ltol, "lse")
    g = rng.normal(0, 1, N).astype(np.float32)
    d = tim.processed_logprob_backward(z, R, dev(t), dev(g), lse)
    want, tol = ref.backward_ref(z64[rows], sub, t[rows], g[rows], lse.cpu().numpy()[rows], dtype)
    assert_close(d[rows], want, tol, "gradient")
    z2 = z.clone()
    assert torch.equal(tim.processed_logprob_backward(z2, R, dev(t), dev(g), lse, dlogits=z2), d), "gradient in place"
    tim.check()
