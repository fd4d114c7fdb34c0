"""GPU parity of the operators on a head's logits against their fp64 formulas:
processing, the processed log-probability and its gradient, distillation from
top logits; odd sizes, strides, types, histories, masks that leave nothing,
infinities, row invariance, refusals."""
import dataclasses

import numpy as np
import pytest

import logits_ref as ref

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import rollout_logprob_mismatch_gb300 as tim  # noqa: E402

DT = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
INF = np.inf


def dev(x):
    return torch.from_numpy(np.ascontiguousarray(x)).cuda()


def draw_logits(N, V, dtype, seed, std=3.0, stride=None, offset=0):
    """(device tensor [N, V], its values in fp64): rows `stride` apart, starting
    `offset` elements into a buffer."""
    rng = np.random.default_rng(seed)
    stride = V if stride is None else stride
    buf = torch.from_numpy(rng.normal(0, std, offset + N * stride).astype(np.float32)).to(DT[dtype]).cuda()
    z = buf[offset:].as_strided((N, V), (stride, 1), buf.storage_offset() + offset)
    return z, z.double().cpu().numpy()


def draw_rules(N, V, seed, hist=40, bias=3, masked=0.5, which="all"):
    rng = np.random.default_rng([seed, 7])
    r = {}
    if which in ("all", "temperature"):
        r["temperature"] = rng.uniform(0.5, 1.6, N).astype(np.float32)
    if which in ("all", "history"):
        r["repetition"] = rng.choice([1.0, 1.1, 1.5, 0.8], N).astype(np.float32)
        r["presence"] = rng.choice([0.0, 0.7, -0.4], N).astype(np.float32)
        r["frequency"] = rng.choice([0.0, 0.2, -0.1], N).astype(np.float32)
        lens = rng.integers(0, hist + 1, N)
        lens[0] = 0
        lens[-1] = hist
        H = int(lens.sum()) + 5
        r["history"] = (rng.random(H) ** 3 * V).astype(np.int32)
        r["history"][rng.random(H) < 0.05] = -1
        r["history"][rng.random(H) < 0.02] = V
        b = np.concatenate([[0], np.cumsum(lens)[:-1]])
        r["history_spans"] = np.stack([b, b + rng.integers(0, lens + 1), b + lens], 1).astype(np.int32)
    if which in ("all", "bias"):
        k = min(bias, V)
        n = np.where(rng.random(N) < 0.7, k, 0)
        r["bias_offsets"] = np.concatenate([[0], np.cumsum(n)]).astype(np.int32)
        ids = [np.sort(rng.choice(V, k, replace=False)) for c in n if c]
        r["bias_ids"] = np.concatenate(ids + [np.zeros(0)]).astype(np.int32)
        r["bias_values"] = rng.uniform(-5, 5, r["bias_ids"].size).astype(np.float32)
        if r["bias_values"].size:
            r["bias_values"][0] = -INF
    if which in ("all", "mask"):
        R = max(1, int(N * masked))
        words = (V + 31) // 32
        r["allowed"] = rng.integers(-2 ** 31, 2 ** 31, (R, words + 1)).astype(np.int32)
        if R > 1:
            r["allowed"][-1] = 0                    # nothing is left
        r["allowed_rows"] = rng.integers(-1, R, N).astype(np.int32)
        r["allowed_rows"][-1] = R - 1
    return r


def rules(r):
    return tim.LogitsRules(**{k: dev(v) for k, v in r.items()})


def assert_close(got, want, tol, what=""):
    g = got.double().cpu().numpy() if isinstance(got, torch.Tensor) else got
    assert g.shape == want.shape, (what, g.shape, want.shape)
    bad = np.isnan(g) != np.isnan(want)
    bad |= (np.isinf(g) | np.isinf(want)) & (g != want)
    with np.errstate(invalid="ignore"):
        bad |= np.isfinite(g) & np.isfinite(want) & ~(np.abs(g - want) <= tol)
    if bad.any():
        i = np.unravel_index(int(np.argmax(bad)), bad.shape)
        raise AssertionError("%s: %d of %d off, first at %s: got %r want %r tol %r"
                             % (what, int(bad.sum()), bad.size, i, g[i], want[i], np.broadcast_to(tol, bad.shape)[i]))


# (N, V, stride, offset): one column, odd rows, slices that end inside, several segments
SHAPES = [(1, 1, 1, 0), (3, 7, 7, 0), (5, 33, 40, 1), (2, 1023, 1023, 0), (4, 1024, 1024, 0), (3, 1025, 1028, 3),
          (2, 4097, 4099, 5), (7, 5000, 5000, 0), (2, 16384, 16384, 0), (3, 16391, 16400, 8), (1, 40001, 40001, 0),
          (2, 151936, 151936, 0)]


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("N,V,stride,offset", SHAPES)
def test_process_shapes(N, V, stride, offset, dtype):
    z, z64 = draw_logits(N, V, dtype, V + N, stride=stride, offset=offset)
    r = draw_rules(N, V, V)
    for out_dtype in {dtype, "f32"}:
        want, tol = ref.process_ref(z64, r, out_dtype)
        got = tim.process_logits(z, rules(r), out_dtype=DT[out_dtype])
        tim.check()
        assert_close(got, want, tol, "%s -> %s" % (dtype, out_dtype))


@pytest.mark.parametrize("which", ["none", "temperature", "history", "bias", "mask", "all"])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_process_rules_and_in_place(which, dtype):
    """Each rule alone, outputs written over the logits and into a strided view."""
    N, V = 6, 3001
    z, z64 = draw_logits(N, V, dtype, 5, stride=3010, offset=2)
    r = draw_rules(N, V, 3, which=which)
    want, tol = ref.process_ref(z64, r, dtype)
    R = None if which == "none" else rules(r)
    buf = torch.full((N, 3020), 7.0, dtype=DT[dtype], device="cuda")
    tim.process_logits(z, R, out=buf[:, 3:3 + V])
    tim.check()
    assert_close(buf[:, 3:3 + V], want, tol, "strided")
    assert bool((buf[:, :3] == 7).all()) and bool((buf[:, 3 + V:] == 7).all())
    tim.process_logits(z, R, out=z)
    tim.check()
    assert_close(z, want, tol, "in place")


@pytest.mark.parametrize("hist", [1, 511, 513, 5000, 40000])
def test_long_histories(hist):
    """Histories of every length against the scan's strides, ids repeated often."""
    N, V = 3, 20011
    z, z64 = draw_logits(N, V, "bf16", hist)
    r = draw_rules(N, V, hist, hist=hist, bias=100)
    want, tol = ref.process_ref(z64, r, "f32")
    assert_close(tim.process_logits(z, rules(r), out_dtype=torch.float32), want, tol)
    t = np.arange(N, dtype=np.int32) * 777
    lp, lse, ltol = ref.logprob_ref(z64, r, t)
    g_lp, g_lse = tim.processed_logprob(z, rules(r), dev(t))
    tim.check()
    assert_close(g_lse, lse, ltol, "lse")
    assert_close(g_lp, lp, ltol, "logp")


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("N,V,stride,offset", SHAPES)
def test_logprob_and_gradient_shapes(N, V, stride, offset, dtype):
    z, z64 = draw_logits(N, V, dtype, 3 * V + N, stride=stride, offset=offset)
    r = draw_rules(N, V, 11 * V)
    rng = np.random.default_rng(V)
    t = rng.integers(0, V, N).astype(np.int32)
    if N > 2:
        t[1] = -100
        t[2] = V
    R = rules(r)
    lp, lse, tol = ref.logprob_ref(z64, r, t)
    g_lp, g_lse = tim.processed_logprob(z, R, dev(t))
    tim.check()
    assert_close(g_lse, lse, tol, "lse")
    assert_close(g_lp, lp, tol, "logp")
    g = rng.normal(0, 1, N).astype(np.float32)
    if N > 3:
        g[3] = 0
    want, gtol = ref.backward_ref(z64, r, t, g, g_lse.cpu().numpy(), dtype)
    d = tim.processed_logprob_backward(z, R, dev(t), dev(g), g_lse)
    tim.check()
    assert_close(d, want, gtol, "gradient")
    tim.processed_logprob_backward(z, R, dev(t), dev(g), g_lse, dlogits=z)
    tim.check()
    assert torch.equal(z, d), "gradient in place"


def test_logprob_without_rules_and_with_each():
    N, V = 5, 2500
    z, z64 = draw_logits(N, V, "f32", 1)
    t = np.array([0, 1, 2499, 77, 1024], np.int32)
    for which in ("none", "temperature", "history", "bias", "mask"):
        r = draw_rules(N, V, 2, which=which)
        R = None if which == "none" else rules(r)
        lp, lse, tol = ref.logprob_ref(z64, r, t)
        g_lp, g_lse = tim.processed_logprob(z, R, dev(t))
        assert_close(g_lp, lp, tol, which)
        assert_close(g_lse, lse, tol, which)
        g = np.linspace(-1, 1, N).astype(np.float32)
        want, gtol = ref.backward_ref(z64, r, t, g, g_lse.cpu().numpy(), "f32")
        assert_close(tim.processed_logprob_backward(z, R, dev(t), dev(g), g_lse), want, gtol, which)
    tim.check()


def test_rows_with_nothing_left_and_masked_infinities():
    """NaN, infinities and the type's lowest value in masked places do not count;
    a row whose mask leaves nothing has lse = logp = -inf and gradient 0."""
    N, V = 5, 2049
    for dtype in ("f32", "bf16", "f16"):
        z, _ = draw_logits(N, V, dtype, 9)
        low = torch.finfo(DT[dtype]).min
        z[:, 5], z[:, 6], z[:, 7], z[:, 8] = float("nan"), INF, -INF, low
        z[4, 100] = -INF                                     # an allowed id the model rules out
        ok = np.ones((N, V), bool)
        ok[:, 5:9] = False
        ok[1] = False
        ok[2] = False
        ok[2, 2048] = True                                   # one id left, in the last column
        words = np.zeros((N, 65), np.uint32)
        for i, v in zip(*np.nonzero(ok)):
            words[i, v >> 5] |= np.uint32(1) << np.uint32(v & 31)
        r = {"allowed": words.view(np.int32), "temperature": np.full(N, 0.7, np.float32),
             "history": np.array([5, 6, 7, 8, 9, 9], np.int32), "history_spans": np.tile([0, 2, 6], (N, 1)).astype(np.int32),
             "repetition": np.full(N, 1.2, np.float32), "frequency": np.full(N, 0.3, np.float32)}
        t = np.array([9, 10, 2048, 6, 100], np.int32)
        z64 = z.double().cpu().numpy()
        with np.errstate(invalid="ignore"):
            want, tol = ref.process_ref(z64, r, dtype)
            lp, lse, ltol = ref.logprob_ref(z64, r, t)
        assert_close(tim.process_logits(z, rules(r)), want, np.nan_to_num(tol, nan=0.0, posinf=0.0), dtype)
        g_lp, g_lse = tim.processed_logprob(z, rules(r), dev(t))
        tim.check()
        assert_close(g_lse, lse, ltol, dtype)
        assert_close(g_lp, lp, ltol, dtype)
        assert g_lse[1].item() == -INF and g_lp[1].item() == -INF and g_lp[2].item() == 0.0
        g = np.ones(N, np.float32)
        with np.errstate(invalid="ignore"):
            gw, gtol = ref.backward_ref(z64, r, t, g, g_lse.cpu().numpy(), dtype)
        d = tim.processed_logprob_backward(z, rules(r), dev(t), dev(g), g_lse)
        assert_close(d, gw, np.nan_to_num(gtol, nan=0.0, posinf=0.0), dtype)
        assert bool((d[1] == 0).all()) and d[4, 100].item() == 0.0


def test_allowed_nan_and_inf_make_the_row_nan():
    z, _ = draw_logits(3, 1500, "f32", 2)
    z[0, 1400] = float("nan")
    z[1, 3] = INF
    lp, lse = tim.processed_logprob(z, None, dev(np.array([1, 1, 1], np.int32)))
    assert torch.isnan(lp[:2]).all() and torch.isnan(lse[:2]).all() and torch.isfinite(lse[2])


def test_gradient_against_differences():
    """Central differences of the forward itself, step h: the third derivative of a
    log-sum-exp along one logit is below 0.0963 slope^3."""
    V, h = 37, 2.0 ** -4
    z, z64 = draw_logits(1, V, "f32", 21, std=2.0)
    r1 = draw_rules(1, V, 5, hist=30, masked=1.0)
    r1["allowed"] = np.array([[0x5fff7fff, 0x1f, 0]], np.uint32).view(np.int32)
    r1["allowed_rows"] = np.zeros(1, np.int32)
    t = 4
    base = z.repeat(2 * V, 1)
    eye = torch.eye(V, device="cuda") * h
    pert = base + torch.cat([eye, -eye])
    many = {k: (np.repeat(v, 2 * V, 0) if k in ("temperature", "repetition", "presence", "frequency",
                                                "history_spans", "allowed_rows") else v) for k, v in r1.items()}
    n = r1["bias_offsets"][1]
    many["bias_offsets"] = (np.arange(2 * V + 1) * n).astype(np.int32)
    many["bias_ids"] = np.tile(r1["bias_ids"], 2 * V)
    many["bias_values"] = np.tile(r1["bias_values"], 2 * V)
    lp, lse = tim.processed_logprob(pert, rules(many), dev(np.full(2 * V, t, np.int32)))
    num = ((lp[:V].double() - lp[V:].double()) / (2 * h)).cpu().numpy()
    lp0, lse0 = tim.processed_logprob(z, rules(r1), dev(np.array([t], np.int32)))
    d = tim.processed_logprob_backward(z, rules(r1), dev(np.array([t], np.int32)), dev(np.ones(1, np.float32)), lse0)
    y, slope, a = ref.processed(z64[0], r1, 0)
    # a logit whose processed value bends at 0 within the step has no two-sided difference
    bent = np.abs(z64[0]) <= 2 * h
    if "bias_ids" in r1 and n:
        bent[r1["bias_ids"]] = True
    fwd = ref.U * (8 * (ref.top(y) + 1) + 96)
    tol = 0.0963 * h * h / 6 * slope ** 3 + fwd / h + 1e-6
    got = d[0].double().cpu().numpy()
    assert np.all((np.abs(got - num) <= tol) | bent), np.abs(got - num).max()
    assert (~bent).sum() > V // 2


# ----------------------------------------------------------------------------- distillation
def draw_teacher(N, V, K, seed, holes=True, tail=True):
    rng = np.random.default_rng([seed, 3])
    ids = np.stack([rng.choice(V, K, replace=False) for _ in range(N)]).astype(np.int32)
    if holes and K > 1:
        for i in range(N):
            ids[i, rng.integers(0, K + 1):] = -1 if i % 2 else V
        ids[0] = -1
    t = np.sort(rng.normal(4, 2.5, (N, K)), 1)[:, ::-1].astype(np.float32)
    tlse = None
    if tail:
        m = np.where((ids >= 0) & (ids < V), np.exp(t.astype(np.float64)), 0).sum(1)
        tlse = np.log(np.maximum(m, 1e-3) / (1 - rng.uniform(0.002, 0.4, N))).astype(np.float32)
    return ids, t, tlse


def run_distill(z, ids, t, tlse, tau):
    return tim.distill_topk(z, dev(ids), dev(t), None if tlse is None else dev(tlse), temperature=tau)


DISTILL = [(1, 1, 1, 1, 0), (3, 7, 7, 3, 0), (4, 33, 40, 33, 1), (3, 1025, 1028, 20, 3), (5, 5000, 5000, 64, 0),
           (2, 16391, 16400, 513, 8), (2, 40001, 40001, 1024, 0), (3, 151936, 151936, 100, 0)]


@pytest.mark.parametrize("tail", [False, True])
@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("N,V,stride,K,offset", DISTILL)
def test_distill_shapes(N, V, stride, K, offset, dtype, tail):
    z, z64 = draw_logits(N, V, dtype, V + K, stride=stride, offset=offset)
    tau = float(np.float32(1.0 if V % 2 else 0.7))
    ids, t, tlse = draw_teacher(N, V, K, V, tail=tail)
    if tail and tau != 1.0:
        tlse = np.array([np.log(np.sum(np.exp(t[i].astype(np.float64) / tau)) * 1.1) for i in range(N)], np.float32)
    g = np.random.default_rng(V).normal(0, 1, N).astype(np.float32)
    if N > 2:
        g[1] = 0
    o = run_distill(z, ids, t, tlse, tau)
    tim.check()
    w = ref.distill_ref(z64, ids, t, tlse, tau)
    assert_close(o["lse"], w["lse"], w["lse_tol"], "lse")
    assert_close(o["loss"], w["loss"], w["loss_tol"], "loss")
    if tail:
        assert_close(o["lse_tail"], w["lse_tail"], w["lse_tol"], "lse_tail")
    else:
        assert o["lse_tail"] is None
    given = (o["lse"].cpu().numpy(), o["lse_tail"].cpu().numpy() if tail else None)
    w = ref.distill_ref(z64, ids, t, tlse, tau, g, dtype, given)
    tl = None if tlse is None else dev(tlse)
    d = tim.distill_topk_backward(z, dev(ids), dev(t), dev(g), o["lse"], o["lse_tail"], teacher_lse=tl, temperature=tau)
    tim.check()
    assert_close(d, w["dlogits"], w["dlogits_tol"], "gradient")
    s = tim.distill_topk_step(z, dev(ids), dev(t), dev(g), teacher_lse=tl, temperature=tau)
    tim.check()
    for k in ("loss", "lse") + (("lse_tail",) if tail else ()):
        assert torch.equal(s[k], o[k]), k
    assert_close(s["dlogits"], w["dlogits"], w["dlogits_tol"], "step")
    s2 = tim.distill_topk_step(z.clone(), dev(ids), dev(t), dev(g), teacher_lse=tl, temperature=tau)
    assert torch.equal(s2["dlogits"], s["dlogits"])
    z2 = z.clone()
    tim.distill_topk_backward(z2, dev(ids), dev(t), dev(g), o["lse"], o["lse_tail"], teacher_lse=tl, temperature=tau,
                              dlogits=z2)
    assert torch.equal(z2, d), "backward in place"
    tim.distill_topk_step(z, dev(ids), dev(t), dev(g), teacher_lse=tl, temperature=tau, dlogits=z)
    assert torch.equal(z, s["dlogits"]), "step in place"
    tim.check()


@pytest.mark.parametrize("tail", [False, True])
def test_distill_ids_listed_more_than_once_add_up(tail):
    N, V, K = 4, 3000, 40
    z, z64 = draw_logits(N, V, "f32", 8)
    ids, t, tlse = draw_teacher(N, V, K, 8, holes=False, tail=tail)
    ids[:, 5:12] = ids[:, 4:5]
    ids[2] = 17
    g = np.ones(N, np.float32)
    w = ref.distill_ref(z64, ids, t, tlse, 1.0, g)
    s = tim.distill_topk_step(z, dev(ids), dev(t), dev(g), teacher_lse=None if tlse is None else dev(tlse))
    tim.check()
    assert_close(s["loss"], w["loss"], w["loss_tol"])
    assert_close(s["dlogits"], w["dlogits"], w["dlogits_tol"])


def test_distill_edges():
    """Teachers that put everything on one id, students that give an id nothing,
    a list that covers the vocabulary (no tail is left), rows that list nothing."""
    V = 24
    z, _ = draw_logits(5, V, "f32", 4)
    z[1, 3] = -INF
    z[4] = -INF
    K = V
    ids = np.tile(np.arange(V, dtype=np.int32), (5, 1))
    ids[2] = -1
    t = np.zeros((5, K), np.float32)
    t[0] = -INF
    t[0, 2] = 5.0
    tlse = np.log(np.exp(t.astype(np.float64)).sum(1)).astype(np.float32)
    g = np.ones(5, np.float32)
    z64 = z.double().cpu().numpy()
    for tl in (None, tlse):
        s = tim.distill_topk_step(z, dev(ids), dev(t), dev(g), teacher_lse=None if tl is None else dev(tl))
        tim.check()
        loss = s["loss"].cpu().numpy()
        w = ref.distill_ref(z64[:4], ids[:4], t[:4], None if tl is None else tl[:4], 1.0, g[:4])
        assert loss[1] == INF and loss[4] == INF
        if tl is None:
            assert_close(s["loss"][:4], w["loss"], w["loss_tol"])
            assert loss[2] == 0 and bool((s["dlogits"][2] == 0).all())
            assert_close(s["dlogits"][4], -np.full(V, 1 / V), 8 * ref.U)
        assert_close(s["dlogits"][:2], w["dlogits"][:2], w["dlogits_tol"][:2])
        assert not torch.isnan(s["dlogits"]).any()


def test_distill_gradient_against_differences():
    V, K, h = 41, 9, 2.0 ** -4
    for tail in (False, True):
        z, z64 = draw_logits(1, V, "f32", 31, std=1.5)
        ids, t, tlse = draw_teacher(1, V, K, 31, holes=False, tail=tail)
        eye = torch.eye(V, device="cuda") * h
        pert = z + torch.cat([eye, -eye])
        n = 2 * V
        o = run_distill(pert, np.repeat(ids, n, 0), np.repeat(t, n, 0), None if tlse is None else np.repeat(tlse, n), 1.0)
        num = ((o["loss"][:V].double() - o["loss"][V:].double()) / (2 * h)).cpu().numpy()
        s = tim.distill_topk_step(z, dev(ids), dev(t), dev(np.ones(1, np.float32)),
                                  teacher_lse=None if tlse is None else dev(tlse))
        w = ref.distill_ref(z64, ids, t, tlse, 1.0)
        # the loss is lse minus a q_o multiple of lse_tail and a linear term: two log-sum-exps
        tol = 2 * 0.0963 * h * h / 6 + w["loss_tol"][0] / h + 1e-6
        assert np.abs(s["dlogits"][0].double().cpu().numpy() - num).max() <= tol
    tim.check()


# ----------------------------------------------------------------------------- invariance
@pytest.mark.parametrize("V", [1024, 5003, 151936])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_row_bits_do_not_depend_on_the_batch(V, dtype):
    """A row alone, among others and in another place gives the same bits, however
    many CTAs share it and however its storage is aligned."""
    N = 700 if V < 100000 else 330
    z, _ = draw_logits(N, V, dtype, 77)
    r = draw_rules(N, V, 13, hist=60)
    t = np.random.default_rng(1).integers(0, V, N).astype(np.int32)
    lp, lse = tim.processed_logprob(z, rules(r), dev(t))
    y = tim.process_logits(z, rules(r))
    g = dev(np.ones(N, np.float32))
    d = tim.processed_logprob_backward(z, rules(r), dev(t), g, lse)
    ids, tt, tlse = draw_teacher(N, V, 16, 5)
    o = tim.distill_topk_step(z, dev(ids), dev(tt), g, teacher_lse=dev(tlse))
    again = tim.processed_logprob(z, rules(r), dev(t))
    assert torch.equal(again[0].view(torch.int32), lp.view(torch.int32))
    for rows in ([5], [N - 1, 3, 200]):
        sub = dict(r)
        for k in ("temperature", "repetition", "presence", "frequency", "history_spans", "allowed_rows"):
            sub[k] = r[k][rows]
        o0 = r["bias_offsets"]
        parts = [slice(o0[i], o0[i + 1]) for i in rows]
        sub["bias_offsets"] = np.concatenate([[0], np.cumsum([p.stop - p.start for p in parts])]).astype(np.int32)
        sub["bias_ids"] = np.concatenate([r["bias_ids"][p] for p in parts])
        sub["bias_values"] = np.concatenate([r["bias_values"][p] for p in parts])
        n = len(rows)
        for off, stride in ((0, V), (1, V + 1)):
            buf = torch.empty(off + n * stride, dtype=DT[dtype], device="cuda")
            zs = buf.as_strided((n, V), (stride, 1), off)
            zs.copy_(z[rows])
            lp2, lse2 = tim.processed_logprob(zs, rules(sub), dev(t[rows]))
            assert torch.equal(lp2.view(torch.int32), lp[rows].view(torch.int32))
            assert torch.equal(lse2.view(torch.int32), lse[rows].view(torch.int32))
            assert torch.equal(tim.process_logits(zs, rules(sub)).view(torch.uint8), y[rows].contiguous().view(torch.uint8))
            d2 = tim.processed_logprob_backward(zs, rules(sub), dev(t[rows]), g[:n], lse2)
            assert torch.equal(d2, d[rows])
            o2 = tim.distill_topk_step(zs, dev(ids[rows]), dev(tt[rows]), g[:n], teacher_lse=dev(tlse[rows]))
            for k in ("loss", "lse", "lse_tail", "dlogits"):
                assert torch.equal(o2[k], o[k][rows]), k
    tim.check()


def test_packed_sequences_and_another_stream():
    """packed_spans against a loop; the calls run on the stream they are given."""
    off = np.array([0, 5, 5, 12, 13], np.int32)
    pl = np.array([2, 0, 9, 1], np.int32)
    s = tim.packed_spans(dev(off), dev(pl), 13).cpu().numpy()
    for q in range(4):
        for i in range(off[q], off[q + 1]):
            assert s[i].tolist() == [off[q], min(off[q] + pl[q], i + 1), i + 1]
    V = 4099
    side = torch.cuda.Stream()
    tok = dev((np.arange(13) * 311 % V).astype(np.int32))
    with torch.cuda.stream(side):
        z = torch.randn(13, V, device="cuda")
        R = tim.LogitsRules(history=tok, history_spans=dev(s), repetition=torch.full((13,), 1.3, device="cuda"))
        lp, lse = tim.processed_logprob(z, R, tok)
    side.synchronize()
    r = {"history": tok.cpu().numpy(), "history_spans": s, "repetition": np.full(13, 1.3, np.float32)}
    w, wl, tol = ref.logprob_ref(z.double().cpu().numpy(), r, tok.cpu().numpy())
    assert_close(lp, w, tol)
    assert_close(lse, wl, tol)


# ----------------------------------------------------------------------------- refusals
def test_bad_rows_are_reported_and_nan():
    """Parameters, spans, bias entries and mask rows that break their limits: that
    row is NaN, the others are right, tim_check reports it."""
    N, V = 4, 1500
    z, z64 = draw_logits(N, V, "f32", 6)
    t = np.array([3, 4, 5, 6], np.int32)
    good = draw_rules(N, V, 9, which="all", hist=10)

    def spoil(name, row, value):
        r = {k: v.copy() for k, v in good.items()}
        r[name][row] = value
        return r

    b1 = int(good["bias_offsets"][-1])
    cases = [(spoil("temperature", 2, 0.0), 2), (spoil("temperature", 2, np.nan), 2), (spoil("temperature", 2, INF), 2),
             (spoil("repetition", 2, -1.0), 2), (spoil("presence", 2, INF), 2), (spoil("frequency", 2, np.nan), 2),
             (spoil("history_spans", 2, [0, 5, 3]), 2), (spoil("history_spans", 2, [-1, 0, 3]), 2),
             (spoil("history_spans", 2, [0, 0, good["history"].size + 1]), 2), (spoil("allowed_rows", 2, 1000), 2)]
    unsorted = {k: v.copy() for k, v in good.items()}
    unsorted["bias_offsets"] = np.array([0, 0, 0, 2, 2], np.int32)
    unsorted["bias_ids"], unsorted["bias_values"] = np.array([9, 9], np.int32), np.ones(2, np.float32)
    outside = {k: v.copy() for k, v in unsorted.items()}
    outside["bias_ids"] = np.array([9, V], np.int32)
    crossed = {k: v.copy() for k, v in good.items()}
    crossed["bias_offsets"] = np.array([0, 0, 0, b1 + 1, b1], np.int32)
    cases += [(unsorted, 2), (outside, 2)]
    for r, row in cases:
        y = tim.process_logits(z, rules(r))
        with pytest.raises(tim.TimError) as e:
            tim.check()
        assert e.value.code == tim.TIM_ERR_BAD_INPUT
        lp, lse = tim.processed_logprob(z, rules(r), dev(t))
        d = tim.processed_logprob_backward(z, rules(r), dev(t), dev(np.ones(N, np.float32)), lse.nan_to_num(nan=0.0))
        with pytest.raises(tim.TimError):
            tim.check()
        assert torch.isnan(y[row]).all() and torch.isnan(lp[row]) and torch.isnan(lse[row]) and torch.isnan(d[row]).all()
        rest = [i for i in range(N) if i != row]
        assert not torch.isnan(y[rest]).any() and not torch.isnan(lse[rest]).any()
    y = tim.process_logits(z, rules(crossed))
    with pytest.raises(tim.TimError):
        tim.check()
    assert torch.isnan(y[2:]).all()


def test_checked_build_records_targets_and_gradients():
    """libtim_debug.so: a target past the vocabulary and a non-finite upstream
    gradient are recorded, clean calls are not, and the bits are the release build's."""
    N, V = 3, 1200
    z, _ = draw_logits(N, V, "f32", 6)
    t, g = np.array([1, 2, 3], np.int32), np.ones(N, np.float32)
    R = rules(draw_rules(N, V, 3))
    ids, tt, tlse = draw_teacher(N, V, 9, 2)
    lp, lse = tim.processed_logprob(z, R, dev(t))
    s = tim.distill_topk_step(z, dev(ids), dev(tt), dev(g), teacher_lse=dev(tlse))
    with tim.checked():
        lp2, lse2 = tim.processed_logprob(z, R, dev(t))
        s2 = tim.distill_topk_step(z, dev(ids), dev(tt), dev(g), teacher_lse=dev(tlse))
        tim.check()
        assert torch.equal(lp, lp2) and torch.equal(lse, lse2)
        assert all(torch.equal(s[k], s2[k]) for k in s)
        tim.processed_logprob(z, R, dev(np.array([1, V, -100], np.int32)))
        assert tim.tim_debug_violation() == ("target", 1, V)
        tim.processed_logprob_backward(z, R, dev(t), dev(np.array([1, 1, np.nan], np.float32)), lse)
        assert tim.tim_debug_violation()[:2] == ("backward_input", 2)
        tim.distill_topk_step(z, dev(ids), dev(tt), dev(np.array([1, np.inf, 1], np.float32)))
        assert tim.tim_debug_violation()[:2] == ("backward_input", 1)
        with pytest.raises(tim.TimError):
            tim.check()
    tim.check()


def test_wrapper_refusals():
    z = torch.zeros(4, 100, device="cuda")
    t = torch.zeros(4, dtype=torch.int32, device="cuda")
    f = torch.ones(4, device="cuda")
    L = tim.LogitsRules
    bad = [
        (TypeError, lambda: tim.process_logits(z.double(), None)),
        (ValueError, lambda: tim.process_logits(z.cpu(), None)),
        (ValueError, lambda: tim.process_logits(z[0], None)),
        (ValueError, lambda: tim.process_logits(z.t(), None)),
        (ValueError, lambda: tim.process_logits(z[:1].expand(4, 100), None)),
        (TypeError, lambda: tim.process_logits(z, None, out=z.half())),
        (ValueError, lambda: tim.process_logits(z, None, out=z[:3])),
        (ValueError, lambda: tim.process_logits(z, L(temperature=f[:3]))),
        (TypeError, lambda: tim.process_logits(z, L(temperature=f.double()))),
        (ValueError, lambda: tim.process_logits(z, L(history=t))),
        (ValueError, lambda: tim.process_logits(z, L(bias_offsets=torch.zeros(5, dtype=torch.int32, device="cuda")))),
        (ValueError, lambda: tim.process_logits(z, L(allowed=torch.zeros(4, 3, dtype=torch.int32, device="cuda")))),
        (ValueError, lambda: tim.process_logits(z, L(allowed=torch.zeros(3, 4, dtype=torch.int32, device="cuda")))),
        (ValueError, lambda: tim.process_logits(z, L(allowed_rows=t))),
        (ValueError, lambda: tim.processed_logprob(z, None, t[:3])),
        (TypeError, lambda: tim.processed_logprob(z, None, t.long())),
        (ValueError, lambda: tim.processed_logprob_backward(z, None, t, f[:2], f)),
        (ValueError, lambda: tim.distill_topk(z, t.view(4, 1)[:3], f.view(4, 1)[:3])),
        (ValueError, lambda: tim.distill_topk(z, t.view(4, 1), f.view(2, 2))),
        (ValueError, lambda: tim.distill_topk(z, t.view(4, 1)[:, :0], f.view(4, 1)[:, :0])),
        (tim.TimError, lambda: tim.distill_topk(z, t.view(4, 1), f.view(4, 1), temperature=0.0)),
        (ValueError, lambda: tim.distill_topk_backward(z, t.view(4, 1), f.view(4, 1), f, f, lse_tail=f)),
    ]
    for kind, call in bad:
        with pytest.raises(kind):
            call()
    flat = torch.zeros(1000, device="cuda")
    with pytest.raises(tim.TimError):
        tim.process_logits(flat[:400].view(4, 100), None, out=flat[100:500].view(4, 100))
    for empty in (tim.process_logits(z[:0], None), tim.processed_logprob(z[:0], None, t[:0])[0]):
        assert empty.shape[0] == 0
    assert tim.distill_topk(z[:0], t.view(4, 1)[:0], f.view(4, 1)[:0])["loss"].shape[0] == 0
    tim.check()


def test_rules_are_a_dataclass_of_optional_tensors():
    assert all(getattr(tim.LogitsRules(), f.name) is None for f in dataclasses.fields(tim.LogitsRules))


# ----------------------------------------------------------------------------- together
def test_example_runs_the_operators_together():
    """The example's engine and trainer agree under the rules (both sides in fp32 on
    two matrix products: rounding only) and not without them; no drawn token breaks
    its grammar; its gradients are finite."""
    import importlib.util
    import os
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "processed_rollout.py")
    spec = importlib.util.spec_from_file_location("processed_rollout", path)
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    r = mod.main()
    # |y| stays below 40: a dozen roundings of it on each side
    assert r["mean_abs_delta"] < 40 * 24 * ref.U
    assert r["mean_abs_delta_without_the_rules"] > 0.05
    tok = r["sampled"].cpu().numpy()
    for b in range(tok.shape[0]):
        if b % 2:
            made = tok[b, 12:]
            assert (made % 7 != 0).all() if b // 2 % 2 == 0 else (made % 2 == 0).all()
    assert np.isfinite(r["grad_norm"]) and r["grad_norm"] > 0 and r["distill_loss"] > 0
    # no gradient on the prompt's positions
    assert bool((r["kd"]["dlogits"][r["weight"] == 0] == 0).all())


# ----------------------------------------------------------------------------- sizes past the usual
@pytest.mark.parametrize("V", [9001, 70001])
def test_rows_that_share_a_long_history(V):
    """More touched columns than a table holds, in rows that share their tokens (the
    table is built for halves of the columns), in place and not."""
    N, H = 30, 9000
    z, z64 = draw_logits(N, V, "bf16", V)
    rng = np.random.default_rng(V)
    tok = rng.integers(0, V, H).astype(np.int32)
    end = np.sort(rng.integers(H // 2, H + 1, N))
    r = {"history": tok, "history_spans": np.stack([np.zeros(N), end // 3, end], 1).astype(np.int32),
         "repetition": np.full(N, 1.3, np.float32), "frequency": np.full(N, 0.1, np.float32),
         "presence": np.full(N, 0.2, np.float32), "temperature": rng.uniform(0.5, 1.5, N).astype(np.float32)}
    R = rules(r)
    want, tol = ref.process_ref(z64, r, "bf16")
    y = tim.process_logits(z, R)
    assert_close(y, want, tol)
    t = rng.integers(0, V, N).astype(np.int32)
    lp, lse = tim.processed_logprob(z, R, dev(t))
    w, wl, ltol = ref.logprob_ref(z64, r, t)
    assert_close(lse, wl, ltol)
    assert_close(lp, w, ltol)
    g = rng.normal(0, 1, N).astype(np.float32)
    gw, gtol = ref.backward_ref(z64, r, t, g, lse.cpu().numpy(), "bf16")
    d = tim.processed_logprob_backward(z, R, dev(t), dev(g), lse)
    assert_close(d, gw, gtol)
    z2 = z.clone()
    assert torch.equal(tim.process_logits(z2, R, out=z2), y)
    z2 = z.clone()
    assert torch.equal(tim.processed_logprob_backward(z2, R, dev(t), dev(g), lse, dlogits=z2), d)
    tim.check()


@pytest.mark.parametrize("V", [300001, 1 << 20])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_widest_vocabularies(V, dtype):
    """Rows wider than a table and than what a cluster's shared memory holds."""
    N = 2
    z, z64 = draw_logits(N, V, dtype, 3)
    r = draw_rules(N, V, 4, hist=500, bias=50)
    r["allowed_rows"][:] = -1
    t = np.array([V - 1, 12345], np.int32)
    R = rules(r)
    w, wl, tol = ref.logprob_ref(z64, r, t)
    lp, lse = tim.processed_logprob(z, R, dev(t))
    assert_close(lp, w, tol)
    assert_close(lse, wl, tol)
    want, ptol = ref.process_ref(z64, r, "f32")
    assert_close(tim.process_logits(z, R, out_dtype=torch.float32), want, ptol)
    g = np.array([1.0, -0.5], np.float32)
    gw, gtol = ref.backward_ref(z64, r, t, g, lse.cpu().numpy(), dtype)
    assert_close(tim.processed_logprob_backward(z, R, dev(t), dev(g), lse), gw, gtol)
    ids, tt, tlse = draw_teacher(N, V, 300, 7, holes=False)
    o = tim.distill_topk_step(z, dev(ids), dev(tt), dev(g), teacher_lse=dev(tlse))
    dw = ref.distill_ref(z64, ids, tt, tlse, 1.0, g, dtype)
    assert_close(o["loss"], dw["loss"], dw["loss_tol"])
    assert_close(o["lse_tail"], dw["lse_tail"], dw["lse_tol"])
    assert_close(o["dlogits"], dw["dlogits"], dw["dlogits_tol"])
    f = tim.distill_topk(z, dev(ids), dev(tt), dev(tlse))
    assert torch.equal(f["loss"], o["loss"])
    b = tim.distill_topk_backward(z, dev(ids), dev(tt), dev(g), f["lse"], f["lse_tail"], teacher_lse=dev(tlse))
    bw = ref.distill_ref(z64, ids, tt, tlse, 1.0, g, dtype, (f["lse"].cpu().numpy(), f["lse_tail"].cpu().numpy()))
    assert_close(b, bw["dlogits"], bw["dlogits_tol"])
    tim.check()


def test_offsets_past_32_bits():
    """3.0e9 logits (6 GB): the last rows have the bits they have alone."""
    N, V = 20000, 151936
    z = torch.empty(N, V, dtype=torch.bfloat16, device="cuda")
    for i in range(0, N, 2000):
        z[i:i + 2000].normal_(generator=None)
    last = slice(N - 3, N)
    t = torch.arange(N, device="cuda", dtype=torch.int32)
    one = torch.ones(N, device="cuda")
    tau = one * 0.8
    lp, lse = tim.processed_logprob(z, tim.LogitsRules(temperature=tau), t)
    few = tim.LogitsRules(temperature=tau[last])
    lp3, lse3 = tim.processed_logprob(z[last], few, t[last])
    assert torch.equal(lp[last], lp3) and torch.equal(lse[last], lse3)
    out = tim.process_logits(z, tim.LogitsRules(temperature=tau))
    assert torch.equal(out[last], tim.process_logits(z[last], few))
    d = tim.processed_logprob_backward(z, tim.LogitsRules(temperature=tau), t, one, lse, dlogits=out)
    assert torch.equal(d[last], tim.processed_logprob_backward(z[last], few, t[last], one[:3], lse3))
    ids = (torch.arange(8, device="cuda").repeat(N, 1) * 100 + t.view(-1, 1) % 50).int().contiguous()
    tl = torch.zeros(N, 8, device="cuda")
    s = tim.distill_topk_step(z, ids, tl, one, dlogits=out)
    s3 = tim.distill_topk_step(z[last], ids[last], tl[last], one[:3])
    assert torch.equal(s["loss"][last], s3["loss"]) and torch.equal(s["dlogits"][last], s3["dlogits"])
    tim.check()


def test_outputs_given_to_a_stream_stay_its_own():
    """Outputs that a call allocates for another stream come from that stream's memory:
    dropping them at once does not let the current stream write over them early."""
    V, N = 151936, 64
    z = torch.randn(N, V, device="cuda")
    want = tim.process_logits(z, None)
    t = torch.zeros(N, dtype=torch.int32, device="cuda")
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for _ in range(20):
        y = tim.process_logits(z, None, stream=side)
        keep = [tim.processed_logprob(z, None, t, stream=side)[1] for _ in range(2)]
        del keep
        junk = torch.full((N, V), 7.0, device="cuda")     # would take a freed block of the current stream
        side.synchronize()
        assert torch.equal(y, want)
        del junk, y
    tim.check()
