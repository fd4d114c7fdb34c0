"""The operators beside the head's table against their definitions in fp64: low-rank
adapters on its logits, embedding lookup, and their gradients.

Tolerances, element by element, from the arithmetic (half = half a unit of the last
place of a type, relative: 2^-24, 2^-8, 2^-11 for fp32, bf16, fp16):
  * a product of k steps of 16 on the tensor cores adds at most (k + 8) 2^-23 of the
    sum of its terms' magnitudes (each step rounds, or cuts, the running sum);
  * t is held in two bf16 parts for 16-bit logits (2^-16 of it is left at most: each
    part leaves half a unit, 2^-8), in three for fp32 logits and in the gradient, and so
    are fp32 dlogits and du (2^-24; products of parts of that size are left out).
"""
import math

import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import rollout_logprob_mismatch_gb300 as tim  # noqa: E402

F64 = torch.float64
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
HALF = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8, "f16": 2.0 ** -11}
TINY = {"f32": 2.0 ** -140, "bf16": 2.0 ** -130, "f16": 2.0 ** -25}
U = 2.0 ** -23


def draw(N, V, D, R, n, dtype, seed, stride=None, offset=0):
    """Logits [N, V] (rows `stride` apart, `offset` elements into their buffer), h, adapters, rows."""
    gen = torch.Generator(device="cuda").manual_seed(seed)
    stride = V if stride is None else stride
    buf = (torch.randn(offset + N * stride + 64, generator=gen, device="cuda") * 2).to(TYPES[dtype])
    z = torch.as_strided(buf, (N, V), (stride, 1), offset)
    h = torch.randn((N, D), generator=gen, device="cuda").to(torch.bfloat16)
    A = ((torch.rand((n, R, D), generator=gen, device="cuda") * 2 - 1) / math.sqrt(D)).to(torch.bfloat16)
    B = (torch.randn((n, V, R), generator=gen, device="cuda") * 0.3).to(torch.bfloat16)
    scale = torch.rand(n, generator=gen, device="cuda") * 2 + 0.25
    rows = torch.randint(-1, n + 1, (N,), generator=gen, device="cuda", dtype=torch.int32)
    return z, h, tim.Adapters(A, B, scale), rows


def live(rows, n):
    return (rows >= 0) & (rows < n)


def parts64(h, ad, rows):
    """(t, bound on the rounding of its sums) [N, R] in fp64."""
    n, R, D = ad.A.shape
    a = rows.long().clamp(0, n - 1)
    s = (torch.ones(n, device=h.device) if ad.scale is None else ad.scale).to(F64)[a].view(-1, 1)
    t = torch.zeros((h.shape[0], R), dtype=F64, device=h.device)
    m = torch.zeros_like(t)
    for k in range(n):
        i = torch.nonzero(rows == k).view(-1)
        t[i] = s[i] * (h[i].to(F64) @ ad.A[k].to(F64).t())
        m[i] = s[i] * (h[i].to(F64).abs() @ ad.A[k].to(F64).abs().t())
    # a chain: two steps for every 16th 32 columns, then 16 shares
    return t, m * ((D + 31) // 32 / 2 + 24) * U


def logits64(z, h, ad, rows, dtype):
    """(y, its tolerance) [N, V]."""
    n, V, R = ad.B.shape
    t, dt = parts64(h, ad, rows)
    y, tol = z.to(F64).clone(), torch.zeros(z.shape, dtype=F64, device=z.device)
    left = 2.0 ** -24 if dtype == "f32" else 2.0 ** -16
    for k in range(n):
        i = torch.nonzero(rows == k).view(-1)
        B = ad.B[k].to(F64).t()
        y[i] += t[i] @ B
        tol[i] = (dt[i] + t[i].abs() * (left + (3 * (R + 15) // 16 + 8) * U)) @ B.abs() + y[i].abs() * (HALF[dtype] + U) + TINY[dtype]
    return y, tol


def check(got, want, tol, what=""):
    got = got.to(F64)
    bad = ~((got - want).abs() <= tol) & ~((got == want) | (got.isnan() & want.isnan()))
    if bool(bad.any()):
        i = torch.nonzero(bad)[0].tolist()
        raise AssertionError("%s: %d wrong, first at %s: %r, expected %r within %r"
                             % (what, int(bad.sum()), i, float(got[tuple(i)]), float(want[tuple(i)]), float(tol[tuple(i)])))


def bits(x):
    return x.contiguous().view(torch.int32 if x.dtype == torch.float32 else torch.int16)


# ----------------------------------------------------------------------------- adapters on logits
CASES = [  # N, V, D, R, n, dtype, stride past V, offset
    (1, 1000, 64, 8, 1, "bf16", 0, 0), (1, 257, 8, 128, 3, "f32", 0, 0), (17, 333, 72, 16, 3, "f32", 0, 0),
    (70, 4099, 136, 24, 5, "f16", 0, 0), (200, 1024, 256, 32, 2, "bf16", 0, 0), (33, 777, 64, 64, 40, "bf16", 0, 0),
    (300, 515, 128, 128, 3, "f32", 0, 0), (65, 2048, 520, 40, 7, "bf16", 8, 0), (129, 600, 64, 16, 1, "f16", 5, 3),
    (40, 301, 1000, 72, 4, "bf16", 3, 1), (600, 100, 64, 16, 200, "f32", 1, 3), (16, 1, 64, 16, 2, "bf16", 0, 0),
    (1000, 31, 64, 8, 6, "bf16", 0, 5), (257, 8, 24, 16, 2, "f16", 0, 0), (31, 40000, 64, 16, 3, "bf16", 0, 0),
    (5000, 40, 64, 16, 3, "bf16", 0, 0), (12000, 24, 64, 8, 2, "f16", 0, 0)]


@pytest.mark.parametrize("N,V,D,R,n,dtype,more,offset", CASES)
def test_adapter_logits(N, V, D, R, n, dtype, more, offset):
    z, h, ad, rows = draw(N, V, D, R, n, dtype, 1, V + more, offset)
    y, tol = logits64(z, h, ad, rows, dtype)
    before = z.clone()
    out = tim.adapter_logits(z, h, ad, rows)
    tim.check()
    assert torch.equal(bits(z), bits(before))
    check(out, y, tol, "out of place")
    none = ~live(rows, n)
    assert torch.equal(bits(out[none]), bits(z[none]))
    other = torch.full((N, V + 11), 7.0, dtype=z.dtype, device="cuda")
    assert tim.adapter_logits(z, h, ad, rows, out=other[:, 3:3 + V]).data_ptr() == other[:, 3:].data_ptr()
    assert torch.equal(bits(other[:, 3:3 + V]), bits(out))
    assert bool((other[:, :3] == 7).all()) and bool((other[:, 3 + V:] == 7).all())
    around = z._base.clone() if z._base is not None else None
    tim.adapter_logits(z, h, ad, rows, out=z)
    tim.check()
    assert torch.equal(bits(z), bits(out))
    if around is not None:   # nothing between or behind the rows
        torch.as_strided(around, z.shape, z.stride(), z.storage_offset()).copy_(out)
        assert torch.equal(bits(around), bits(z._base))


def test_adapter_logits_without_scale_and_contiguous_runs():
    z, h, ad, _ = draw(700, 1200, 64, 16, 4, "bf16", 2)
    ad = tim.Adapters(ad.A, ad.B)
    rows = torch.tensor([2] * 300 + [-1] * 50 + [0] * 300 + [2] * 50, dtype=torch.int32, device="cuda")
    y, tol = logits64(z, h, ad, rows, "bf16")
    check(tim.adapter_logits(z, h, ad, rows), y, tol)


def test_a_row_has_the_same_bits_whatever_rows_are_beside_it():
    z, h, ad, rows = draw(150, 3001, 264, 32, 9, "bf16", 3)
    out = tim.adapter_logits(z, h, ad, rows)
    for i in (0, 1, 17, 77, 149):
        one = tim.adapter_logits(z[i:i + 1], h[i:i + 1], ad, rows[i:i + 1])
        assert torch.equal(bits(one[0]), bits(out[i]))
    perm = torch.randperm(150, device="cuda")
    again = tim.adapter_logits(z[perm].contiguous(), h[perm].contiguous(), ad, rows[perm].contiguous())
    assert torch.equal(bits(again), bits(out[perm]))


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
def test_a_rows_bits_are_those_of_larger_batches(dtype):
    """Batches that are ordered and projected in one launch, in two, and in two with
    more CTAs than SMs."""
    z, h, ad, rows = draw(6000, 700, 520, 40, 5, dtype, 15)
    out = tim.adapter_logits(z, h, ad, rows)
    for n in (1, 40, 256, 257, 2000):
        part = tim.adapter_logits(z[:n], h[:n], ad, rows[:n])
        assert torch.equal(bits(part), bits(out[:n])), n
    y, tol = logits64(z, h, ad, rows, dtype)
    check(out, y, tol)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_one_tenants_infinities_reach_no_other(dtype):
    z, h, ad, rows = draw(64, 900, 64, 16, 6, dtype, 4)
    clean = tim.adapter_logits(z, h, ad, rows)
    A, B = ad.A.clone(), ad.B.clone()
    B[2] = float("nan")
    A[4] = float("inf")
    B[5, 17, 3] = float("inf")
    out = tim.adapter_logits(z, h, tim.Adapters(A, B, ad.scale), rows)
    other = (rows != 2) & (rows != 4) & (rows != 5)
    assert torch.equal(bits(out[other]), bits(clean[other]))
    assert bool(out[rows == 2].isnan().all())
    five = torch.nonzero(rows == 5).view(-1)
    keep = torch.ones(900, dtype=torch.bool, device="cuda")
    keep[17] = False
    assert torch.equal(bits(out[five][:, keep]), bits(clean[five][:, keep]))
    assert not bool(out[five, 17].isfinite().any())
    g = tim.adapter_logits_backward(z, h, ad, rows)
    b = tim.adapter_logits_backward(z, h, tim.Adapters(A, B, ad.scale), rows)
    assert torch.equal(g[0][other], b[0][other])
    for a in (0, 1, 3):
        assert torch.equal(g[1][a], b[1][a]) and torch.equal(g[2][a], b[2][a])


def test_logits_of_masked_ids_and_special_values():
    z, h, ad, rows = draw(40, 640, 64, 8, 3, "bf16", 5)
    rows[:8] = -1
    rows[8:] = torch.arange(32, device="cuda", dtype=torch.int32) % 3
    z[:, 5] = float("-inf")
    z[:, 9] = torch.finfo(torch.bfloat16).min
    z[3, 11], z[12, 11], z[4, 12] = float("nan"), float("nan"), -0.0
    z[2].view(torch.int16)[20] = 0x7fa1   # a NaN with a payload, in a row that is copied
    out = tim.adapter_logits(z, h, ad, rows)
    assert bool((out[:, 5] == float("-inf")).all())
    assert torch.equal(bits(out[:8]), bits(z[:8]))
    assert bool(out[12, 11].isnan())
    y, tol = logits64(z, h, ad, rows, "bf16")
    ok = y.isfinite()
    check(out[ok], y[ok], tol[ok])


def test_empty_batches_and_no_adapters():
    z, h, ad, rows = draw(12, 100, 64, 16, 2, "f32", 6)
    none = tim.Adapters(ad.A[:0], ad.B[:0], ad.scale[:0])
    assert torch.equal(tim.adapter_logits(z, h, none, rows), z)
    dh, dA, dB = tim.adapter_logits_backward(z, h, none, rows)
    assert dA.shape[0] == 0 and not bool(dh.any())
    out = tim.adapter_logits(z[:0], h[:0], ad, rows[:0])
    assert out.shape == (0, 100)
    dh, dA, dB = tim.adapter_logits_backward(z[:0], h[:0], ad, rows[:0])
    assert not bool(dA.any()) and not bool(dB.any())
    rows[:] = -1
    dh, dA, dB = tim.adapter_logits_backward(z, h, ad, rows)
    assert not bool(dh.any()) and not bool(dA.any()) and not bool(dB.any())
    tim.check()


# ----------------------------------------------------------------------------- gradient
def grads64(dy, h, ad, rows, dtype):
    """{name: (value, tolerance)}."""
    n, R, D = ad.A.shape
    N, V = dy.shape
    d, x = dy.to(F64), h.to(F64)
    t, dt = parts64(h, ad, rows)
    left = 5 * 2.0 ** -24   # t's and dlogits' third parts, three products of parts
    z = lambda *s: torch.zeros(s, dtype=F64, device=dy.device)   # noqa: E731
    dh, th, dA, tA, dB, tB = z(N, D), z(N, D), z(n, R, D), z(n, R, D), z(n, V, R), z(n, V, R)
    s = torch.ones(n, dtype=F64, device=dy.device) if ad.scale is None else ad.scale.to(F64)
    for k in range(n):
        i = torch.nonzero(rows == k).view(-1)
        A, B = ad.A[k].to(F64), ad.B[k].to(F64)
        m = i.numel()
        dB[k] = d[i].t() @ t[i]
        tB[k] = d[i].abs().t() @ (t[i].abs() * (left + (m / 4 + 16) * U) + dt[i])
        du = s[k] * (d[i] @ B)
        # steps of a slab, slabs by eight, eight parts: far fewer than V / 16
        tu = s[k] * (d[i].abs() @ B.abs()) * (96 + V / 1024) * U
        dA[k] = du.t() @ x[i]
        tA[k] = (tu + du.abs() * (m / 4 + 16) * U).t() @ x[i].abs()
        dh[i] = du @ A
        th[i] = (tu + du.abs() * (3 * (R + 15) // 16 + 8) * U) @ A.abs()
    tiny = 2.0 ** -120
    return {"dh": (dh, th + tiny), "dA": (dA, tA + tiny), "dB": (dB, tB + tiny)}


GRADS = [(1, 1000, 64, 8, 1, "bf16", 0, 0), (17, 333, 72, 16, 3, "f32", 0, 0), (70, 4099, 136, 24, 5, "f16", 0, 0),
         (200, 1024, 256, 32, 2, "bf16", 0, 0), (33, 776, 64, 64, 40, "bf16", 0, 0), (300, 515, 128, 128, 3, "f32", 0, 0),
         (65, 2050, 520, 40, 7, "bf16", 6, 0), (129, 600, 64, 16, 1, "f16", 5, 3), (40, 301, 1000, 72, 4, "bf16", 3, 1),
         (600, 100, 64, 16, 200, "f32", 1, 3), (16, 1, 64, 16, 2, "bf16", 0, 0), (16, 3, 64, 16, 2, "f32", 0, 1),
         (300, 1500, 64, 128, 2, "bf16", 4, 0), (48, 130000, 64, 16, 2, "bf16", 0, 0), (48, 125001, 64, 32, 2, "bf16", 0, 0),
         (40, 70000, 64, 64, 2, "bf16", 0, 0), (33, 66000, 64, 32, 2, "f32", 0, 0), (33, 66001, 64, 64, 2, "f16", 0, 0),
         (1500, 3000, 64, 16, 2, "bf16", 0, 0), (1500, 2999, 64, 64, 2, "bf16", 1, 0)]


@pytest.mark.parametrize("N,V,D,R,n,dtype,more,offset", GRADS)
def test_adapter_logits_backward(N, V, D, R, n, dtype, more, offset):
    dy, h, ad, rows = draw(N, V, D, R, n, dtype, 7, V + more, offset)
    want = grads64(dy, h, ad, rows, dtype)
    dh, dA, dB = tim.adapter_logits_backward(dy, h, ad, rows)
    tim.check()
    for name, got in (("dh", dh), ("dA", dA), ("dB", dB)):
        check(got, *want[name], name)
    again = tim.adapter_logits_backward(dy, h, ad, rows)
    assert all(torch.equal(x, y) for x, y in zip((dh, dA, dB), again))
    # accumulating: the sum of what was there and the gradient, one rounding
    base = [torch.randn_like(x) for x in (dh, dA, dB)]
    acc = [x.clone() for x in base]
    tim.adapter_logits_backward(dy, h, ad, rows, *acc, accumulate_dh=True, accumulate_adapters=True)
    for x, b, g in zip(acc, base, (dh, dA, dB)):
        assert torch.equal(x, b + g)
    tim.check()


def test_gradient_of_a_batch_in_parts():
    """More rows than the partial sums of one launch have room for (2^30 bytes): adapters
    whose rows span the parts, and one that has none."""
    N, V, D, R = 17000, 131072, 64, 64
    gen = torch.Generator(device="cuda").manual_seed(8)
    dy = torch.empty((N, V), dtype=torch.bfloat16, device="cuda")
    for i in range(0, N, 1000):
        dy[i:i + 1000] = torch.randn((1000, V), generator=gen, device="cuda")
    h = torch.randn((N, D), generator=gen, device="cuda").to(torch.bfloat16)
    A = (torch.rand((3, R, D), generator=gen, device="cuda") * 0.2 - 0.1).to(torch.bfloat16)
    B = torch.randn((3, V, R), generator=gen, device="cuda").to(torch.bfloat16)
    rows = torch.where(torch.arange(N, device="cuda") % 3 == 0, 0, 2).to(torch.int32)
    ad = tim.Adapters(A, B)
    dh, dA, dB = tim.adapter_logits_backward(dy, h, ad, rows)
    tim.check()
    assert not bool(dA[1].any()) and not bool(dB[1].any())
    for k in (0, 2):
        i = torch.nonzero(rows == k).view(-1)
        t, dt = parts64(h[i], tim.Adapters(A[k:k + 1], B[k:k + 1]), torch.zeros_like(rows[i]))
        steps = i.numel() / 8 + 16
        tt = t.abs() * 2 * steps * U + dt
        wB, mB = torch.zeros((V, R), dtype=F64, device="cuda"), torch.zeros((V, R), dtype=F64, device="cuda")
        du = torch.empty((i.numel(), R), dtype=F64, device="cuda")
        mu = torch.empty_like(du)
        for j in range(0, i.numel(), 1000):
            d = dy[i[j:j + 1000]].to(F64)
            wB += d.t() @ t[j:j + 1000]
            mB += d.abs().t() @ tt[j:j + 1000]
            du[j:j + 1000] = d @ B[k].to(F64)
            mu[j:j + 1000] = d.abs() @ B[k].to(F64).abs()
        check(dB[k], wB, mB, "dB")
        tu = mu * (96 + V / 1024) * U
        check(dh[i], du @ A[k].to(F64), (tu + du.abs() * 32 * U) @ A[k].to(F64).abs(), "dh")
        check(dA[k], du.t() @ h[i].to(F64), (tu + du.abs() * steps * 2 * U).t() @ h[i].to(F64).abs(), "dA")


def test_gradient_against_differences():
    """The forward is linear in each of h, A and B: differences of its fp32 outputs have
    no error but their roundings."""
    N, V, D, R, n = 24, 200, 64, 16, 3
    z, h, ad, rows = draw(N, V, D, R, n, "f32", 9)
    w = torch.randn((N, V), device="cuda")
    grads = dict(zip(("h", "A", "B"), tim.adapter_logits_backward(w, h, ad, rows)))
    here = {"h": h, "A": ad.A, "B": ad.B}

    def outputs(x):
        return tim.adapter_logits(z, x["h"], tim.Adapters(x["A"], x["B"], ad.scale), rows)

    y0 = outputs(here)
    for name in ("h", "A", "B"):
        moved = (here[name].float() + torch.randn(here[name].shape, device="cuda")).to(torch.bfloat16)
        y1 = outputs({**here, name: moved})
        got = ((y1.to(F64) - y0.to(F64)) * w.to(F64)).sum()
        delta = moved.to(F64) - here[name].to(F64)
        want = (grads[name].to(F64) * delta).sum()
        # each output's roundings, and 2^-13 of the gradient's terms (its parts and sums, above)
        room = (w.to(F64).abs() * (y0.abs() + y1.abs() + z.abs()).to(F64)).sum() * 64 * U
        room = float(room + (grads[name].to(F64) * delta).abs().sum() * 2.0 ** -13)
        assert abs(float(got - want)) <= room, (name, float(got), float(want), room)


# ----------------------------------------------------------------------------- embedding
@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("out", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("N,V,D", [(1, 10, 8), (5, 1, 1), (300, 500, 257), (77, 1000, 1024), (9, 33, 3000), (600, 64, 256)])
def test_embedding(N, V, D, dtype, out):
    gen = torch.Generator(device="cuda").manual_seed(N + D)
    W = torch.randn((V, D), generator=gen, device="cuda").to(TYPES[dtype])
    t = torch.randint(-2, V + 2, (N,), generator=gen, device="cuda", dtype=torch.int32)
    scale = 1.7
    got = tim.embedding(t, W, scale, out_dtype=TYPES[out])
    on = (t >= 0) & (t < V)
    want = torch.where(on.view(-1, 1), W[t.long().clamp(0, V - 1)].to(F64) * float(np.float32(scale)), 0.0)
    check(got, want, want.abs() * (HALF[out] * (1 + 2.0 ** -20) + 2.0 ** -24) + TINY[out])
    assert not bool(got[~on].any())
    tim.check()


def test_embedding_takes_views_that_start_anywhere():
    W = torch.randn(2 + 50 * 37, device="cuda").to(torch.bfloat16)[1:1 + 50 * 37].view(50, 37)
    t = torch.randint(0, 50, (90,), device="cuda", dtype=torch.int32)
    buf = torch.full((3 + 90 * 37 + 5,), 9.0, device="cuda", dtype=torch.bfloat16)
    out = tim.embedding(t, W, out=buf[3:3 + 90 * 37].view(90, 37))
    assert torch.equal(out, W[t.long()])
    assert bool((buf[:3] == 9).all()) and bool((buf[3 + 90 * 37:] == 9).all())
    g = torch.randn(1 + 90 * 37, device="cuda")[1:].view(90, 37)
    buf = torch.full((1 + 50 * 37 + 3,), 9.0, device="cuda")
    dW = tim.embedding_backward(t, g, 50, dW=buf[1:1 + 50 * 37].view(50, 37))
    want = torch.zeros((50, 37), dtype=F64, device="cuda").index_add_(0, t.long(), g.to(F64))
    size = torch.zeros((50, 37), dtype=F64, device="cuda").index_add_(0, t.long(), g.to(F64).abs())
    check(dW, want, size * 100 * 2.0 ** -24)
    assert float(buf[0]) == 9 and bool((buf[1 + 50 * 37:] == 9).all())


def tokens_like(kind, N, V, gen):
    if kind == "uniform":
        return torch.randint(0, V, (N,), generator=gen, device="cuda", dtype=torch.int32)
    if kind == "one":
        return torch.full((N,), V - 1, device="cuda", dtype=torch.int32)
    if kind == "few":
        return (torch.randint(0, 3, (N,), generator=gen, device="cuda") * (V // 3)).to(torch.int32)
    if kind == "out":
        return torch.randint(-V, 2 * V, (N,), generator=gen, device="cuda", dtype=torch.int32)
    t = (torch.rand(N, generator=gen, device="cuda") ** 4 * V).to(torch.int32).clamp_(max=V - 1)
    return t


@pytest.mark.parametrize("kind", ["uniform", "one", "few", "out", "text"])
@pytest.mark.parametrize("N,V,D,dtype", [(1, 7, 8, "bf16"), (33, 1025, 40, "f32"), (65, 50, 257, "f16"),
                                          (1000, 5000, 1032, "bf16"), (5000, 3000, 64, "bf16"), (2048, 512, 100, "f32"),
                                          (20001, 2000, 72, "bf16"), (70000, 700, 33, "f16")])
def test_embedding_backward(kind, N, V, D, dtype):
    gen = torch.Generator(device="cuda").manual_seed(N)
    t = tokens_like(kind, N, V, gen)
    g = torch.randn((N, D), generator=gen, device="cuda").to(TYPES[dtype])
    scale = 0.3
    on = torch.nonzero((t >= 0) & (t < V)).view(-1)
    x = g[on].to(F64) * float(np.float32(scale))
    want = torch.zeros((V, D), dtype=F64, device="cuda").index_add_(0, t[on].long(), x)
    size = torch.zeros((V, D), dtype=F64, device="cuda").index_add_(0, t[on].long(), x.abs())
    count = torch.zeros(V, dtype=F64, device="cuda").index_add_(0, t[on].long(), torch.ones_like(on, dtype=F64))
    # a chain of at most max(64, tile) tokens, or a tile's and then the tiles; and the product with the scale
    tile = 32
    while 16 * tile * tile < N:
        tile *= 2
    chain = torch.where(count <= max(64, tile), count, tile + count / tile + 2).view(-1, 1)
    tol = size * (chain + 1) * 2.0 ** -24
    dW = tim.embedding_backward(t, g, V, scale)
    tim.check()
    check(dW, want, tol)
    assert torch.equal(dW, tim.embedding_backward(t, g, V, scale))
    base = torch.randn((V, D), generator=gen, device="cuda")
    acc = base.clone()
    tim.embedding_backward(t, g, V, scale, dW=acc, accumulate_dW=True)
    tim.check()
    assert torch.equal(acc, base + dW)
    assert torch.equal(bits(acc[count == 0]), bits(base[count == 0]))


def test_embedding_gradient_of_an_empty_batch():
    t, g = torch.zeros(0, dtype=torch.int32, device="cuda"), torch.zeros((0, 24), device="cuda")
    assert not bool(tim.embedding_backward(t, g, 9, dW=torch.ones((9, 24), device="cuda")).any())
    dW = torch.ones((9, 24), device="cuda")
    assert bool((tim.embedding_backward(t, g, 9, dW=dW, accumulate_dW=True) == 1).all())
    assert tim.embedding(t, dW).shape == (0, 24)


def test_embedding_gradient_against_differences():
    N, V, D = 50, 20, 33
    t = torch.randint(-1, V, (N,), device="cuda", dtype=torch.int32)
    W, w = torch.randn((V, D), device="cuda"), torch.randn((N, D), device="cuda")
    dW = tim.embedding_backward(t, w, V, 3.0)
    for _ in range(3):
        moved = W + torch.randn((V, D), device="cuda")
        got = ((tim.embedding(t, moved, 3.0).to(F64) - tim.embedding(t, W, 3.0).to(F64)) * w.to(F64)).sum()
        want = (dW.to(F64) * (moved.to(F64) - W.to(F64))).sum()
        # two roundings of each row's product, and a chain of up to 50 in dW
        room = float((w.abs().sum() * 3 * (W.abs().max() + moved.abs().max())) * 60 * 2.0 ** -24)
        assert abs(float(got - want)) <= room


# ----------------------------------------------------------------------------- used together
def test_a_tied_head_with_adapters_as_it_is_trained():
    """tokens -> embedding -> head's logits -> adapters -> the chosen tokens'
    log-probability, and back: dA, dB, and dW from both ends of the table; against
    automatic differentiation in fp64."""
    V, D, R, n, N = 700, 64, 16, 2, 96
    gen = torch.Generator(device="cuda").manual_seed(11)
    W = (torch.randn((V, D), generator=gen, device="cuda") * 0.2).to(torch.bfloat16)
    _, _, ad, rows = draw(N, V, D, R, n, "f32", 12)
    tokens = torch.randint(-1, V, (N,), generator=gen, device="cuda", dtype=torch.int32)
    targets = torch.randint(0, V, (N,), generator=gen, device="cuda", dtype=torch.int32)
    g = torch.randn(N, generator=gen, device="cuda")
    s = math.sqrt(D)

    h = tim.embedding(tokens, W, s)
    z = (h.to(F64) @ W.to(F64).t()).float()
    tim.adapter_logits(z, h, ad, rows, out=z)
    logp, lse = tim.processed_logprob(z, None, targets)
    dz = tim.processed_logprob_backward(z, None, targets, g, lse)
    dh = (dz.to(F64) @ W.to(F64)).float()
    dW = (dz.to(F64).t() @ h.to(F64)).float()
    _, dA, dB = tim.adapter_logits_backward(dz, h, ad, rows, dh=dh, accumulate_dh=True)
    tim.embedding_backward(tokens, dh, V, s, dW=dW, accumulate_dW=True)
    tim.check()

    on = live(rows, n)
    a = rows.long().clamp(0, n - 1)
    h64 = h.to(F64).requires_grad_(True)
    W1, A1, B1 = (x.to(F64).requires_grad_(True) for x in (W, ad.A, ad.B))
    u = torch.einsum("nd,nrd->nr", h64, A1[a]) * ad.scale.to(F64)[a].view(-1, 1)
    y = h64 @ W1.t() + torch.where(on.view(-1, 1), torch.einsum("nr,nvr->nv", u, B1[a]), 0.0)
    want = torch.log_softmax(y, 1).gather(1, targets.long().view(-1, 1)).view(-1)
    (want * g.to(F64)).sum().backward()
    live_t = (tokens >= 0).view(-1, 1)
    wW = W1.grad.index_add(0, tokens.long().clamp(min=0), torch.where(live_t, h64.grad * s, 0.0))
    rel = lambda x, y: float((x.to(F64) - y).norm() / y.norm())   # noqa: E731
    # fp32 logits of size up to some 30 hold 2^-24 of it, and so do lse and the
    # probabilities' exponents: 1e-5 of a probability
    assert float((logp.to(F64) - want.detach()).abs().max()) <= 2e-5
    for got, ref in ((dh, h64.grad), (dA, A1.grad), (dB, B1.grad), (dW, wW)):
        assert rel(got, ref) <= 6e-5


# ----------------------------------------------------------------------------- streams, graphs
def test_streams_and_graphs():
    dy, h, ad, rows = draw(200, 1500, 128, 16, 4, "bf16", 13)
    tokens = torch.randint(-1, 1500, (400,), device="cuda", dtype=torch.int32)
    W = torch.randn((1500, 128), device="cuda").to(torch.bfloat16)
    g = torch.randn((400, 128), device="cuda")

    def calls():
        return (tim.adapter_logits(dy, h, ad, rows), *tim.adapter_logits_backward(dy, h, ad, rows),
                tim.embedding(tokens, W, 2.0), tim.embedding_backward(tokens, g, 1500))

    want = calls()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        other = calls()
    s.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(want, other))
    graphs = []
    for _ in range(2):   # two graphs, replayed in turn and at the same time on two streams
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = calls()
        graphs.append((graph, out))
    for _ in range(3):
        for graph, out in graphs:
            for x in out:
                x.fill_(3)
            graph.replay()
            torch.cuda.synchronize()
            assert all(torch.equal(x, y) for x, y in zip(want, out))
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(10):
        for st, (graph, _) in zip(streams, graphs):
            with torch.cuda.stream(st):
                graph.replay()
    torch.cuda.synchronize()
    for _, out in graphs:
        assert all(torch.equal(x, y) for x, y in zip(want, out))
    tim.check()


def test_wrappers_refuse():
    z, h, ad, rows = draw(6, 100, 64, 16, 2, "bf16", 14)
    bad = [dict(h=h.float()), dict(h=h[:5]), dict(rows=rows.long()), dict(rows=rows[:5]), dict(adapters=(ad.A, ad.B)),
           dict(adapters=tim.Adapters(ad.A[:, :4], ad.B)), dict(adapters=tim.Adapters(ad.A.float(), ad.B)),
           dict(adapters=tim.Adapters(ad.A, ad.B[:, :99].contiguous())), dict(adapters=tim.Adapters(ad.A, ad.B[:1])),
           dict(adapters=tim.Adapters(ad.A, ad.B, ad.scale.double())), dict(adapters=tim.Adapters(ad.A, ad.B, ad.scale[:1])),
           dict(adapters=tim.Adapters(None, ad.B)), dict(z=z.double()), dict(z=z.t()), dict(z=z[:, ::2])]
    for b in bad:
        args = {"z": z, "h": h, "adapters": ad, "rows": rows, **b}
        for f in (tim.adapter_logits, tim.adapter_logits_backward):
            with pytest.raises((TypeError, ValueError)):
                f(args["z"], args["h"], args["adapters"], args["rows"])
    with pytest.raises((TypeError, ValueError)):
        tim.adapter_logits(z, h, ad, rows, out=torch.empty_like(z).float())
    with pytest.raises(tim.TimError):
        tim.adapter_logits(z[:5], h[:5], ad, rows[:5].contiguous(), out=z[1:])
    with pytest.raises(ValueError):
        tim.adapter_logits_backward(z, h, ad, rows, accumulate_dh=True)
    with pytest.raises((TypeError, ValueError)):
        tim.adapter_logits_backward(z, h, ad, rows, dA=torch.empty((2, 16, 65), device="cuda"))
    t = torch.zeros(6, dtype=torch.int32, device="cuda")
    for f in (lambda: tim.embedding(t.long(), z), lambda: tim.embedding(t, z.double()), lambda: tim.embedding(t, z.t()),
              lambda: tim.embedding(t, z, out=torch.empty((5, 100), dtype=z.dtype, device="cuda")),
              lambda: tim.embedding(t, z, out_dtype=torch.float64), lambda: tim.embedding_backward(t[:3], z, 9),
              lambda: tim.embedding_backward(t, z, 9, accumulate_dW=True),
              lambda: tim.embedding_backward(t, z, 9, dW=torch.empty((8, 100), device="cuda"))):
        with pytest.raises((TypeError, ValueError)):
            f()


# ----------------------------------------------------------------------------- the far ends
@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("V,R", [(130, 16), (130, 32), (300, 64), (2050, 8), (2050, 128)])
def test_gradient_of_adapters_of_many_steps(V, R, dtype):
    """Adapters of none to 21 steps of rows: dB's sums, taken in turn, that have something or not."""
    counts = [1, 0, 32, 129, 300, 0, 500, 1300, 17]
    gen = torch.Generator(device="cuda").manual_seed(V + R)
    N, n = sum(counts) + 11, len(counts)
    dy, h, ad, rows = draw(N, V, 72, R, n, dtype, 21)
    ids = torch.cat([torch.full((c,), k, dtype=torch.int32) for k, c in enumerate(counts)] + [torch.full((11,), -7, dtype=torch.int32)])
    rows = ids.cuda()[torch.randperm(N, generator=gen, device="cuda")].contiguous()
    want = grads64(dy, h, ad, rows, dtype)
    for name, got in zip(("dh", "dA", "dB"), tim.adapter_logits_backward(dy, h, ad, rows)):
        check(got, *want[name], name)
    tim.check()


def test_as_many_adapters_as_there_can_be():
    n, N, V, D, R = 65535, 300, 24, 16, 8
    z, h, ad, rows = draw(N, V, D, R, n, "bf16", 22)
    rows[:4] = torch.tensor([65534, 0, 65535, 65534], dtype=torch.int32, device="cuda")
    on = live(rows, n)
    some = rows[on].long().unique()
    slot = torch.full((n + 2,), -1, dtype=torch.int32, device="cuda")
    slot[some] = torch.arange(some.numel(), dtype=torch.int32, device="cuda")
    few = tim.Adapters(ad.A[some].contiguous(), ad.B[some].contiguous(), ad.scale[some].contiguous())
    short = torch.where(on, slot[rows.long().clamp(0, n + 1)], -1).to(torch.int32)
    assert torch.equal(bits(tim.adapter_logits(z, h, ad, rows)), bits(tim.adapter_logits(z, h, few, short)))
    dh, dA, dB = tim.adapter_logits_backward(z, h, ad, rows)
    fh, fA, fB = tim.adapter_logits_backward(z, h, few, short)
    tim.check()
    assert torch.equal(dh, fh) and torch.equal(dA[some], fA) and torch.equal(dB[some], fB)
    assert int((dA != 0).any(2).any(1).sum()) <= some.numel() and int((dB != 0).any(2).any(1).sum()) <= some.numel()
    check(tim.adapter_logits(z, h, few, short), *logits64(z, h, few, short, "bf16"))


def test_offsets_past_32_bits():
    """Logits, factors, a table and gradients of more than 2^32 bytes, and 2^31 elements."""
    N, V, D, R, n = 16500, 131072, 64, 64, 270
    gen = torch.Generator(device="cuda").manual_seed(23)
    last = torch.arange(N - 70, N, device="cuda")
    z = torch.zeros((N, V), dtype=torch.bfloat16, device="cuda")
    z[last] = torch.randn((70, V), generator=gen, device="cuda").to(torch.bfloat16)
    h = torch.randn((N, D), generator=gen, device="cuda").to(torch.bfloat16)
    A = torch.zeros((n, R, D), dtype=torch.bfloat16, device="cuda")
    B = torch.zeros((n, V, R), dtype=torch.bfloat16, device="cuda")
    A[-1] = (torch.rand((R, D), generator=gen, device="cuda") * 0.2 - 0.1).to(torch.bfloat16)
    B[-1] = torch.randn((V, R), generator=gen, device="cuda").to(torch.bfloat16)
    rows = torch.full((N,), -1, dtype=torch.int32, device="cuda")
    rows[last] = n - 1
    ad, one = tim.Adapters(A, B), tim.Adapters(A[-1:].contiguous(), B[-1:].contiguous())
    under = torch.zeros(70, dtype=torch.int32, device="cuda")
    dh, dA, dB = tim.adapter_logits_backward(z, h, ad, rows)
    tim.check()
    want = grads64(z[last], h[last], one, under, "bf16")
    check(dh[last], *want["dh"], "dh")
    check(dA[-1:], *want["dA"], "dA")
    check(dB[-1:], *want["dB"], "dB")
    assert not bool(dh[:N - 70].any()) and not bool(dA[:-1].any()) and float(dB[:-1].abs().amax()) == 0
    del dh, dA, dB
    y, tol = logits64(z[last], h[last], one, under, "bf16")
    tim.adapter_logits(z, h, ad, rows, out=z)
    tim.check()
    check(z[last], y, tol)
    assert float(z[:N - 70].abs().amax()) == 0
    del z, A, B, ad, y, tol
    V, D = 1 << 20, 2056
    W = torch.zeros((V, D), dtype=torch.bfloat16, device="cuda")
    W[-3:] = torch.randn((3, D), generator=gen, device="cuda").to(torch.bfloat16)
    t = torch.tensor([V - 1, 0, V - 3, V, V - 2, V - 1], dtype=torch.int32, device="cuda")
    out = tim.embedding(t, W)
    zero = torch.zeros(D, dtype=W.dtype, device="cuda")
    assert torch.equal(out, torch.stack([W[-1], zero, W[-3], zero, W[-2], W[-1]]))
    del W
    dW = tim.embedding_backward(t, out, V)
    tim.check()
    assert torch.equal(dW[-1], 2 * out[0].float()) and torch.equal(dW[-3], out[2].float()) and torch.equal(dW[-2], out[4].float())
    assert float(dW[:-3].abs().amax()) == 0


def test_calls_side_by_side_on_two_streams():
    cases = [draw(700, 3001, 256, 32, 5, "f16", 24), draw(300, 5000, 512, 16, 9, "bf16", 25)]
    tokens = torch.randint(-1, 900, (3000,), device="cuda", dtype=torch.int32)
    g = torch.randn((3000, 257), device="cuda")

    def calls(c):
        return (tim.adapter_logits(*c), *tim.adapter_logits_backward(*c), tim.embedding_backward(tokens, g, 900))

    want = [calls(c) for c in cases]
    torch.cuda.synchronize()
    streams, got = [torch.cuda.Stream(), torch.cuda.Stream()], [[], []]
    for _ in range(5):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i].append(calls(cases[i]))
    torch.cuda.synchronize()
    tim.check()
    for w, g_ in zip(want, got):
        assert all(torch.equal(bits(x), bits(y)) for one in g_ for x, y in zip(w, one))
