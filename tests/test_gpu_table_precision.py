"""What the operators beside the head's table hold of their values, where a sum's
worst-case bound (tests/test_gpu_table.py) would not show a loss.

Tolerances, from the arithmetic:
  * dB is a sum of chains on the tensor cores, each of at most 48 products of 16 rows, joined
    in fp32.  A product cuts at most a unit, 2^-23, off its chain's running sum.  For values
    of either sign the running sum after i of n products has sqrt(i / n) of the chain's
    norm, so that a chain loses at most 2 / 3 n 2^-23 of its own norm, the chains together
    that of dB's; a join rounds by at most 2^-24 of the running sum, of either sign, and t's
    parts and sums leave less than 2^-21.  A chain over all of an adapter's rows would lose
    in proportion to them.
"""
import math

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import rollout_logprob_mismatch_gb300 as tim  # noqa: E402

F64 = torch.float64
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


# ----------------------------------------------------------------------------- long adapters
def _normal(shape, gen, dtype, size=1.0):
    out = torch.empty(shape, dtype=dtype, device="cuda")
    step = max(1, (1 << 27) // shape[1])
    for i in range(0, shape[0], step):
        out[i:i + step] = torch.randn((min(step, shape[0] - i), shape[1]), generator=gen, device="cuda") * size
    return out


# one tile a slab to as many as there can be, every type's steps, with and without a sum for the low products
LONG = [(9000, 151936, 16, "bf16"), (8200, 151936, 32, "bf16"), (8200, 140000, 64, "bf16"), (8200, 128256, 16, "bf16"),
        (8200, 70000, 128, "bf16"), (8200, 128256, 32, "f32"), (8200, 151936, 16, "f32"), (8200, 75000, 64, "f32"),
        (8200, 151936, 32, "f16"), (8200, 66000, 64, "f16"), (65536, 2048, 16, "bf16"), (65536, 1000, 64, "f32"), (65536, 999, 24, "f16")]


@pytest.mark.parametrize("N,V,R,dtype", LONG)
def test_dB_of_a_long_adapter(N, V, R, dtype):
    gen = torch.Generator(device="cuda").manual_seed(N + V + R)
    D = 256
    dy = _normal((N, V), gen, TYPES[dtype])
    h = torch.randn((N, D), generator=gen, device="cuda").to(torch.bfloat16)
    A = (torch.randn((2, R, D), generator=gen, device="cuda") / math.sqrt(D)).to(torch.bfloat16)
    B = torch.randn((2, V, R), generator=gen, device="cuda").to(torch.bfloat16)
    rows = torch.zeros(N, dtype=torch.int32, device="cuda")
    rows[5::97] = 1
    rows[7::89] = -1
    dh, dA, dB = tim.adapter_logits_backward(dy, h, tim.Adapters(A, B), rows)
    tim.check()
    assert bool(dh.isfinite().all()) and bool(dA.isfinite().all())
    i = torch.nonzero(rows == 0).view(-1)
    t = h[i].to(F64) @ A[0].to(F64).t()
    cols = torch.randperm(V, generator=gen, device="cuda")[:3000]
    want = torch.cat([dy[:, c][i].to(F64).t() @ t for c in cols.split(500)])
    got = dB[0][cols].to(F64)
    products = 48
    joins = N / 512
    bound = 2 / 3 * products * 2.0 ** -23 + math.sqrt(joins) * 2.0 ** -24 + 2.0 ** -21
    error = float((got - want).norm() / want.norm())
    print("dB of %d x %d %s, rank %d: %.2e of %.2e" % (N, V, dtype, R, error, bound))
    assert error <= bound


# ----------------------------------------------------------------------------- parts
def parts(x, k):
    """What k bf16 parts hold of fp32 x, each the rest rounded to nearest."""
    got, left = torch.zeros_like(x, dtype=F64), x.to(F64)
    for _ in range(k):
        p = left.float().to(torch.bfloat16).to(F64)
        got, left = got + p, left - p
    return got


def mantissas(count, bits, gen):
    """fp32 values in [1, 2) of `bits` bits; of 24: values of which two parts leave 2^-18 at least."""
    x = 1 + torch.randint(0, 1 << (bits - 1), (64 * count,), generator=gen).to(F64) * 2.0 ** (1 - bits)
    if bits == 24:
        x = x[(parts(x.float(), 2) - x).abs() >= 2.0 ** -18]
    return x[:count].float()


def powers(shape, gen):
    return (torch.randint(0, 2, shape, generator=gen) * 2 - 1) * 2.0 ** torch.randint(-3, 4, shape, generator=gen)


def singles(M, V, R, dtype, seed):
    """Two adapters of M rows each, R of which (in any order) have one logit, one element of h and
    one rank of their own: every t, du and element of dh, dA, dB is one product, or zero."""
    gen = torch.Generator().manual_seed(seed)
    n, D, N = 2, R + 8, 2 * M + 3
    order = torch.randperm(N, generator=gen)
    rows, h, dy = torch.full((N,), -1, dtype=torch.int32), torch.zeros((N, D)), torch.zeros((N, V))
    A, B, scale = torch.zeros((n, R, D)), torch.zeros((n, V, R)), mantissas(n, 24, gen)
    bits = {"f32": 24, "bf16": 8, "f16": 11}[dtype]
    at = []
    for a in range(n):
        mine = order[a * M:(a + 1) * M]
        rows[mine] = a
        i, r = mine[torch.randperm(M, generator=gen)[:R]], torch.arange(R)
        v = torch.randperm(V, generator=gen)[:R]
        v[0] = V - 1 if not bool((v[1:] == V - 1).any()) else v[0]
        h[i, r], A[a, r, r], B[a, v, r] = powers((R,), gen), powers((R,), gen), powers((R,), gen)
        dy[i, v] = (mantissas(R, bits, gen) * powers((R,), gen)).float()
        at.append((i, v, r))
    ad = tim.Adapters(A.to(torch.bfloat16).cuda(), B.to(torch.bfloat16).cuda(), scale.cuda())
    return dy.to(TYPES[dtype]).cuda(), h.to(torch.bfloat16).cuda(), ad, rows.cuda(), at


def off(got, want):
    return float(((got.to(F64) - want) / want).abs().max())


SINGLES = [(300, 130, 16), (150, 1000, 32), (200, 700, 64), (140, 300, 128), (60, 400, 24), (300, 33000, 16), (70, 33000, 40),
           (100, 70000, 32), (100, 70000, 64), (150, 70000, 128), (40, 140000, 8), (50, 140000, 32), (80, 140000, 64)]


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("M,V,R", SINGLES)
def test_gradient_of_single_products(M, V, R, dtype):
    """t, du and fp32 dlogits are held to 2^-24.  dB: what their three parts leave, the products
    of parts that are left out, six cuts and the sums' joins: below 2^-19.  dA, dh: three cuts or
    roundings of du's planes, one with the scale, what du's parts leave and three cuts: below 2^-20.
    Two parts of any of them leave 2^-18 and more."""
    dy, h, ad, rows, at = singles(M, V, R, dtype, M + V + R)
    dh, dA, dB = tim.adapter_logits_backward(dy, h, ad, rows)
    tim.check()
    zero_h, zero_A, zero_B = dh.clone(), dA.clone(), dB.clone()
    for a, (i, v, r) in enumerate(at):
        d, s = dy[i, v].to(F64), ad.scale[a].to(F64)
        x, w, b = h[i, r].to(F64), ad.A[a, r, r].to(F64), ad.B[a, v, r].to(F64)
        t, du = s * x * w, s * b * d
        assert off(dB[a, v, r], d * t) <= 2.0 ** -19
        assert off(dA[a, r, r], du * x) <= 2.0 ** -20 and off(dh[i, r], du * w) <= 2.0 ** -20
        short = parts((s * x * w).float().cpu(), 2).cuda()   # the bounds tell: t, then dlogits and du, in two parts
        assert off(d * short, d * t) > 2.0 ** -19
        assert off(parts(du.float().cpu(), 2).cuda() * x, du * x) > 2.0 ** -20
        if dtype == "f32":
            assert off(parts(dy[i, v].cpu(), 2).cuda() * t, d * t) > 2.0 ** -19
        zero_h[i, r], zero_A[a, r, r], zero_B[a, v, r] = 0, 0, 0
    assert not bool(zero_h.any()) and not bool(zero_A.any()) and not bool(zero_B.any())


@pytest.mark.parametrize("M,V,R", SINGLES)
def test_fp32_logits_of_single_products(M, V, R):
    """t of fp32 logits is held to 2^-24; three cuts, one rounding: below 2^-21."""
    dy, h, ad, rows, at = singles(M, V, R, "f32", M + V + R)
    out = tim.adapter_logits(torch.zeros_like(dy), h, ad, rows)
    tim.check()
    for a, (i, v, r) in enumerate(at):
        t, b = ad.scale[a].to(F64) * h[i, r].to(F64) * ad.A[a, r, r].to(F64), ad.B[a, v, r].to(F64)
        assert off(out[i, v], t * b) <= 2.0 ** -21
        assert off(parts(t.float().cpu(), 2).cuda() * b, t * b) > 2.0 ** -21
        out[i, v] = 0
    assert not bool(out.any())


@pytest.mark.parametrize("R", [16, 32, 64, 128])
@pytest.mark.parametrize("x", [3.4e38, -3.3961e38, 3.392e38])
def test_values_between_bf16s_largest_and_fp32s(x, R):
    """Finite fp32 values that a bf16 part rounds to infinity, or whose rest it loses."""
    N, V, D = 3, 200, 64
    rows = torch.tensor([0, -1, 0], dtype=torch.int32, device="cuda")
    z = torch.zeros((N, V), device="cuda")
    h, A, B = torch.zeros((N, D), device="cuda"), torch.zeros((1, R, D), device="cuda"), torch.zeros((1, V, R), device="cuda")
    h[2, 5], A[0, 3, 5], B[0, 150, 3] = 1.0, 1.0, 2.0 ** -20
    h, A, B = (y.to(torch.bfloat16) for y in (h, A, B))
    big = torch.full((1,), x, device="cuda")
    value = float(big.to(F64))
    out = tim.adapter_logits(z, h, tim.Adapters(A, B, big), rows)
    assert abs(float(out[2, 150].to(F64)) / (value * 2.0 ** -20) - 1) <= 2.0 ** -21 and int((out != 0).sum()) == 1
    # t, then du, of that size; then dlogits
    dy = z.clone()
    dy[2, 150] = 2.0 ** -4
    dh, dA, dB = tim.adapter_logits_backward(dy, h, tim.Adapters(A, B * 16, big), rows)
    assert abs(float(dB[0, 150, 3].to(F64)) / (value * 2.0 ** -4) - 1) <= 2.0 ** -19
    dh, dA, dB = tim.adapter_logits_backward(dy, h * 2.0 ** -6, tim.Adapters(A * 2.0 ** -6, B * 2.0 ** 24, big), rows)
    assert abs(float(dA[0, 3, 5].to(F64)) / (value * 2.0 ** -6) - 1) <= 2.0 ** -20
    assert abs(float(dh[2, 5].to(F64)) / (value * 2.0 ** -6) - 1) <= 2.0 ** -20
    dy[2, 150] = big[0]
    dh, dA, dB = tim.adapter_logits_backward(dy, h, tim.Adapters(A * 2.0 ** -20, B), rows)
    tim.check()
    assert abs(float(dB[0, 150, 3].to(F64)) / (value * 2.0 ** -20) - 1) <= 2.0 ** -19
    assert abs(float(dA[0, 3, 5].to(F64)) / (value * 2.0 ** -20) - 1) <= 2.0 ** -20
    for got in (dh, dA, dB):
        assert int((got != 0).sum()) == 1


@pytest.mark.parametrize("N,V,R,dtype", [(6000, 1500, 16, "bf16"), (3000, 70000, 64, "f16"), (5000, 300, 24, "f32")])
def test_long_adapters_in_graphs_and_on_two_streams(N, V, R, dtype):
    """dB's later chains add to what the first one wrote: replayed, and beside another call's."""
    gen = torch.Generator(device="cuda").manual_seed(N)
    dy, h = _normal((N, V), gen, TYPES[dtype]), torch.randn((N, 128), generator=gen, device="cuda").to(torch.bfloat16)
    A, B = (torch.randn(s, generator=gen, device="cuda").to(torch.bfloat16) for s in ((2, R, 128), (2, V, R)))
    ad, rows = tim.Adapters(A, B), torch.randint(-1, 2, (N,), generator=gen, device="cuda", dtype=torch.int32)
    other = rows.flip(0).contiguous()
    want = [tim.adapter_logits_backward(dy, h, ad, r) for r in (rows, other)]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = tim.adapter_logits_backward(dy, h, ad, rows)
    for _ in range(3):
        for x in out:
            x.fill_(7)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(out, want[0]))
    streams, got = [torch.cuda.Stream(), torch.cuda.Stream()], [[], []]
    for _ in range(4):
        for k, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[k].append(tim.adapter_logits_backward(dy, h, ad, (rows, other)[k]))
    torch.cuda.synchronize()
    tim.check()
    for k in range(2):
        assert all(torch.equal(x, y) for one in got[k] for x, y in zip(one, want[k]))
