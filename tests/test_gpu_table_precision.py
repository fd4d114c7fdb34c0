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
