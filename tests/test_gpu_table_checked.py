"""The operators beside the head's table under the checked build: the same bits as the
release's, and no check of an index, a copy or a store fails."""
import math

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import rollout_logprob_mismatch_gb300 as tim  # noqa: E402

TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


def bits(x):
    return x.contiguous().view(torch.int32 if x.dtype == torch.float32 else torch.int16)


def twice(calls):
    want = calls()
    tim.check()
    assert tim.tim_debug_build() == 0
    with tim.checked():
        assert tim.tim_debug_build() == 1
        got = calls()
        tim.check()
        assert tim.tim_debug_violation() == ("none", 0, 0)
    assert len(want) == len(got) and all(torch.equal(bits(x), bits(y)) for x, y in zip(want, got))


CASES = [  # N, V, D, R, n, stride past V, offset
    (1, 1000, 64, 8, 1, 0, 0), (17, 333, 72, 16, 3, 0, 0), (70, 4099, 136, 24, 5, 0, 0), (200, 1024, 256, 32, 2, 0, 0),
    (300, 515, 128, 128, 3, 0, 0), (600, 100, 64, 16, 200, 1, 3), (16, 1, 64, 16, 2, 0, 0), (1500, 2999, 64, 64, 2, 1, 1),
    (5000, 24, 64, 40, 2, 0, 0), (300, 24, 16, 8, 65535, 0, 0), (40, 140000, 64, 32, 2, 0, 0), (2500, 700, 520, 16, 1, 8, 0)]


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("N,V,D,R,n,more,offset", CASES)
def test_adapters(N, V, D, R, n, more, offset, dtype):
    gen = torch.Generator(device="cuda").manual_seed(N + V)
    buf = torch.randn(offset + N * (V + more) + 8, generator=gen, device="cuda").to(TYPES[dtype])
    z = torch.as_strided(buf, (N, V), (V + more, 1), offset)
    h = torch.randn((N, D), generator=gen, device="cuda").to(torch.bfloat16)
    A = (torch.randn((n, R, D), generator=gen, device="cuda") / math.sqrt(D)).to(torch.bfloat16)
    B = torch.randn((n, V, R), generator=gen, device="cuda").to(torch.bfloat16)
    ad = tim.Adapters(A, B, torch.rand(n, generator=gen, device="cuda") + 0.5)
    rows = torch.randint(-1, n + 1, (N,), generator=gen, device="cuda", dtype=torch.int32)

    def calls():
        place = z.clone()
        tim.adapter_logits(place, h, ad, rows, out=place)
        return (tim.adapter_logits(z, h, ad, rows), place, *tim.adapter_logits_backward(z, h, ad, rows))

    twice(calls)


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("N,V,D", [(1, 7, 8), (33, 1025, 40), (65, 50, 257), (5000, 3000, 64), (70000, 700, 33)])
def test_embedding(N, V, D, dtype):
    gen = torch.Generator(device="cuda").manual_seed(N)
    W = torch.randn((V, D), generator=gen, device="cuda").to(TYPES[dtype])
    g = torch.randn((N, D), generator=gen, device="cuda").to(TYPES[dtype])
    some = torch.randint(-2, V + 2, (N,), generator=gen, device="cuda", dtype=torch.int32)
    same = torch.full((N,), V - 1, dtype=torch.int32, device="cuda")

    def calls():
        return [f for t in (some, same) for f in (tim.embedding(t, W, 0.7), tim.embedding_backward(t, g, V, 0.7))]

    twice(calls)
