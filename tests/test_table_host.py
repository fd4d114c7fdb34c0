"""Host-side argument checks and struct layout of the operators beside the head's
table (no GPU: every call here is refused before any CUDA call, or empty)."""
import ctypes
import math
import os
import subprocess

import pytest

import rollout_logprob_mismatch_gb300 as tim
from rollout_logprob_mismatch_gb300 import build as tim_build

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
E = tim.TIM_ERR_INVALID_ARG
P = 1 << 20   # aligned addresses that are never dereferenced
Q, S, T, U = 1 << 40, 1 << 41, 1 << 42, 1 << 43


@pytest.fixture(scope="module", autouse=True)
def lib():
    tim_build.build()
    return tim.load()


def adapters(A=S, B=T, scale=None, rank=16, n=2):
    d = tim.tim_adapters()
    d.A, d.B, d.scale, d.rank, d.num_adapters = A, B, scale, rank, n
    return ctypes.byref(d)


def test_struct_layout(tmp_path):
    names = [n for n, _ in tim.tim_adapters._fields_]
    src = tmp_path / "l.c"
    src.write_text('#include <stdio.h>\n#include <stddef.h>\n#include "tim.h"\nint main(void){printf("%zu", sizeof(tim_adapters));'
                   + "".join('printf(" %%zu", offsetof(tim_adapters, %s));' % n for n in names)
                   + "return TIM_ADAPTER_MAX_RANK == 128 && TIM_ADAPTER_MAX_COUNT == 65535 ? 0 : 1;}\n")
    exe = tmp_path / "l"
    subprocess.run(["gcc", "-std=c99", "-Wall", "-Werror", "-I", os.path.join(ROOT, "include"), str(src), "-o", str(exe)],
                   check=True)
    out = subprocess.run([str(exe)], check=True, capture_output=True, text=True).stdout
    C = tim.tim_adapters
    assert [int(x) for x in out.split()] == [ctypes.sizeof(C)] + [getattr(C, n).offset for n in names]
    assert (tim.ADAPTER_MAX_RANK, tim.ADAPTER_MAX_COUNT) == (128, 65535)


HEADS = [(P, 3, 4, 100, 100), (P, 0, -1, 100, 100), (P, 0, 1 << 30, 1, 1), (P, 0, 4, 0, 100),
         (P, 0, 4, (1 << 20) + 1, 1 << 21), (P, 0, 4, 100, 99), (None, 0, 4, 100, 100), (P + 2, 0, 4, 100, 100),
         (P + 1, 1, 4, 100, 100)]
HEAD = (P, 0, 4, 100, 100)


def forward(head=HEAD, h=Q, D=64, ad=None, rows=Q + 4096, out=U, stride=100):
    return tim.tim_adapter_logits(*head, h, D, adapters() if ad is None else ad, rows, out, stride, None)


def backward(head=HEAD, h=Q, D=64, ad=None, rows=Q + 4096, dh=U, dA=U + (1 << 20), dB=U + (1 << 21)):
    return tim.tim_adapter_logits_backward(*head, h, D, adapters() if ad is None else ad, rows, dh, dA, dB, 0, 0, None)


@pytest.mark.parametrize("head", HEADS)
def test_bad_logits(head):
    assert forward(head) == E and backward(head) == E
    assert tim.tim_last_error()


@pytest.mark.parametrize("bad", [dict(rank=0), dict(rank=4), dict(rank=12), dict(rank=136), dict(n=-1), dict(n=65536),
                                 dict(A=None), dict(B=None), dict(A=S + 8), dict(B=T + 2), dict(scale=2)])
def test_bad_adapters(bad):
    assert forward(ad=adapters(**bad)) == E
    assert backward(ad=adapters(**bad)) == E


@pytest.mark.parametrize("bad", [dict(D=0), dict(D=12), dict(D=65544), dict(h=None), dict(h=Q + 8), dict(rows=None),
                                 dict(rows=Q + 2)])
def test_bad_rows(bad):
    assert forward(**bad) == E
    assert backward(**bad) == E


def test_null_adapters():
    assert tim.tim_adapter_logits(*HEAD, Q, 64, None, Q, U, 100, None) == E
    assert tim.tim_adapter_logits_backward(*HEAD, Q, 64, None, Q, U, U, U, 0, 0, None) == E


def test_bad_outputs():
    assert forward(out=None) == E
    assert forward(stride=99) == E
    assert forward(out=P + 400) == E                       # overlaps without being the logits
    for over in (Q, Q + 4096, S, T):                        # h, rows, A, B
        assert forward(out=over) == E
    assert forward(ad=adapters(scale=U + 64)) == E
    for k in ("dh", "dA", "dB"):
        assert backward(**{k: None}) == E
        assert backward(**{k: U + 8}) == E
        for over in (P, Q, Q + 4096, S, T):
            assert backward(**{k: over}) == E
    assert backward(dh=U, dA=U) == E


def test_empty_adapter_calls():
    empty = (None, 1, 0, 100, 100)
    assert tim.tim_adapter_logits(*empty, None, 64, adapters(n=0, A=None, B=None), None, None, 100, None) == 0
    assert tim.tim_adapter_logits(*empty, None, 64, adapters(), None, None, 100, None) == 0
    assert tim.tim_adapter_logits(*empty, None, 60, adapters(), None, None, 100, None) == E
    # in place without adapters: nothing to do
    assert tim.tim_adapter_logits(*HEAD, Q, 64, adapters(n=0, A=None, B=None), Q, P, 100, None) == 0
    assert tim.tim_adapter_logits_backward(*empty, None, 64, adapters(n=0, A=None, B=None), None, None, None, None, 0, 0,
                                           None) == 0


def lookup(tokens=Q, N=4, W=P, dtype=1, V=100, D=64, scale=1.0, out=U, out_dtype=1):
    return tim.tim_embedding(tokens, N, W, dtype, V, D, scale, out, out_dtype, None)


def gradient(tokens=Q, N=4, grad=P, dtype=1, V=100, D=64, scale=1.0, dW=U, accumulate=0):
    return tim.tim_embedding_backward(tokens, N, grad, dtype, V, D, scale, dW, accumulate, None)


@pytest.mark.parametrize("bad", [dict(tokens=None), dict(tokens=Q + 2), dict(N=-1), dict(N=1 << 30), dict(dtype=3),
                                 dict(V=0), dict(V=(1 << 20) + 1), dict(D=0), dict(D=65537), dict(N=1 << 24, D=65536),
                                 dict(scale=math.inf), dict(scale=math.nan)])
def test_bad_embedding_arguments(bad):
    assert lookup(**bad) == E and gradient(**bad) == E


def test_bad_embedding_buffers():
    for bad in (dict(W=None), dict(W=P + 1), dict(out=None), dict(out=U + 1), dict(out_dtype=3), dict(out_dtype=-1),
                dict(out=P + 128), dict(out=Q)):
        assert lookup(**bad) == E, bad
    for bad in (dict(grad=None), dict(grad=P + 1), dict(dW=None), dict(dW=U + 2), dict(dW=P), dict(dW=Q)):
        assert gradient(**bad) == E, bad


def test_empty_embedding_calls():
    assert lookup(tokens=None, N=0, W=None, out=None) == 0
    assert gradient(tokens=None, N=0, grad=None, accumulate=1) == 0
    assert gradient(tokens=None, N=0, grad=None, dW=None, accumulate=1) == E


def test_wrappers_refuse_cpu_tensors():
    torch = pytest.importorskip("torch")
    z, h = torch.zeros(4, 100), torch.zeros(4, 64, dtype=torch.bfloat16)
    ad = tim.Adapters(torch.zeros(1, 16, 64, dtype=torch.bfloat16), torch.zeros(1, 100, 16, dtype=torch.bfloat16))
    rows = torch.zeros(4, dtype=torch.int32)
    with pytest.raises(ValueError):
        tim.adapter_logits(z, h, ad, rows)
    with pytest.raises(ValueError):
        tim.adapter_logits_backward(z, h, ad, rows)
    with pytest.raises(ValueError):
        tim.embedding(rows, z)
    with pytest.raises(ValueError):
        tim.embedding_backward(rows, z, 100)
