"""Host-side argument checks and struct layout of the operators on a head's
logits (no GPU: every call here is refused before any CUDA call, or empty)."""
import ctypes
import math
import os
import subprocess

import numpy as np
import pytest

import logits_ref as ref
import rollout_logprob_mismatch_gb300 as tim
from rollout_logprob_mismatch_gb300 import build as tim_build

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
E = tim.TIM_ERR_INVALID_ARG
P = 1 << 20   # an aligned address that is never dereferenced


@pytest.fixture(scope="module", autouse=True)
def lib():
    tim_build.build()
    return tim.load()


def test_struct_layout(tmp_path):
    names = [n for n, _ in tim.tim_logits_rules._fields_]
    src = tmp_path / "l.c"
    src.write_text('#include <stdio.h>\n#include <stddef.h>\n#include "tim.h"\nint main(void){printf("%zu", sizeof(tim_logits_rules));'
                   + "".join('printf(" %%zu", offsetof(tim_logits_rules, %s));' % n for n in names)
                   + "return TIM_F32 == 0 && TIM_BF16 == 1 && TIM_F16 == 2 && TIM_DISTILL_MAX_K == 1024 ? 0 : 1;}\n")
    exe = tmp_path / "l"
    subprocess.run(["gcc", "-std=c99", "-Wall", "-Werror", "-I", os.path.join(ROOT, "include"), str(src), "-o", str(exe)],
                   check=True)
    out = subprocess.run([str(exe)], check=True, capture_output=True, text=True).stdout
    S = tim.tim_logits_rules
    assert [int(x) for x in out.split()] == [ctypes.sizeof(S)] + [getattr(S, n).offset for n in names]


HEADS = [(P, 3, 4, 100, 100), (P, 0, -1, 100, 100), (P, 0, 1 << 31, 100, 100), (P, 0, 4, 0, 100),
         (P, 0, 4, (1 << 20) + 1, 1 << 21), (P, 0, 4, 100, 99), (None, 0, 4, 100, 100), (P + 2, 0, 4, 100, 100),
         (P + 1, 1, 4, 100, 100), (P, 0, (1 << 31) - 1, 2048, 2048)]


@pytest.mark.parametrize("head", HEADS)
def test_bad_logits(head):
    Q = 1 << 40
    assert tim.tim_process_logits(*head, None, Q, 0, 100, None) == E
    assert tim.tim_processed_logprob(*head, None, Q, Q, Q, None) == E
    assert tim.tim_processed_logprob_backward(*head, None, Q, Q, Q, Q, 100, None) == E
    assert tim.tim_distill_topk(*head, Q, Q, None, 4, 1.0, Q, Q, None, None) == E
    assert tim.tim_distill_topk_backward(*head, Q, Q, None, 4, 1.0, Q, Q, None, Q, 100, None) == E
    assert tim.tim_distill_topk_step(*head, Q, Q, None, 4, 1.0, Q, Q, Q, None, Q, 100, None) == E
    assert tim.tim_last_error()


def test_bad_outputs_and_arrays():
    head, Q = (P, 1, 4, 100, 128), 1 << 40
    call = tim.tim_process_logits
    assert call(*head, None, None, 1, 100, None) == E
    assert call(*head, None, Q, 2, 100, None) == E           # bf16 -> fp16 is not offered
    assert call(*head, None, Q, 1, 99, None) == E
    assert call(*head, None, Q + 1, 1, 100, None) == E
    assert call(*head, None, P, 0, 128, None) == E           # fp32 over the bf16 logits
    assert call(*head, None, P, 1, 100, None) == E           # over the logits at another stride
    assert call(*head, None, P + 2 * 483, 1, 128, None) == E  # overlaps the last row
    assert "overlaps" in tim.tim_last_error()
    assert tim.tim_processed_logprob(*head, None, None, Q, Q, None) == E
    assert tim.tim_processed_logprob(*head, None, Q, Q + 2, Q, None) == E
    assert tim.tim_processed_logprob_backward(*head, None, Q, None, Q, Q, 100, None) == E
    for K in (0, 1025):
        assert tim.tim_distill_topk(*head, Q, Q, None, K, 1.0, Q, Q, None, None) == E
    for tau in (0.0, -1.0, math.nan, math.inf, 1e-45):
        assert tim.tim_distill_topk(*head, Q, Q, None, 4, tau, Q, Q, None, None) == E
    assert tim.tim_distill_topk(*head, None, Q, None, 4, 1.0, Q, Q, None, None) == E
    assert tim.tim_distill_topk(*head, Q, Q, Q, 4, 1.0, Q, Q, None, None) == E      # a tail needs lse_tail
    assert tim.tim_distill_topk_backward(*head, Q, Q, Q, 4, 1.0, Q, Q, None, Q, 100, None) == E
    assert tim.tim_distill_topk_step(*head, Q, Q, None, 4, 1.0, None, Q, Q, None, Q, 100, None) == E


@pytest.mark.parametrize("fields", [
    {"num_history": -1}, {"num_history": 1 << 30}, {"num_bias": -1}, {"num_bias": 1 << 30}, {"num_allowed": -1}, {"history_spans": P, "num_history": 3},
    {"bias_offsets": P, "num_bias": 2, "bias_ids": P}, {"allowed": P, "allowed_stride": 3, "num_allowed": 4},
    {"allowed": P, "allowed_stride": 4, "num_allowed": 3}, {"allowed_rows": P}, {"temperature": P + 2}])
def test_bad_rules(fields):
    r = tim.tim_logits_rules()
    for k, v in fields.items():
        setattr(r, k, v)
    assert tim.tim_process_logits(P, 0, 4, 100, 100, ctypes.byref(r), 1 << 40, 0, 100, None) == E
    assert tim.tim_last_error()


def test_empty_batches_are_no_ops():
    head = (None, 0, 0, 100, 100)
    assert tim.tim_process_logits(*head, None, None, 0, 100, None) == tim.TIM_OK
    assert tim.tim_processed_logprob(*head, None, None, None, None, None) == tim.TIM_OK
    assert tim.tim_processed_logprob_backward(*head, None, None, None, None, None, 100, None) == tim.TIM_OK
    assert tim.tim_distill_topk(*head, None, None, None, 4, 1.0, None, None, None, None) == tim.TIM_OK


def test_the_reference_formulas_agree_with_differences():
    """The fp64 gradients the GPU tests compare with, against central differences
    of the fp64 forward (error h^2 / 6 times a third derivative below 1, and u / h)."""
    rng = np.random.default_rng(3)
    V, h = 19, 1e-4
    z = rng.normal(0, 2, (1, V)) + 0.01
    r = {"temperature": np.array([0.8]), "repetition": np.array([1.3]), "presence": np.array([0.4]),
         "frequency": np.array([0.2]), "history": np.array([1, 2, 2, 5, 5, 5], np.int32),
         "history_spans": np.array([[0, 2, 6]], np.int32), "allowed": np.array([[0x7ffdf]], np.int32),
         "bias_offsets": np.array([0, 2]), "bias_ids": np.array([2, 7]), "bias_values": np.array([1.5, -2.0])}
    t = np.array([2], np.int32)
    lse = ref.logprob_ref(z, r, t)[1]
    d, _ = ref.backward_ref(z, r, t, np.ones(1), lse, "f32")
    ids, tl, tlse = np.array([[3, 9, -1, 11]], np.int32), np.array([[1.0, 0.5, 9.0, -1.0]]), np.array([2.0])
    dd = {tail: ref.distill_ref(z, ids, tl, tlse if tail else None, 0.7, np.ones(1))["dlogits"] for tail in (0, 1)}
    for v in range(V):
        e = np.zeros((1, V))
        e[0, v] = h
        num = (ref.logprob_ref(z + e, r, t)[0] - ref.logprob_ref(z - e, r, t)[0]) / (2 * h)
        assert abs(num[0] - d[0, v]) <= 1e-7, v
        for tail in (0, 1):
            f = [ref.distill_ref(z + s * e, ids, tl, tlse if tail else None, 0.7)["loss"][0] for s in (1, -1)]
            assert abs((f[0] - f[1]) / (2 * h) - dd[tail][0, v]) <= 1e-7, (tail, v)


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
def test_the_rounding_bound_is_half_a_unit(dtype):
    """Correctly rounded values stay within the bound, and reach 0.99 of it."""
    torch = pytest.importorskip("torch")
    x = torch.from_numpy(np.random.default_rng(1).uniform(1, 4, 100000))
    y = x.to({"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}[dtype]).double()
    ratio = ((y - x).abs().numpy() / ref.rounding(x.numpy(), dtype))
    assert 0.99 < ratio.max() <= 1.0
