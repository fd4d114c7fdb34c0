"""Edges of the operators on a head's logits: rows whose probabilities, masks or
lists leave nothing on one side, values at the types' limits, long segments in
place, outputs on other streams."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import rollout_logprob_mismatch_gb300 as tim  # noqa: E402
from test_gpu_logits import dev, draw_logits, draw_teacher  # noqa: E402


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
