"""Host-side refusals of the operators on a head's logits at the ends of their
ranges (no GPU: every call here is refused before any CUDA call)."""
import pytest

import rollout_logprob_mismatch_gb300 as tim
from rollout_logprob_mismatch_gb300 import build as tim_build

E = tim.TIM_ERR_INVALID_ARG
P, Q = 1 << 20, 1 << 40   # aligned addresses that are never dereferenced


@pytest.fixture(scope="module", autouse=True)
def lib():
    tim_build.build()
    return tim.load()


def test_rows_past_the_address_space():
    """A stride in its range times a row count in its range may pass 64 bits: no logits
    reach that far, and no check may be made on what is left of the product."""
    far = (P, 0, (1 << 31) - 1, 100, 1 << 40)
    assert tim.tim_process_logits(*far, None, Q, 0, 100, None) == E
    assert "address" in tim.tim_last_error()
    assert tim.tim_processed_logprob(*far, None, Q, Q, Q, None) == E
    assert tim.tim_processed_logprob_backward(*far, None, Q, Q, Q, Q, 100, None) == E
    assert tim.tim_distill_topk(*far, Q, Q, None, 4, 1.0, Q, Q, None, None) == E
    assert tim.tim_distill_topk_backward(*far, Q, Q, None, 4, 1.0, Q, Q, None, Q, 100, None) == E
    assert tim.tim_distill_topk_step(*far, Q, Q, None, 4, 1.0, Q, Q, Q, None, Q, 100, None) == E
    near = (P, 0, (1 << 31) - 1, 100, 100)
    assert tim.tim_process_logits(*near, None, Q, 0, 1 << 40, None) == E
    assert "address" in tim.tim_last_error()
    assert tim.tim_process_logits(P, 2, 1 << 22, 100, 1 << 38, None, Q, 2, 100, None) == E
