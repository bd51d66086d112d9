"""The order of beam selection's candidates whose scores are equal, or no longer differ as
fp64 sums: within a beam the larger logit, then the lower token; else the lower beam."""
import pytest
import torch

from cross_model_kv_transfer_gb300 import kvx

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("V", [300, 9001, 70000])
def test_logits_too_near_for_their_scores(V, dtype):
    """1e-20 beside 0: both less log V are one fp64 number, and the logits are two."""
    logits = torch.zeros((3, V), dtype=dtype, device="cuda")
    for row in logits:
        row[V - 1], row[V // 2], row[3], row[1] = 1e-20, 1e-20, 1e-21, -1e-20
    order = [V // 2, V - 1, 3, 0, 2, 4]
    tokens, parents, new, _ = kvx.beam_select(logits[:1], torch.zeros((1, 1), device="cuda"), beams=6)
    assert tokens.tolist() == [order] and (parents == 0).all() and (new == new[0, 0]).all()
    for n in (1, 2, 3):                  # the last place too
        assert kvx.beam_select(logits[:1], torch.zeros((1, 1), device="cuda"), beams=n)[0].tolist() == [order[:n]]
    # of several beams the lowest
    tokens, parents, _, _ = kvx.beam_select(logits, torch.tensor([[-1.0, 0.0, 0.0]], device="cuda"), beams=6)
    assert tokens.tolist() == [order] and (parents == 1).all()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_ended_beams_beside_equal_scores(dtype):
    """An ended beam's one candidate among others of the same score."""
    logits = torch.full((3, 2), float("-inf"), dtype=dtype, device="cuda")
    logits[0, 1] = logits[2, 0] = 5.0    # the only candidates: log-probability 0
    done = torch.tensor([[False, True, False]], device="cuda")
    tokens, parents, new, ended = kvx.beam_select(logits, torch.full((1, 3), -2.0, device="cuda"), eos=0, done=done)
    assert tokens.tolist() == [[1, 0, 0]] and parents.tolist() == [[0, 1, 2]]
    assert new.tolist() == [[-2.0] * 3] and ended.tolist() == [[False, True, True]]
