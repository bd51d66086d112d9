"""The beam-search example with fewer candidates than beams: rows without one hold no
tokens, and the others their own."""
import os
import sys

import pytest
import torch

pytestmark = pytest.mark.gpu
sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
import beams_after_transfer as example  # noqa: E402


@pytest.mark.parametrize("prompts,beams,vocab,steps", [((20, 33), 4, 2, (2, 2)), ((18,), 8, 3, (3, 1)),
                                                       ((5, 16, 40), 5, 4, (1, 1))])
def test_rows_without_a_candidate_hold_no_tokens(prompts, beams, vocab, steps):
    rows, none = [[] for _ in range(len(prompts) * beams)], []

    def watch(stage, **t):
        nonlocal rows
        if stage == "select":
            tokens, parents = t["tokens"].view(-1).tolist(), t["parents"].view(-1).tolist()
            none.append(parents.count(-1))
            rows = [rows[p] + [x] if p >= 0 else [-1] * (len(rows[0]) + 1) for p, x in zip(parents, tokens)]
        elif stage == "compact":
            rows = rows[beams:]

    history, scores, flags = example.run(prompts=prompts, layers=1, beams=beams, steps=steps, vocab=vocab, watch=watch)
    assert flags == 0 and none[0] == len(prompts) * (beams - vocab)
    assert history.tolist() == rows
    empty = torch.isneginf(scores).view(-1).tolist()
    assert [h == [-1] * sum(steps) for h in history.tolist()] == empty
