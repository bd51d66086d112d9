"""Beam search on transferred prompts as examples/beams_after_transfer.py runs it: every
attention against fp64 of the beam's whole sequence, every selection against a sort, the
pages against rows that are walked one by one, and what a beam's pages hold against the
same tokens written one after another into a cache of its own."""
import os
import sys

import numpy as np
import pytest
import torch

import continuation_reference as cref
from cross_model_kv_transfer_gb300 import kvx
from test_gpu_attend8_shared import compare

pytestmark = pytest.mark.gpu
sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
import beams_after_transfer as example  # noqa: E402


@pytest.mark.parametrize("prompts,beams,steps", [((70, 200), 4, (9, 10)), ((33,), 3, (20, 3)), ((16, 5, 90), 1, (3, 4))])
def test_every_step(prompts, beams, steps):
    seen = {"attend": 0, "select": 0, "fork": 0, "compact": 0}
    layers, written = 2, {}

    def watch(stage, **t):
        seen[stage] += 1
        host = {k: v.cpu().numpy() if torch.is_tensor(v) and v.dtype != torch.bfloat16 else v for k, v in t.items()}
        if stage == "attend":
            c = t["cache"]
            parts = [cref.Joined(codes.cpu().numpy(), scale.cpu().numpy())
                     for codes, scale in ((c.k_codes, c.k_scale), (c.v_codes, c.v_scale))]
            R = len(host["lens"])
            want = cref.shared_attend(t["q"].double().cpu().numpy(), *parts, host["prefix"], host["before"],
                                      host["groups"], host["table"], host["lens"], range(R + 1),
                                      c.head_dim ** -0.5)
            compare(t["out"], t["lse"], want, True, max(prompts) + sum(steps))
            # the keys and values of each row's history, for the last check
            rows = written.setdefault(t["layer"], [[] for _ in range(R)])
            for r in range(R):
                rows[r] = rows[r] + [(t["k"][r].clone(), t["v"][r].clone())]
            if t["layer"] == layers - 1:
                check_pages(t["cache"], rows, t["table"], t["lens"])
        elif stage == "select":
            B, K = host["scores"].shape
            x = t["logits"].double().cpu().numpy()
            for b in range(B):
                tokens, parents, scores = cref.beam(x[b * K:(b + 1) * K], host["scores"][b], host["done"][b], K, 1)
                assert host["tokens"][b].tolist() == tokens
                assert host["parents"][b].tolist() == [b * K + p for p in parents]
                assert np.abs(host["new_scores"][b] - scores).max() <= 2.0 ** -17 + 2.0 ** -24 * np.abs(scores).max()
        elif stage == "fork":
            parents = host["parents"]
            want = [[x if i < -(-n // 16) else -1 for i, x in enumerate(host["old"][p])]
                    for p, n in zip(parents, host["old_lens"][parents])]
            assert host["table"].tolist() == want and (host["lens"] == host["old_lens"][parents]).all()
            check_refs(t["pages"], t["table"], t["prefix"])
            for layer in written:
                written[layer] = [written[layer][p] for p in parents]
        else:
            check_refs(t["pages"], t["table"], t["prefix"])
            assert int(t["used"].item()) == int((t["pages"].refs > 0).sum().item())
            assert (t["pages"].refs[int(t["used"].item()):] == 0).all()
            for layer in written:
                written[layer] = written[layer][beams:]

    history, scores, flags = example.run(prompts=prompts, layers=layers, beams=beams, steps=steps, watch=watch)
    assert flags == 0
    left = max(1, len(prompts) - 1)
    assert history.shape == (left * beams, sum(steps)) and scores.shape == (left, beams)
    assert seen["attend"] == layers * sum(steps) and seen["select"] == seen["fork"] == sum(steps)
    assert seen["compact"] == (len(prompts) > 1)
    # beams of one prompt differ, and their scores fall
    for b in range(left):
        assert len({tuple(h) for h in history[b * beams:(b + 1) * beams].tolist()}) == beams
        assert (scores[b].diff() <= 0).all()


def check_refs(pages, table, prefix):
    held = torch.cat([table[table >= 0], prefix[prefix >= 0]]).long()
    assert torch.equal(pages.refs, torch.bincount(held, minlength=pages.num_blocks).int())


def check_pages(cache, rows, table, lens):
    """A row's pages hold what its tokens, written one by one, leave in a cache of its own."""
    bs = cache.block_size
    for r, tokens in enumerate(rows):
        n = len(tokens)
        assert int(lens[r].item()) == n
        alone = kvx.Cache8.empty(-(-n // bs), cache.heads, cache.head_dim, bs)
        own = torch.arange(-(-n // bs), dtype=torch.int32, device="cuda")[None]
        for j, (k, v) in enumerate(tokens):
            alone.write(k[None], v[None], own, start=torch.tensor([j], dtype=torch.int32, device="cuda"))
        pages = table[r, :own.shape[1]].long()
        for a, b in ((alone.k_codes, cache.k_codes), (alone.v_codes, cache.v_codes)):
            got = b[pages].transpose(1, 2).reshape(-1, cache.heads, cache.head_dim)[:n]
            want = a.transpose(1, 2).reshape(-1, cache.heads, cache.head_dim)[:n]
            assert torch.equal(got, want)
        assert torch.equal(cache.k_scale[pages], alone.k_scale) and torch.equal(cache.v_scale[pages], alone.v_scale)
