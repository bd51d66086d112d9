"""Beam search's selection (kvx_beam_select) against fp64: tokens and parents equal,
scores to fp32's rounding.

Tolerances.  A row's sum of exponentials: arguments (x - max) log2 e are off by 2^-23
of themselves, for terms that count (within 16 of the maximum in base 2) 2^-19 at most
and by far less where most of the sum is, the exponential by 2^-22, the fp32
additions by 2^-24 each over 75 terms a thread at most: 2^-17 of the sum is a bound,
and 2^-17 + 2^-24 |score| one of a score.  The inputs' candidates are further apart
than twice that where they belong to different beams (checked), so that tokens and
parents have one right answer."""
import numpy as np
import pytest
import torch

import continuation_reference as cref
from cross_model_kv_transfer_gb300 import kvx

pytestmark = pytest.mark.gpu


def check(logits, scores, n, eos=None, done=None, **kw):
    B, K = scores.shape
    tokens, parents, new, new_done = kvx.beam_select(logits, scores, beams=n, eos=eos, done=done, **kw)
    assert tokens.shape == parents.shape == new.shape == (B, n)
    x, s = logits.double().cpu().numpy(), scores.double().cpu().numpy()
    for b in range(B):
        more = cref.beam(x[b * K:(b + 1) * K], s[b], None if done is None else done[b].tolist(), n + 1, eos)
        t, p, v = (list(y[:n]) for y in more)
        apart = [abs(a - c) for a, c, i, j in zip(more[2], more[2][1:], more[1], more[1][1:]) if i != j]
        assert not apart or min(apart) == 0 or min(a for a in apart if a) > 2.0 ** -15, "candidates too near each other"
        fill = n - len(t)
        assert tokens[b].tolist() == t + [-1] * fill
        assert parents[b].tolist() == [b * K + k for k in p] + [-1] * fill
        got = new[b].double().cpu().numpy()
        assert np.isneginf(got[len(v):]).all()
        v = np.array(v)
        assert (np.abs(got[:len(v)] - v) <= 2.0 ** -17 + 2.0 ** -24 * np.abs(v)).all()
        if eos is not None:
            assert new_done[b].tolist() == [y == eos for y in t] + [False] * fill
    if eos is None:
        assert new_done is None
    return tokens, parents, new, new_done


def draw(B, K, V, dtype, seed, spread=3.0):
    g = torch.Generator().manual_seed(seed)
    logits = (spread * torch.randn((B * K, V), generator=g)).to(dtype).cuda()
    return logits, (-9.0 + 2.0 * torch.randn((B, K), generator=g)).cuda()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("B,K,n,V", [
    (1, 1, 1, 1), (1, 1, 4, 2), (2, 3, 5, 7), (3, 2, 2, 50), (1, 4, 4, 1000), (2, 8, 8, 4099),
    (1, 32, 32, 300), (2, 5, 17, 8192), (1, 2, 32, 33333), (1, 3, 3, 128256), (4, 1, 6, 70000),
    (1, 2, 7, 262144)])
def test_matches_fp64(B, K, n, V, dtype):
    check(*draw(B, K, V, dtype, 3 * V + K), n)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("eos", [0, 6, 499])
def test_ended_beams(eos, dtype):
    logits, scores = draw(4, 5, 500, dtype, 11)
    done = torch.rand((4, 5), generator=torch.Generator().manual_seed(2)) < 0.4
    done[3] = True
    scores[1, 0] = float("-inf")
    check(logits, scores, 5, eos, done.cuda())
    check(logits, scores, 9, eos, done.cuda())
    check(logits, scores, 5, eos)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_the_first_step(dtype):
    """All beams alike but for their scores: one beam goes on in several ways."""
    logits, _ = draw(1, 1, 5000, dtype, 13)
    scores = torch.full((1, 4), float("-inf"), device="cuda")
    scores[0, 0] = 0.0
    tokens, parents, _, _ = check(logits.expand(4, -1).contiguous(), scores, 4)
    assert (parents == 0).all()
    # without such scores equal candidates go to the lowest beam, then token
    tokens, parents, _, _ = check(logits.expand(4, -1).contiguous(), torch.zeros((1, 4), device="cuda"), 4)
    assert parents.tolist() == [[0, 1, 2, 3]] and (tokens == tokens[0, 0]).all()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("V", [10, 3000, 70001])
def test_equal_logits_go_to_the_lowest_token(V, dtype):
    logits = torch.zeros((2, V), dtype=dtype, device="cuda")
    tokens, parents, _, _ = check(logits, torch.tensor([[0.0, -0.5]], device="cuda"), 8)
    assert tokens.tolist() == [list(range(8))] and (parents == 0).all()
    logits[:, ::2] *= -1.0            # -0 and 0 are equal
    assert check(logits, torch.tensor([[0.0, -0.5]], device="cuda"), 8)[0].tolist() == [list(range(8))]
    # rising and falling rows: the bound moves with every chunk, or never
    ramp = torch.arange(V, dtype=torch.float32).remainder(200).sub(150).to(dtype).cuda()
    both = torch.stack([ramp, ramp.flip(0)])
    check(both, torch.tensor([[0.0, -0.01]], device="cuda"), 32 if V > 3000 else 8)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_masked_and_bad_logits(dtype):
    logits, scores = draw(3, 2, 9000, dtype, 17)
    logits[0] = float("-inf")                          # a beam without candidates
    logits[1, 5:] = float("-inf")
    logits[2, ::2] = float("-inf")
    logits[3, 17] = torch.finfo(dtype).min             # the type's lowest value is a logit
    logits[3, 18:] = torch.finfo(dtype).min
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    check(logits, scores, 16, status=status)
    assert int(status.item()) == 0
    logits[4, 100], logits[4, 8999], logits[5, 3] = float("nan"), float("inf"), float("inf")
    check(logits, scores, 16, status=status)
    assert int(status.item()) == kvx.KVX_FLAG_NOT_FINITE
    status.zero_()
    scores[0, 1], scores[1, 0], scores[2, 0] = float("nan"), float("inf"), float("-inf")
    check(logits[:4], scores[:2], 16, status=status)
    assert int(status.item()) == kvx.KVX_FLAG_NOT_FINITE
    # nothing at all
    none = torch.full((2, 100), float("-inf"), dtype=dtype, device="cuda")
    tokens, parents, new, _ = kvx.beam_select(none, torch.zeros((1, 2), device="cuda"))
    assert (tokens == -1).all() and (parents == -1).all() and torch.isneginf(new).all()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_strides_and_odd_rows(dtype):
    g = torch.Generator().manual_seed(5)
    big = (3 * torch.randn((12, 1503), generator=g)).to(dtype).cuda()
    scores = (-9.0 + 2.0 * torch.randn((2, 3), generator=g)).cuda()
    for view in (big[::2, 1:1400], big[:6, 3:], big[6:, :1501], big[::2, :1000]):
        check(view, scores, 5)


def test_large_logits_and_scores():
    for dtype in (torch.float32, torch.bfloat16):
        logits, scores = draw(2, 3, 4000, dtype, 23, spread=40.0)
        check(logits + 3000.0, scores - 500.0, 6)


def test_outputs_workspace_stream_and_graph():
    logits, scores = draw(4, 8, 20000, torch.bfloat16, 29)
    done = torch.zeros((4, 8), dtype=torch.bool, device="cuda")
    done[0, 1] = done[2, 7] = True
    want = check(logits, scores, 8, 2, done)
    ws = kvx.beam_workspace(requests=9, beams=16, vocab=50000, out=32)
    ws.fill_(0xFF)
    outs = dict(tokens=torch.empty((4, 8), dtype=torch.int32, device="cuda"),
                parents=torch.empty((4, 8), dtype=torch.int32, device="cuda"),
                new_scores=torch.empty((4, 8), device="cuda"),
                new_done=torch.empty((4, 8), dtype=torch.bool, device="cuda"))
    got = kvx.beam_select(logits, scores, eos=2, done=done, workspace=ws, **outs)
    assert all(a.data_ptr() == b.data_ptr() for a, b in zip(got, outs.values()))
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = kvx.beam_select(logits, scores, eos=2, done=done, stream=side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = kvx.beam_select(logits, scores, eos=2, done=done, workspace=ws)
    for _ in range(2):
        for t in got:
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
