"""Eviction by accumulated weight (kvx_evict8) against its definition: kept slots
and their order, weights, lengths, moved codes and scales, all exact (values are
code times a power of two)."""
import numpy as np
import pytest
import torch

import decode_reference as ref
from cross_model_kv_transfer_gb300 import kvx

pytestmark = pytest.mark.gpu


def dev(t):
    return torch.tensor(np.asarray(t), dtype=torch.int32).cuda()


def make(H, d, bs, lens, keep, seed, scales="pow2", cap=None):
    src = sum(-(-n // bs) for n in lens)
    dst = [-(-min(n, keep) // bs) for n in lens]
    nb = src + sum(dst) + 2
    kc, ks = ref.random_cache(nb, H, bs, d, seed, scales)
    vc, vs = ref.random_cache(nb, H, bs, d, seed + 1, scales)
    both = ref.block_table(list(lens) + [n * bs for n in dst], bs, nb, seed)
    table, to = both[:len(lens)], both[len(lens):, :max(-(-min(max(lens), keep) // bs), 1)].copy()
    used = [n for n in lens]
    codes, scale = (kc, vc), (ks, vs)
    for c, s in zip(codes, scale):
        # slots that no request holds, and the destination, hold NaN
        ref.poison(c, s, table, used, bs)
    cap = max(lens) + 3 if cap is None else cap
    w = np.exp(2 * np.random.default_rng(seed).standard_normal((len(lens), H, cap))).astype(np.float32)
    return dict(kc=kc, ks=ks, vc=vc, vs=vs, table=table, to=to, w=w, lens=list(lens),
                cache=kvx.Cache8(*(torch.tensor(t).cuda() for t in (kc, vc, ks, vs))))


def check(c, keep, sinks, recent, exact=True, **kw):
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    kept, kw_, new = c["cache"].evict(torch.tensor(c["w"]).cuda(), dev(c["table"]), dev(c["lens"]),
                                      dev(c["to"]), max_len=max(c["lens"]), keep=keep, sinks=sinks,
                                      recent=recent, status=status, **kw)
    torch.cuda.synchronize()
    assert int(status.item()) == 0
    want = ref.evict(c["w"], c["lens"], keep, sinks, recent)
    kept = kept.cpu().numpy()
    assert np.array_equal(kept, want)
    assert np.array_equal(new.cpu().numpy(), np.minimum(c["lens"], keep))
    live = want >= 0
    got_w = kw_.cpu().numpy()
    exp_w = np.take_along_axis(c["w"], np.maximum(want, 0), 2)
    assert np.array_equal(got_w[live], exp_w[live], equal_nan=True) and (got_w[~live] == 0).all()
    bs = c["cache"].block_size
    for codes, scale, old, olds in ((c["cache"].k_codes, c["cache"].k_scale, c["kc"], c["ks"]),
                                    (c["cache"].v_codes, c["cache"].v_scale, c["vc"], c["vs"])):
        src = ref.RefCache(old, olds)
        got, gs = codes.cpu().numpy(), scale.cpu().numpy()
        untouched = np.ones(len(got), dtype=bool)
        for r, n in enumerate(c["lens"]):
            m = min(n, keep)
            P = -(-m // bs)
            untouched[c["to"][r][:P]] = False
            for h in range(got.shape[1]):
                rows = src.rows(c["table"][r], want[r, h, :m], h)
                for b in range(P):
                    page, part = c["to"][r][b], rows[b * bs:(b + 1) * bs]
                    s = ref.pow2_scale(np.float32(np.abs(part).max()))
                    assert gs[page, h] == s
                    val = ref.E4M3[got[page, h, :len(part)]]
                    if exact:
                        assert np.array_equal(val, ref.e4m3_round(part / s))
                    else:      # code * scale is rounded to fp32: a tie may fall the other way
                        assert np.mean(val != ref.e4m3_round(part / s)) < 1e-2
                    # slots past the kept ones are left alone
                    assert np.array_equal(got[page, h, len(part):], old[page, h, len(part):])
        assert np.array_equal(got[untouched], old[untouched])
        assert np.array_equal(gs[untouched], olds[untouched], equal_nan=True)


@pytest.mark.parametrize("H,d,bs,lens,keep,sinks,recent", [
    (2, 64, 16, [100], 32, 4, 8), (1, 128, 16, [5, 33, 200, 1], 33, 0, 0),
    (8, 128, 16, [300, 7], 64, 4, 60), (3, 16, 7, [50, 51], 20, 20, 0),
    (1, 256, 64, [1025, 1024], 100, 1, 0), (2, 80, 1, [30], 29, 3, 26),
    (1, 64, 128, [2500], 700, 4, 64), (2, 64, 24, [40, 0, 90], 1, 0, 1),
    (1, 32, 16, [5000, 1500], 1000, 0, 17), (1, 16, 16, [40000], 9000, 4, 100)])
def test_matches_its_definition(H, d, bs, lens, keep, sinks, recent):
    check(make(H, d, bs, lens, keep, 3), keep, sinks, recent)


def test_ties_zeros_negatives_infinities_and_nan():
    c = make(2, 16, 16, [200, 130], 64, 5)
    c["w"][0, 0, :] = 1.0                                     # all equal: the lowest slots
    c["w"][0, 1, :] = np.random.default_rng(1).choice([0.0, 0.5, 2.0], c["w"].shape[2])
    c["w"][1, 0, ::2] = 0.0
    c["w"][1, 0, 1::4] = -0.0
    c["w"][1, 1, ::3] = np.nan
    c["w"][1, 1, 1::3] = np.inf
    c["w"][1, 1, 2::9] = -np.inf
    c["w"][1, 1, 5::9] = -1.5
    check(c, 64, 2, 5)
    c = make(1, 16, 16, [300], 250, 6)
    c["w"][:] = np.nan                                        # only NaN: again the lowest
    check(c, 250, 0, 10)
    c = make(1, 16, 16, [300], 100, 6)
    c["w"] = np.float32(1) + np.float32(2 ** -23) * np.random.default_rng(0).integers(
        0, 60, c["w"].shape).astype(np.float32)               # keys that differ in the last bits
    check(c, 100, 0, 0)


def test_scales_that_are_no_powers_of_two():
    check(make(2, 64, 16, [150, 90], 50, 8, scales="any"), 50, 2, 8, exact=False)


def test_a_workspace_and_another_stream_and_a_graph():
    c = make(2, 64, 16, [600, 90], 128, 9)
    ws = c["cache"].evict_workspace(num_requests=2, max_len=600, keep=128)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    for _ in range(3):
        check(c, 128, 4, 16, workspace=ws, stream=s)
    w, t, n, to = torch.tensor(c["w"]).cuda(), dev(c["table"]), dev(c["lens"]), dev(c["to"])
    outs = c["cache"].evict(w, t, n, to, max_len=600, keep=128, sinks=4, recent=16, workspace=ws)
    first = [o.clone() for o in outs] + [c["cache"].k_codes.clone()]
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        c["cache"].evict(w, t, n, to, max_len=600, keep=128, sinks=4, recent=16, workspace=ws,
                         kept=outs[0], kept_weights=outs[1], new_lens=outs[2])
    for o in outs:
        o.fill_(77)
    g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(first, list(outs) + [c["cache"].k_codes]))


def test_flags():
    c = make(1, 16, 16, [100, 50], 32, 10)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    run = lambda t, n, to: c["cache"].evict(torch.tensor(c["w"]).cuda(), dev(t), dev(n), dev(to),
                                            max_len=100, keep=32, status=status)
    _, _, new = run(c["table"], [101, -3], c["to"])
    assert int(status.item()) == kvx.KVX_FLAG_BAD_LENGTH and new.tolist() == [0, 0]
    status.zero_()
    bad = c["to"].copy()
    bad[0, 1] = c["cache"].num_blocks
    run(c["table"], c["lens"], bad)
    assert int(status.item()) == kvx.KVX_FLAG_BAD_BLOCK
    status.zero_()
    bad = c["table"].copy()
    bad[1, :] = -1
    run(bad, c["lens"], c["to"])
    assert int(status.item()) == kvx.KVX_FLAG_BAD_BLOCK
    assert not c["cache"].k_codes[int(c["to"][1][0])].any()


def test_kept_tokens_past_32_bit_offsets():
    H, d, bs = 2, 128, 64
    nb = 2 ** 32 // (H * bs * d) + 8
    small = make(H, d, bs, [300], 100, 12)
    big = kvx.Cache8.empty(nb, H, d, bs)
    at = [nb - 1, 5, nb - 2, nb - 7, 1]
    for a, b in ((big.k_codes, small["cache"].k_codes), (big.v_codes, small["cache"].v_codes),
                 (big.k_scale, small["cache"].k_scale), (big.v_scale, small["cache"].v_scale)):
        a[torch.tensor(at).cuda()] = b[torch.tensor(small["table"][0]).long().cuda()]
    w = torch.tensor(small["w"]).cuda()
    args = dict(max_len=300, keep=100, sinks=4, recent=10)
    one = small["cache"].evict(w, dev(small["table"]), dev([300]), dev(small["to"]), **args)
    two = big.evict(w, dev([at]), dev([300]), dev([[nb - 4, nb - 3]]), **args)
    assert all(torch.equal(a, b) for a, b in zip(one, two))
    for a, b in ((big.k_codes, small["cache"].k_codes), (big.v_codes, small["cache"].v_codes)):
        x, y = a[[nb - 4, nb - 3]], b[torch.tensor(small["to"][0]).long().cuda()]
        assert torch.equal(x[0], y[0]) and torch.equal(x[1, :, :36], y[1, :, :36])
