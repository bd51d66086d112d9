"""Attention over the 8-bit paged cache (kvx_attend8) against fp64: outputs,
log-sum-exps and accumulated weights; grouped heads, single tokens and chunks,
blocks that end inside a tile, empty rows, poisoned slots, strides, flags.

Tolerances.  A score is a sum of d products in fp32 (tensor cores truncate
where they align): its error is at most d * 2^-24 of scale * sum |q k| (`reach`),
taken as xe = 2^-16 reach for d <= 256.  A probability is then off by 2 xe + n
2^-23 relative (its own score, and the sum over n slots), and for bf16 queries
by another 2^-10 for its rounding before the product with v; an output by that
times sum p |v| (`mass`) and, in bf16, by half an ulp of itself.  Weights add
up `rows` probabilities in fp32."""
import numpy as np
import pytest
import torch

import decode_reference as ref
from cross_model_kv_transfer_gb300 import kvx

pytestmark = pytest.mark.gpu


def dev(t):
    return torch.tensor(np.asarray(t), dtype=torch.int32).cuda()


def make(H, G, d, bs, lens, news, dtype, seed, scales="pow2", qscale=1.5, spare=3):
    nb = sum(-(-n // bs) for n in lens) + spare
    kc, ks = ref.random_cache(nb, H, bs, d, seed, scales)
    vc, vs = ref.random_cache(nb, H, bs, d, seed + 1, scales)
    table = ref.block_table(lens, bs, nb, seed)
    ref.poison(kc, ks, table, lens, bs)
    ref.poison(vc, vs, table, lens, bs)
    cu = np.concatenate([[0], np.cumsum(news)]).astype(np.int32)
    q = torch.tensor(qscale * np.random.default_rng(seed + 2).standard_normal((cu[-1], H * G, d)))
    return dict(cache=kvx.Cache8(*(torch.tensor(t).cuda() for t in (kc, vc, ks, vs))),
                rk=ref.RefCache(kc, ks), rv=ref.RefCache(vc, vs), table=table, cu=cu,
                q=q.to(dtype))


def compare(out, lse, w, want, bf16, n, rows):
    o, ls, ws, mass, reach = want
    xe = 2.0 ** -16 * reach
    rel = 2 * xe + n * 2.0 ** -23 + 2.0 ** -21 + (2.0 ** -10 if bf16 else 0)
    tol = rel[..., None] * mass + (2.0 ** -8 * np.abs(o) if bf16 else 0) + 1e-30
    got = out.double().cpu().numpy()
    assert np.isfinite(got).all()
    assert (np.abs(got - o) <= tol).all(), (np.abs(got - o) / tol).max()
    l = lse.double().cpu().numpy()
    empty = np.isneginf(ls)
    assert np.array_equal(np.isneginf(l), empty) and (got[empty] == 0).all()
    assert (np.abs(l[~empty] - ls[~empty]) <=
            (xe + n * 2.0 ** -23 + 2.0 ** -21 * (1 + np.abs(np.where(empty, 0, ls))))[~empty]).all()
    if w is not None:
        ww = w.double().cpu().numpy()[..., :ws.shape[2]]
        wtol = (2 * xe.max(initial=0) + n * 2.0 ** -23 + (rows + 16) * 2.0 ** -23) * ws + 1e-30
        assert (np.abs(ww - ws) <= wtol).all(), (np.abs(ww - ws) / wtol).max()


CASES = [
    # H, G, d, bs, lens, new
    (1, 1, 64, 16, [1], [1]),
    (2, 2, 64, 16, [512], [1]),
    (2, 8, 128, 16, [1, 17, 0, 300], [1, 1, 1, 1]),
    (1, 5, 128, 24, [100, 23, 24, 25], [1, 1, 1, 1]),
    (3, 4, 128, 64, [1000, 63, 65], [1, 1, 1]),
    (1, 16, 128, 16, [129], [1]),
    (1, 12, 64, 7, [50, 201], [1, 1]),
    (2, 1, 256, 32, [90, 257], [1, 1]),
    (1, 3, 80, 16, [33], [1]),
    (2, 2, 96, 8, [70, 31], [1, 1]),
    (1, 2, 16, 1, [19], [1]),
    (1, 8, 128, 16, [2500], [1]),
    # chunks: ragged, with requests without queries, and rows that see nothing
    (2, 2, 64, 16, [5, 40, 9, 12], [2, 0, 9, 12]),
    (2, 4, 128, 16, [200, 131], [61, 5]),
    (1, 8, 128, 16, [300], [300]),
    (1, 5, 128, 24, [170, 129], [128, 129]),
    (1, 1, 128, 16, [3, 0, 7], [5, 2, 9]),
    (2, 8, 64, 128, [257], [130]),
    (1, 2, 256, 16, [150], [70]),
    (1, 3, 80, 5, [44], [20]),
    (1, 16, 128, 16, [140], [33]),
]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("H,G,d,bs,lens,new", CASES)
def test_matches_fp64(H, G, d, bs, lens, new, dtype):
    c = make(H, G, d, bs, lens, new, dtype, 7)
    scale = d ** -0.5
    weights = torch.full((len(lens), H, max(lens) + 5), 0.25, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    out, lse = c["cache"].attend(c["q"].cuda(), dev(c["table"]), dev(lens), max(lens),
                                 cu_seqlens=dev(c["cu"]), max_new=max(new), weights=weights,
                                 status=status)
    want = ref.attend(c["q"].double().numpy(), c["rk"], c["rv"], c["table"], lens, c["cu"], scale)
    used = np.arange(max(lens) + 5)[None, None] < np.array(lens)[:, None, None]
    assert (weights.cpu().numpy()[~np.broadcast_to(used, weights.shape)] == 0.25).all()
    weights -= 0.25
    # the 0.25 that was there costs each of the additions half an ulp of the sum
    w = want[2].copy()
    assert np.abs(weights.double().cpu().numpy()[..., :w.shape[2]] - w).max(initial=0) <= \
        (2 * 2.0 ** -16 * want[4].max(initial=0) + (max(lens) + max(new) * G + 16) * 2.0 ** -23) * \
        (w.max(initial=0) + 0.25)
    compare(out, lse, None, want, dtype == torch.bfloat16, max(lens), max(new) * G)
    assert int(status.item()) == 0


@pytest.mark.parametrize("H,G,R,longest,new", [(8, 2, 45, 700, 1), (4, 8, 60, 300, 3), (8, 1, 40, 400, 130),
                                               (2, 8, 20, 600, 70)])
def test_more_work_than_the_gpu_holds_at_once(H, G, R, longest, new):
    """Several items follow one another on an SM, whole and in parts."""
    lens = [max(new, (longest * (r + 1)) // R) for r in range(R)]
    news = [new if r % 3 else max(1, new // 2) for r in range(R)]
    c = make(H, G, 128, 16, lens, news, torch.bfloat16, 37)
    w = torch.zeros((R, H, max(lens)), device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    out, lse = c["cache"].attend(c["q"].cuda(), dev(c["table"]), dev(lens), max(lens),
                                 cu_seqlens=dev(c["cu"]), max_new=new, weights=w, status=status)
    want = ref.attend(c["q"].double().numpy(), c["rk"], c["rv"], c["table"], lens, c["cu"], 128 ** -0.5)
    assert int(status.item()) == 0
    compare(out, lse, w, want, True, max(lens), new * G)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_the_one_token_form_needs_no_request_table(dtype):
    lens = [40, 1, 133]
    c = make(2, 4, 128, 16, lens, [1, 1, 1], dtype, 3, scales="any")
    w = torch.zeros((3, 2, 133), device="cuda")
    out, lse = c["cache"].attend(c["q"].cuda(), dev(c["table"]), dev(lens), 133, weights=w,
                                 scale=0.2)
    want = ref.attend(c["q"].double().numpy(), c["rk"], c["rv"], c["table"], lens, c["cu"], 0.2)
    compare(out, lse, w, want, dtype == torch.bfloat16, 133, 4)
    w2 = w.clone()
    c["cache"].attend(c["q"].cuda(), dev(c["table"]), dev(lens), 133, weights=w2, scale=0.2)
    assert (w2 - 2 * w).abs().max() <= 2.0 ** -22 * w2.max()


@pytest.mark.parametrize("qscale", [0.0, 30.0])
@pytest.mark.parametrize("new", [1, 40])
def test_flat_and_peaked_scores(qscale, new):
    """All scores equal, and scores of several hundred with one slot that takes
    all: no overflow, no lost mass."""
    c = make(1, 4, 128, 16, [700], [new], torch.bfloat16, 9, qscale=qscale)
    w = torch.zeros((1, 1, 700), device="cuda")
    out, lse = c["cache"].attend(c["q"].cuda(), dev(c["table"]), dev([700]), 700,
                                 cu_seqlens=dev(c["cu"]), max_new=new, weights=w, scale=1.0)
    want = ref.attend(c["q"].double().numpy(), c["rk"], c["rv"], c["table"], [700], c["cu"], 1.0)
    compare(out, lse, w, want, True, 700, 4 * new)
    assert abs(float(w.double().sum()) - 4 * new) < 1e-2 * new


def test_block_scales_of_very_different_size():
    """Values of one block a million times those of another, which holds all
    the attention: the small ones must not drown."""
    H, d, bs, n = 1, 128, 16, 64
    c = make(H, 1, d, bs, [n], [1], torch.bfloat16, 5)
    cache, table = c["cache"], c["table"]
    big, small = int(table[0][0]), int(table[0][3])
    cache.v_scale[big] *= 2.0 ** 20
    cache.k_scale[big] = 2.0 ** -40        # scores of about zero
    cache.k_scale[small] = 2.0 ** 3
    rk = ref.RefCache(cache.k_codes.cpu().numpy(), cache.k_scale.cpu().numpy())
    rv = ref.RefCache(cache.v_codes.cpu().numpy(), cache.v_scale.cpu().numpy())
    q = 0.5 * rk.rows(table[0], [n - 1], 0)[None] / 8.0
    q = torch.tensor(q).to(torch.bfloat16)
    out, lse = cache.attend(q.cuda(), dev(table), dev([n]), n, scale=0.25)
    want = ref.attend(q.double().numpy(), rk, rv, table, [n], [0, 1], 0.25)
    compare(out, lse, None, want, True, n, 1)


@pytest.mark.parametrize("new", [1, 19])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_strided_queries_and_outputs(dtype, new):
    lens = [77, 100]
    c = make(2, 2, 64, 16, lens, [new, new], dtype, 13)
    n = 2 * new
    pad = torch.full((n, 9, 64 + 16), 5.0, dtype=dtype)
    pad[:, 2:6, 3:67] = c["q"]
    fused = pad.cuda()
    wide = torch.full((5, n, 72), 3.0, dtype=dtype, device="cuda")
    out = wide[:4, :, 4:68].transpose(0, 1)
    lse = torch.empty((n, 4), device="cuda")
    c["cache"].attend(fused[:, 2:6, 3:67], dev(c["table"]), dev(lens), 100,
                      cu_seqlens=dev(c["cu"]), max_new=new, out=out, lse=lse)
    want = ref.attend(c["q"].double().numpy(), c["rk"], c["rv"], c["table"], lens, c["cu"], 0.125)
    compare(out, lse, None, want, dtype == torch.bfloat16, 100, 1)
    assert (wide[4] == 3).all() and (wide[:, :, :4] == 3).all() and (wide[:, :, 68:] == 3).all()


@pytest.mark.parametrize("new", [1, 33])
def test_a_wider_table_and_looser_bounds_change_nothing(new):
    lens = [150, 60]
    c = make(1, 8, 128, 16, lens, [new, new], torch.bfloat16, 17)
    q = c["q"].cuda()
    a = c["cache"].attend(q, dev(c["table"]), dev(lens), 150, cu_seqlens=dev(c["cu"]), max_new=new)
    wide = np.full((2, 300), -5, dtype=np.int32)
    wide[:, :c["table"].shape[1]] = c["table"]
    b = c["cache"].attend(q, dev(wide), dev(lens), 4700, cu_seqlens=dev(c["cu"]), max_new=4000)
    want = ref.attend(c["q"].double().numpy(), c["rk"], c["rv"], c["table"], lens, c["cu"],
                      128 ** -0.5)
    for out, lse in (a, b):
        compare(out, lse, None, want, True, 150, 8)


@pytest.mark.parametrize("new", [1, 20])
def test_bad_lengths_blocks_and_tables_are_flagged(new):
    lens = [64, 64, 64]
    c = make(1, 2, 64, 16, lens, [new] * 3, torch.float32, 19)
    q, table = c["q"].cuda(), c["table"].copy()
    run = lambda t, n, m, cu, **kw: c["cache"].attend(q, dev(t), dev(n), m, cu_seqlens=dev(cu),
                                                      max_new=new, status=status, **kw)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    out, lse = run(table, [64, 65, -1], 64, c["cu"])
    assert int(status.item()) == kvx.KVX_FLAG_BAD_LENGTH
    want = ref.attend(c["q"].double().numpy(), c["rk"], c["rv"], table, [64, 0, 0], c["cu"], 0.125)
    compare(out, lse, None, want, False, 64, 1)
    status.zero_()
    bad = table.copy()
    bad[1, 3] = c["cache"].num_blocks      # slots 48 .. 63 of request 1 are masked
    w = torch.zeros((3, 1, 64), device="cuda")
    out, lse = run(bad, lens, 64, c["cu"], weights=w)
    assert int(status.item()) == kvx.KVX_FLAG_BAD_BLOCK
    assert torch.isfinite(out).all() and (w[1, 0, 48:] == 0).all()
    want = ref.attend(c["q"].double().numpy(), c["rk"], c["rv"], table, lens, c["cu"], 0.125)
    ok = np.r_[0:new, 2 * new:3 * new]
    compare(out[ok], lse[ok], None, tuple(t[ok] if i != 2 else t for i, t in enumerate(want)),
            False, 64, 1)
    for cu in ([0, new, new - 1, 3 * new], [1, new, 2 * new, 3 * new], [0, new, 2 * new, 3 * new - 1],
               [0, 0, new - 1, 3 * new]):
        status.zero_()
        out.fill_(9.0)
        run(table, lens, 64, cu, out=out)
        assert int(status.item()) == kvx.KVX_FLAG_BAD_SEQLENS and (out == 9).all()


def test_a_workspace_serves_many_calls_and_other_streams():
    lens = [333, 90, 512]
    c = make(2, 4, 128, 16, lens, [1, 1, 1], torch.bfloat16, 23)
    ws = c["cache"].attend_workspace(ntok=3, num_requests=3, q_heads=8, max_len=512, weights=True)
    q, table, n = c["q"].cuda(), dev(c["table"]), dev(lens)
    want = ref.attend(c["q"].double().numpy(), c["rk"], c["rv"], c["table"], lens, c["cu"],
                      128 ** -0.5)
    s = torch.cuda.Stream()
    first = None
    for i in range(6):
        w = torch.zeros((3, 2, 512), device="cuda")
        s.wait_stream(torch.cuda.current_stream())
        out, lse = c["cache"].attend(q, table, n, 512, weights=w, workspace=ws, stream=s)
        torch.cuda.current_stream().wait_stream(s)
        compare(out, lse, w, want, True, 512, 4)
        first = (out, lse, w) if first is None else first
        assert all(torch.equal(a, b) for a, b in zip(first, (out, lse, w)))
    # without a workspace of the caller's
    out, lse = c["cache"].attend(q, table, n, 512, stream=s)
    s.synchronize()
    compare(out, lse, None, want, True, 512, 4)
    # in a graph
    g = torch.cuda.CUDAGraph()
    out.zero_()
    with torch.cuda.graph(g):
        c["cache"].attend(q, table, n, 512, workspace=ws, out=out, lse=lse)
    for _ in range(3):
        out.zero_()
        g.replay()
        torch.cuda.synchronize()
        compare(out, lse, None, want, True, 512, 4)


@pytest.mark.parametrize("new", [1, 130])
def test_blocks_past_32_bit_offsets(new):
    H, d, bs, n = 1, 128, 64, 200
    nb = 2 ** 32 // (H * bs * d) + 5
    c = make(H, 4, d, bs, [n], [new], torch.bfloat16, 29)
    cache = kvx.Cache8.empty(nb, H, d, bs)
    table = np.array([[nb - 1, 2, nb - 3, nb - 2]], dtype=np.int32)
    for big, small in ((cache.k_codes, c["cache"].k_codes), (cache.v_codes, c["cache"].v_codes),
                       (cache.k_scale, c["cache"].k_scale), (cache.v_scale, c["cache"].v_scale)):
        big[torch.tensor(table[0]).cuda().long()] = small[torch.tensor(c["table"][0]).cuda().long()]
    a = cache.attend(c["q"].cuda(), dev(table), dev([n]), n, cu_seqlens=dev(c["cu"]), max_new=new)
    want = ref.attend(c["q"].double().numpy(), c["rk"], c["rv"], c["table"], [n], c["cu"], d ** -0.5)
    compare(*a, None, want, True, n, 1)


def test_no_queries_and_no_slots():
    c = make(1, 1, 64, 16, [20], [1], torch.float32, 31)
    out, lse = c["cache"].attend(torch.empty((0, 1, 64), device="cuda"), dev(c["table"]), dev([20]),
                                 20, cu_seqlens=dev([0, 0]))
    assert out.shape == (0, 1, 64) and lse.shape == (0, 1)
    w = torch.ones((1, 1, 8), device="cuda")
    out, lse = c["cache"].attend(c["q"].cuda(), dev(c["table"]), dev([0]), 0, weights=w)
    assert (out == 0).all() and torch.isneginf(lse).all() and (w == 1).all()


@pytest.mark.parametrize("G,new", [(4, 1), (4, 12), (4, 70), (16, 1), (3, 61)])
@pytest.mark.parametrize("d", [128, 112, 48])
def test_unaligned_rows_of_every_form(d, G, new):
    """bf16 queries and outputs that no 16-byte access can reach, few rows to many,
    with the weights."""
    lens = [new + 77, new + 200]
    c = make(2, G, d, 16, lens, [new, new], torch.bfloat16, 41)
    n, hq = 2 * new, 2 * G
    wide = torch.full((n, hq + 1, d + 3), 7.0, dtype=torch.bfloat16, device="cuda")
    wide[:, 1:, 1:d + 1] = c["q"].cuda()
    into = torch.full((n, hq, d + 5), 3.0, dtype=torch.bfloat16, device="cuda")
    w = torch.zeros((2, 2, max(lens)), device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    out, lse = c["cache"].attend(wide[:, 1:, 1:d + 1], dev(c["table"]), dev(lens), max(lens),
                                 cu_seqlens=dev(c["cu"]), max_new=new, out=into[:, :, 3:d + 3],
                                 weights=w, status=status)
    want = ref.attend(c["q"].double().numpy(), c["rk"], c["rv"], c["table"], lens, c["cu"], d ** -0.5)
    assert int(status.item()) == 0
    compare(out, lse, w, want, True, max(lens), new * G)
    assert (into[:, :, :3] == 3).all() and (into[:, :, d + 3:] == 3).all()


@pytest.mark.parametrize("G,new", [(8, 1), (5, 4)])
def test_weights_where_the_bound_on_lengths_is_too_large_to_keep_scores(G, new):
    """Kept scores would take more than 4 GB: they are formed again instead."""
    lens, bound = [new + 300, new + 77], 1 << 26
    c = make(2, G, 128, 16, lens, [new, new], torch.bfloat16, 43)
    w = torch.zeros((2, 2, bound), device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    out, lse = c["cache"].attend(c["q"].cuda(), dev(c["table"]), dev(lens), bound, cu_seqlens=dev(c["cu"]),
                                 max_new=new, weights=w, status=status)
    want = ref.attend(c["q"].double().numpy(), c["rk"], c["rv"], c["table"], lens, c["cu"], 128 ** -0.5)
    assert int(status.item()) == 0
    compare(out, lse, w[:, :, :max(lens)].contiguous(), want, True, max(lens), new * G)
    assert not w[:, :, max(lens):].any()
