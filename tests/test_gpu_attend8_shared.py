"""Attention of requests that share prefixes (kvx_attend8_shared) against fp64 of
one sequence for each request: grouped heads, single tokens and chunks, prefixes
that end inside a block, empty ones, groups without requests, strides, flags.

Tolerances.  A score is off by xe = 2^-16 reach (reach: scale * sum |q k|), a
probability within its part (prefix or own slots) by 2 xe + n 2^-23 relative, and
for bf16 queries by another 2^-10 for its rounding before the product with v.
A part's share of the whole is formed from the two parts' log-sum-exps, each
off by xe + n 2^-23, in base 2 with an exponential and a logarithm: 2 xe + n 2^-22 +
2^-20.  Outputs are off by the sum of those times sum p |v| (mass) and, in bf16, half
an ulp of themselves; log-sum-exps by xe + n 2^-23 and a few roundings."""
import numpy as np
import pytest
import torch

import continuation_reference as cref
import decode_reference as ref
from cross_model_kv_transfer_gb300 import kvx

pytestmark = pytest.mark.gpu


def dev(t):
    return torch.tensor(np.asarray(t), dtype=torch.int32).cuda()


def make(H, G, d, bs, prefixes, members, lens, news, dtype, seed, scales="pow2", qscale=1.5):
    """prefixes: lengths; members: requests of each; lens, news: of the requests."""
    every = list(prefixes) + list(lens)
    nb = sum(-(-n // bs) for n in every) + 3
    kc, ks = ref.random_cache(nb, H, bs, d, seed, scales)
    vc, vs = ref.random_cache(nb, H, bs, d, seed + 1, scales)
    table = ref.block_table(every, bs, nb, seed)
    ref.poison(kc, ks, table, every, bs)
    ref.poison(vc, vs, table, every, bs)
    cu = np.concatenate([[0], np.cumsum(news)]).astype(np.int32)
    groups = np.concatenate([[0], np.cumsum(members)]).astype(np.int32)
    q = torch.tensor(qscale * np.random.default_rng(seed + 2).standard_normal((cu[-1], H * G, d)))
    P = len(prefixes)
    return dict(cache=kvx.Cache8(*(torch.tensor(t).cuda() for t in (kc, vc, ks, vs))),
                rk=cref.Joined(kc, ks), rv=cref.Joined(vc, vs), prefix_table=table[:P],
                prefixes=list(prefixes), groups=groups, table=table[P:], lens=list(lens), cu=cu,
                news=list(news), q=q.to(dtype))


def call(c, **kw):
    most = max(c["news"] + [1])
    args = dict(max_prefix=max(c["prefixes"]), max_len=max(c["lens"]), groups=dev(c["groups"]),
                cu_seqlens=dev(c["cu"]), max_new=most,
                max_group=int(max(1, np.diff(c["groups"]).max())))
    q = kw.pop("q", None)
    args.update(kw)
    return c["cache"].attend_shared(c["q"].cuda() if q is None else q, dev(c["prefix_table"]),
                                    dev(c["prefixes"]), dev(c["table"]), dev(c["lens"]), **args)


def want_of(c, scale=None):
    d = c["q"].shape[2]
    return cref.shared_attend(c["q"].double().numpy(), c["rk"], c["rv"], c["prefix_table"],
                              c["prefixes"], c["groups"], c["table"], c["lens"], c["cu"],
                              d ** -0.5 if scale is None else scale)


def compare(out, lse, want, bf16, n):
    o, ls, _, mass, reach = want
    xe = 2.0 ** -16 * reach
    rel = 4 * xe + 3 * n * 2.0 ** -23 + 2.0 ** -19 + (2.0 ** -10 if bf16 else 0)
    tol = rel[..., None] * mass + (2.0 ** -8 * np.abs(o) if bf16 else 0) + 1e-30
    got = out.double().cpu().numpy()
    assert np.isfinite(got).all()
    assert (np.abs(got - o) <= tol).all(), (np.abs(got - o) / tol).max()
    l = lse.double().cpu().numpy()
    empty = np.isneginf(ls)
    assert np.array_equal(np.isneginf(l), empty) and (got[empty] == 0).all()
    near = np.abs(l[~empty] - ls[~empty])
    assert (near <= (xe + n * 2.0 ** -23 + 2.0 ** -20 * (1 + np.abs(np.where(empty, 0, ls))))[~empty]).all()


def check(c, **kw):
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    out, lse = call(c, status=status, **kw)
    n = max(c["prefixes"]) + max(c["lens"])
    compare(out, lse, want_of(c), c["q"].dtype == torch.bfloat16, n)
    assert int(status.item()) == 0
    return out, lse


CASES = [
    # H, G, d, bs, prefixes, members, lens, news
    (1, 1, 64, 16, [1], [1], [1], [1]),
    (2, 4, 128, 16, [300], [3], [1, 17, 40], [1, 1, 1]),
    (2, 8, 128, 16, [513, 30], [4, 2], [5, 6, 7, 8, 1, 33], [1] * 6),
    (1, 8, 128, 24, [0, 100], [2, 3], [9, 24, 25, 48, 1], [1] * 5),       # an empty prefix
    (1, 3, 80, 16, [77], [2], [0, 0], [1, 1]),                             # only the prefix
    (2, 2, 96, 8, [65, 40, 9], [1, 0, 2], [3, 4, 5], [1] * 3),             # a group without requests
    (1, 2, 64, 16, [0], [2], [0, 1], [2, 3]),                              # rows that see nothing
    (1, 5, 128, 16, [200], [4], [30, 3, 9, 64], [3, 1, 0, 5]),             # ragged chunks
    (2, 4, 128, 16, [129, 250], [2, 2], [70, 100, 61, 90], [61, 5, 61, 40]),
    (1, 8, 128, 64, [1000], [20], list(range(1, 21)), [1] * 20),           # many rows of a prefix
    (2, 8, 128, 16, [140], [3], [150, 300, 44], [130, 200, 44]),           # own chunks wide
    (2, 1, 256, 32, [90], [2], [257, 5], [1, 1]),
    (1, 12, 64, 7, [50], [2], [20, 9], [1, 2]),
    (1, 2, 16, 1, [19], [3], [2, 3, 4], [1, 1, 1]),
    (1, 16, 128, 16, [2500], [2], [1, 700], [1, 1]),
]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("H,G,d,bs,prefixes,members,lens,news", CASES)
def test_matches_fp64(H, G, d, bs, prefixes, members, lens, news, dtype):
    check(make(H, G, d, bs, prefixes, members, lens, news, dtype, 3))


LONG = [
    (1, 2, 64, 16, [300], [2], [2100, 5], [1, 1]),                         # more own slots than an item's CTA takes
    (1, 13, 128, 16, [90], [2], [100, 30], [5, 4]),                        # 65 rows, one more than it takes
    (1, 16, 64, 32, [5000], [2], [33, 2048], [4, 1]),                      # 64 rows
    (1, 8, 128, 16, [9000], [64], [3] * 64, [1] * 64),                     # a prefix of much work
    (1, 8, 128, 64, [70, 9000], [3, 125], [1 + r % 5 for r in range(128)], [1] * 128),
]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("H,G,d,bs,prefixes,members,lens,news", LONG)
def test_matches_fp64_beyond_each_form(H, G, d, bs, prefixes, members, lens, news, dtype):
    check(make(H, G, d, bs, prefixes, members, lens, news, dtype, 31))


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_without_tables(dtype):
    """One token for each request and one prefix for all: neither table is needed."""
    c = make(2, 4, 64, 16, [200], [7], [3, 1, 5, 9, 2, 17, 30], [1] * 7, dtype, 5)
    a = check(c)
    b = check(c, cu_seqlens=None, groups=None, max_group=None)
    g = check(c, cu_seqlens=None)
    for x in (b, g):
        assert all(torch.equal(s, t) for s, t in zip(a, x))


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_scales_of_any_size_and_far_scores(dtype):
    c = make(1, 4, 128, 16, [300], [3], [40, 50, 60], [1, 2, 1], dtype, 9, scales="any", qscale=300.0)
    check(c)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("way", ["prefix", "own"])
def test_one_part_far_above_the_other(way, dtype):
    """Scores of one part thousands above the other's: it alone counts, and nothing overflows."""
    c = make(1, 2, 64, 16, [48], [2], [32, 20], [1, 1], dtype, 13, qscale=1.0)
    cache = c["cache"]
    mine = sorted({int(x) for x in (c["prefix_table"] if way == "prefix" else c["table"]).ravel() if x >= 0})
    up = torch.tensor(mine).cuda()
    cache.k_scale[up] *= 2.0 ** 14
    c["rk"].scale[mine] *= 2.0 ** 14
    check(c)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_strided_queries_and_outputs_in_place(dtype):
    c = make(2, 4, 64, 16, [100], [3], [30, 3, 9], [3, 1, 5], dtype, 15)
    want = check(c)
    n = c["q"].shape[0]
    big = torch.zeros((n, 11, 72), dtype=dtype, device="cuda")
    view = big[:, 1:9, 4:68]
    view.copy_(c["q"])
    lse = torch.empty((n, 8), device="cuda")
    out, _ = call(c, q=view, out=view, lse=lse)
    assert out.data_ptr() == view.data_ptr() and torch.equal(out, want[0]) and torch.equal(lse, want[1])
    assert (big[:, 0] == 0).all() and (big[:, 9:] == 0).all() and (big[..., :4] == 0).all()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("case", [(8, 8, 1), (8, 4, 9), (1, 1, 1)])
def test_one_workspace_for_several_sizes(case, dtype):
    H, G, members = case
    c = make(2, G, 128, 16, [300], [members], [20] * members, [1] * members, dtype, 17)
    ws = c["cache"].attend_shared_workspace(ntok=200, num_requests=70, q_heads=64, num_prefixes=5,
                                            max_prefix=5000, max_len=900, max_new=9, dtype=dtype)
    ws[1024:].fill_(0xA5)
    for _ in range(2):
        check(c, workspace=ws)
        # an ordinary call between, in the same workspace
        c["cache"].attend(c["q"].cuda(), dev(c["table"]), dev(c["lens"]), 20, workspace=ws)


def test_malformed_tables_write_nothing():
    for dtype in (torch.float32, torch.bfloat16):
        c = make(1, 4, 64, 16, [50, 60], [2, 3], [4, 5, 6, 7, 8], [1, 2, 1, 1, 1], dtype, 19)
        n = c["q"].shape[0]
        for bad in (dict(groups=dev([1, 2, 5])), dict(groups=dev([0, 2, 4])), dict(groups=dev([0, 3, 2])),
                    dict(groups=dev([0, 2 ** 30, 5])), dict(groups=dev([0, -7, 5])),
                    dict(groups=dev([0, 2, 6])), dict(max_group=1),
                    dict(cu_seqlens=dev([0, 1, 3, 2, 5, 6])), dict(max_new=1, max_group=5)):
            out = torch.full((n, 4, 64), 7.0, dtype=dtype, device="cuda")
            lse = torch.full((n, 4), 7.0, device="cuda")
            status = torch.zeros(1, dtype=torch.int32, device="cuda")
            call(c, out=out, lse=lse, status=status, **bad)
            assert (out == 7).all() and (lse == 7).all(), bad
            assert int(status.item()) & kvx.KVX_FLAG_BAD_SEQLENS, bad


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_bad_lengths_and_blocks(dtype):
    c = make(1, 2, 64, 16, [50, 60], [2, 1], [4, 5, 20], [1, 1, 1], dtype, 21)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    # lengths out of bounds count as 0
    got = c["cache"].attend_shared(c["q"].cuda(), dev(c["prefix_table"]), dev([51, 60]), dev(c["table"]),
                                   dev([4, -1, 20]), max_prefix=50, max_len=20, groups=dev(c["groups"]),
                                   status=status)
    assert int(status.item()) == kvx.KVX_FLAG_BAD_LENGTH
    z = dict(c, prefixes=[0, 0], lens=[4, 0, 20])
    compare(*got, want_of(z), dtype == torch.bfloat16, 20)
    # blocks outside the pool are masked, in either part
    status.zero_()
    table, prefix = c["table"].copy(), c["prefix_table"].copy()
    table[2, 0], prefix[0, 1] = 10 ** 6, -1
    got = c["cache"].attend_shared(c["q"].cuda(), dev(prefix), dev([50, 60]), dev(table), dev([4, 5, 20]),
                                   max_prefix=60, max_len=20, groups=dev(c["groups"]), status=status)
    assert int(status.item()) == kvx.KVX_FLAG_BAD_BLOCK
    keep = [[j for j in range(50) if not 16 <= j < 32], list(range(60))]
    z = dict(c, rk=Masked(c["rk"], keep), rv=Masked(c["rv"], keep), prefixes=[34, 60], lens=[4, 5, 4])
    z["table"] = c["table"].copy()
    z["table"][2, 0] = c["table"][2, 1]
    compare(*got, want_of(z), dtype == torch.bfloat16, 80)


class Masked(cref.Joined):
    """Prefix slots by a list of those that count."""

    def __init__(self, of, keep):
        self.values, self.scale, self.keep = of.values, of.scale, keep

    def rows(self, table_row, slots, h):
        before, n, own = table_row
        keep = self.keep[0 if n == 34 else 1]
        total = len(slots)
        return np.concatenate([ref.RefCache.rows(self, before, keep[:min(n, total)], h),
                               ref.RefCache.rows(self, own, range(max(0, total - n)), h)])


@pytest.mark.parametrize("dtype,new", [(torch.bfloat16, 1), (torch.bfloat16, 30), (torch.float32, 1)])
def test_captured_and_on_another_stream(dtype, new):
    c = make(2, 8, 128, 16, [300, 40], [5, 3], [40 + r for r in range(8)], [new] * 8, dtype, 23)
    want = check(c)
    q, tables = c["q"].cuda(), [dev(c[k]) for k in ("prefix_table", "prefixes", "table", "lens", "groups", "cu")]
    args = dict(max_prefix=300, max_len=47, groups=tables[4], max_group=5, cu_seqlens=tables[5], max_new=new)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = c["cache"].attend_shared(q, *tables[:4], stream=side, **args)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    ws = c["cache"].attend_shared_workspace(ntok=8 * new, num_requests=8, num_prefixes=2, q_heads=16,
                                            max_prefix=300, max_len=47, max_group=5, max_new=new, dtype=dtype)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = c["cache"].attend_shared(q, *tables[:4], workspace=ws, **args)
    for _ in range(2):
        for t in got:
            t.fill_(5)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_same_result_every_time():
    """Splits over the GPU are joined in a fixed order."""
    c = make(4, 8, 128, 16, [3000, 700], [9, 6], [20 + 9 * r for r in range(15)], [1] * 15, torch.bfloat16, 29)
    a = call(c)
    for _ in range(3):
        assert all(torch.equal(x, y) for x, y in zip(a, call(c)))
