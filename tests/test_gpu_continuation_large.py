"""Pages beyond 4 GB of a pool, and selections over many rows: results are those of the
same pages in a small pool, and of the same rows alone."""
import pytest
import torch

from cross_model_kv_transfer_gb300 import kvx

pytestmark = pytest.mark.gpu


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def test_pages_beyond_four_gigabytes():
    H, bs, d, blocks, few = 8, 16, 128, 300_000, 40        # 4.9 GB of codes each for keys and values
    g = torch.Generator().manual_seed(3)
    small = kvx.Cache8(*(torch.randint(0, 0x70, (few, H, bs, d), generator=g, dtype=torch.uint8).cuda() for _ in range(2)),
                       *(2.0 ** torch.randint(-12, -6, (few, H), generator=g).cuda().float() for _ in range(2)))
    big = kvx.Cache8.empty(blocks, H, d, bs)
    top = torch.arange(blocks - 3 * few, blocks, 3, device="cuda")       # where the small pool's pages lie
    for a, b in ((big.k_codes, small.k_codes), (big.v_codes, small.v_codes), (big.k_scale, small.k_scale),
                 (big.v_scale, small.v_scale)):
        a[top] = b
    prefix, table = i32([list(range(12)), list(range(12, 24))]), i32([[24, 25], [26, 27], [28, 29], [30, 31], [32, 33]])
    move = lambda t: top[t.long()].int()
    for dtype, new in ((torch.bfloat16, 1), (torch.bfloat16, 20), (torch.float32, 2)):
        q = torch.randn((5 * new, 16, d), generator=g).to(dtype).cuda()
        args = dict(max_prefix=190, max_len=30, groups=i32([0, 3, 5]), max_group=3, max_new=new,
                    cu_seqlens=i32(list(range(0, 5 * new + 1, new))))
        lens = i32([20, 30, 25, 22, 29])
        want = small.attend_shared(q, prefix, i32([190, 180]), table, lens, **args)
        got = big.attend_shared(q, move(prefix), i32([190, 180]), move(table), lens, **args)
        assert all(torch.equal(a, b) for a, b in zip(got, want)) and torch.isfinite(want[0]).all()
    # copies and compaction across the border
    refs = torch.zeros(blocks, dtype=torch.int32, device="cuda")
    refs[top] = 1
    pages, tables = kvx.Pages(refs, bs), [move(prefix), move(table)]
    kvx.copy_pages([big], torch.stack([top[:2].int(), i32([7, blocks - 2])], 1).contiguous())
    assert torch.equal(big.v_codes[7], small.v_codes[0]) and torch.equal(big.k_codes[blocks - 2], small.k_codes[1])
    used, moved = pages.compact(tables, [big])
    assert int(used.item()) == few and torch.equal(moved[top], torch.arange(few, device="cuda").int())
    assert torch.equal(tables[0], prefix) and torch.equal(tables[1], table)
    for a, b in ((big.k_codes, small.k_codes), (big.v_codes, small.v_codes), (big.k_scale, small.k_scale),
                 (big.v_scale, small.v_scale)):
        assert torch.equal(a[:few], b)
    assert (refs[:few] == 1).all() and (refs[few:] == 0).all()


def test_logits_beyond_four_gigabytes():
    rows, V = 8704, 262_144                                  # 4.6 GB in bf16
    g = torch.Generator(device="cuda").manual_seed(5)
    logits = torch.empty((rows, V), dtype=torch.bfloat16, device="cuda")
    for r in range(0, rows, 1088):
        logits[r:r + 1088] = 3 * torch.randn((1088, V), generator=g, device="cuda")
    scores = torch.randn((rows // 8, 8), generator=g, device="cuda")
    tokens, parents, new, _ = kvx.beam_select(logits, scores)
    last = kvx.beam_select(logits[-16:].clone(), scores[-2:])
    assert torch.equal(tokens[-2:], last[0]) and torch.equal(parents[-2:], last[1] + rows - 16)
    # a row's sum of exponentials is formed by other CTAs, in another order
    assert (new[-2:] - last[2]).abs().max() < 2.0 ** -16


def test_many_requests():
    """More rows, groups and requests than threads or lanes anywhere."""
    R, P, H, d, bs = 5000, 2100, 1, 16, 8
    g = torch.Generator().manual_seed(7)
    cuts = torch.randint(0, R + 1, (P - 1,), generator=g).sort()[0].tolist()
    groups = i32([0] + cuts + [R])                          # many groups without requests
    blocks = 4000
    cache = kvx.Cache8(*(torch.randint(0, 0x70, (blocks, H, bs, d), generator=g, dtype=torch.uint8).cuda() for _ in range(2)),
                       *(torch.full((blocks, H), 2.0 ** -9, device="cuda") for _ in range(2)))
    pick = lambda *s: torch.randint(0, blocks, s, generator=g).int().cuda()
    prefix, table = pick(P, 3), pick(R, 2)
    before = torch.randint(0, 25, (P,), generator=g).int().cuda()
    lens = torch.randint(0, 17, (R,), generator=g).int().cuda()
    for dtype in (torch.bfloat16, torch.float32):
        q = torch.randn((R, 2, d), generator=g).to(dtype).cuda()
        status = i32([0])
        most = int((groups[1:] - groups[:-1]).max().item())
        out, lse = cache.attend_shared(q, prefix, before, table, lens, max_prefix=24, max_len=16, groups=groups,
                                       max_group=most, status=status)
        assert int(status.item()) == 0
        # each request as one sequence of its own, in plain fp64
        of = torch.searchsorted(groups[1:].contiguous(), torch.arange(R, device="cuda"), right=True)

        def values(codes, scale, t):
            x = codes[t.long()].view(torch.float8_e4m3fn).double() * scale[t.long()][..., None, None].double()
            return x[:, :, 0].reshape(R, -1, d)

        k = torch.cat([values(cache.k_codes, cache.k_scale, t) for t in (prefix[of], table)], 1)
        v = torch.cat([values(cache.v_codes, cache.v_scale, t) for t in (prefix[of], table)], 1)
        j = torch.arange(40, device="cuda")
        seen = torch.where(j < 24, j < before[of][:, None], j - 24 < lens[:, None])
        x = torch.einsum("rgd,rjd->rgj", q.double(), k) * d ** -0.5
        x = x.masked_fill(~seen[:, None], float("-inf"))
        want = torch.logsumexp(x, -1)
        p = torch.where(seen[:, None], torch.exp(x - want[..., None]), torch.zeros((), dtype=torch.float64, device="cuda"))
        o = p @ v
        empty = ~seen.any(1)
        assert torch.equal(torch.isneginf(lse), empty[:, None].expand(-1, 2)) and (out[empty] == 0).all()
        # scores below 2^5 here, known to 2^-16 of their terms' sum; probabilities in bf16's form to
        # 2^-10, outputs half an ulp besides
        reach = (q.double().abs()[:, :, None] * k.abs()[:, None]).sum(-1).amax() * d ** -0.5
        xe = 2.0 ** -16 * reach
        mass = p @ v.abs()
        tol = (4 * xe + 2.0 ** -17 + (2.0 ** -10 if dtype is torch.bfloat16 else 0)) * mass + \
            (2.0 ** -8 * o.abs() if dtype is torch.bfloat16 else 0) + 1e-30
        assert ((out.double() - o).abs() <= tol).all()
        live = ~empty
        assert ((lse.double() - want)[live].abs() <= xe + 2.0 ** -19 * (1 + want[live].abs())).all()
    # a fork and a reservation of as many rows
    pages = kvx.Pages.empty(30_000, bs)
    t, zero = torch.full((R, 3), -1, dtype=torch.int32, device="cuda"), torch.zeros(R, dtype=torch.int32, device="cuda")
    status = i32([0])
    pages.reserve(t, zero, lens, max_new=16, status=status)
    assert torch.equal((t >= 0).sum(1), (lens + bs - 1) // bs) and t.max() + 1 == (t >= 0).sum()
    parents = torch.randint(0, R, (R,), generator=g).int().cuda()
    n, l = pages.fork(t, lens, parents, status=status)
    assert torch.equal(n, t[parents.long()]) and torch.equal(l, lens[parents.long()])
    assert torch.equal(pages.refs, torch.bincount(n[n >= 0].long(), minlength=30_000).int())
    pages.reserve(n, l, 5, status=status)
    first = n.gather(1, (l.long() // bs)[:, None])
    assert int(status.item()) == 0 and (pages.refs[first.long()] == 1).all()
    assert torch.equal(pages.refs, torch.bincount(n[n >= 0].long(), minlength=30_000).int())
