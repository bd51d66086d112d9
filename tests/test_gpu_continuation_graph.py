"""A beam step captured into a CUDA graph, and the calls on another stream: replays give
what the calls give.  Two graphs share the workspaces."""
import pytest
import torch

from cross_model_kv_transfer_gb300 import kvx

pytestmark = pytest.mark.gpu


def make(dtype, d):
    P, K, H, G, bs, n, V = 2, 3, 2, 4, 16, 90, 700
    R = P * K
    g = torch.Generator().manual_seed(7)
    draw = lambda *s: torch.randn(s, generator=g).to(dtype).cuda()
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")
    fixed = dict(old=(draw(P * n, H, d), draw(P * n, H, d)), q=draw(R, H * G, d), k=draw(R, H, d), v=draw(R, H, d),
                 logits=draw(R, V), scores=torch.randn((P, K), generator=g).cuda(), lens=i32([5, 5, 16, 9, 9, 9]),
                 own=(draw(R * 20, H, d), draw(R * 20, H, d)))
    scratch = {}

    def prepare():
        blocks = 64
        cache, pages = kvx.Cache8.empty(blocks, H, d, bs), kvx.Pages.empty(blocks, bs)
        prefix = torch.full((P, 8), -1, dtype=torch.int32, device="cuda")
        table = torch.full((R, 4), -1, dtype=torch.int32, device="cuda")
        before, groups = i32([n, n - 7]), i32([0, K, R])
        pages.reserve(prefix, i32([0, 0]), n)
        cache.write(*fixed["old"], prefix, cu_seqlens=i32([0, n, 2 * n]))
        # rows 0 and 1, and 3 to 5, share what they hold
        pages.reserve(table, i32([0] * R), fixed["lens"], max_new=20)
        cache.write(*fixed["own"], table, cu_seqlens=i32([0] + fixed["lens"].cumsum(0).tolist()),
                    src_rows=i32(list(range(int(fixed["lens"].sum())))))
        table, lens = pages.fork(table, fixed["lens"], i32([0, 0, 2, 3, 3, 3]))
        if not scratch:
            scratch["pages"] = pages.workspace()
            scratch["attend"] = cache.attend_shared_workspace(ntok=R, num_requests=R, q_heads=H * G, num_prefixes=P,
                                                              max_prefix=n, max_len=40, max_group=K, dtype=dtype)
            scratch["beam"] = kvx.beam_workspace(requests=P, beams=K, vocab=V)
        status = i32([0])
        torch.cuda.synchronize()

        def step(stream=None):
            s = dict(status=status, stream=stream)
            copies = torch.empty((R, 2), dtype=torch.int32, device="cuda")
            pages.reserve(table, lens, 1, caches=[cache], workspace=scratch["pages"], copies=copies, **s)
            cache.write(fixed["k"], fixed["v"], table, start=lens, **s)
            out, lse = cache.attend_shared(fixed["q"], prefix, before, table, after, groups=groups, max_prefix=n,
                                           max_len=40, max_group=K, workspace=scratch["attend"], **s)
            tokens, parents, scores, _ = kvx.beam_select(fixed["logits"], fixed["scores"], workspace=scratch["beam"], **s)
            new_table, new_lens = pages.fork(table, after, parents.view(-1), **s)
            used, moved = pages.compact([prefix, new_table], [cache], workspace=scratch["pages"], **s)
            return (copies, out, lse, tokens, parents, scores, new_table, new_lens, used, moved, prefix, pages.refs,
                    cache.k_codes, cache.v_codes, cache.k_scale, cache.v_scale, status)

        after = lens + 1
        return step
    return prepare


@pytest.mark.parametrize("dtype,d", [(torch.bfloat16, 128), (torch.float32, 64)])
def test_captured_steps_and_streams(dtype, d):
    prepare = make(dtype, d)
    want = [t.clone() for t in prepare()()]
    torch.cuda.synchronize()
    assert int(want[-1].item()) == 0
    same = lambda got: all(torch.equal(a.view(torch.uint8), b.view(torch.uint8)) for a, b in zip(got, want))
    graphs = []
    for _ in range(2):
        step, graph = prepare(), torch.cuda.CUDAGraph()
        torch.cuda.synchronize()
        with torch.cuda.graph(graph):
            got = step()
        graphs.append((graph, got))
    for graph, got in graphs:          # one after the other, in the same workspaces
        graph.replay()
    torch.cuda.synchronize()
    assert all(same(got) for _, got in graphs)
    step, side = prepare(), torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = step(side)
    side.synchronize()
    assert same(got)
