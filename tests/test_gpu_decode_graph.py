"""A decoding step captured into a CUDA graph: replays give what the calls give."""
import pytest
import torch

from cross_model_kv_transfer_gb300 import kvx

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype,d,new", [(torch.bfloat16, 128, 1), (torch.bfloat16, 128, 20),
                                         (torch.float32, 64, 1)])
def test_a_captured_step(dtype, d, new):
    R, H, G, bs, keep, most = 3, 2, 4, 16, 48, 200
    per, fresh = -(-most // bs), -(-keep // bs)
    order = torch.randperm(R * (per + fresh), generator=torch.Generator().manual_seed(3)).int().cuda()
    table, to = order[:R * per].view(R, per), order[R * per:].view(R, fresh)
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")
    held = i32([0, 70, most - new])
    cu, positions = i32(list(range(0, R * new + 1, new))), i32(list(range(R * new)))
    rng = torch.Generator().manual_seed(5)
    draw = lambda n, heads: torch.randn((n, heads, d), generator=rng).to(dtype).cuda()
    q, k, v = draw(R * new, H * G), draw(R * new, H), draw(R * new, H)
    old = draw(R * most, H), draw(R * most, H)
    rope, status = kvx.Rope(d, 1e4), i32([0])
    after = held + new

    def prepare():
        cache = kvx.Cache8.empty(R * (per + fresh), H, d, bs)
        cache.write(*old, table, cu_seqlens=i32([0, most, 2 * most, 3 * most]), status=status)
        scratch = cache.attend_workspace(ntok=R * new, num_requests=R, q_heads=H * G, max_len=most,
                                         max_new=new, dtype=dtype, weights=True)
        room = cache.evict_workspace(num_requests=R, max_len=most, keep=keep)
        weights = torch.zeros((R, H, most), device="cuda")

        def step():
            rq, rk = rope.apply(q, k, positions, status=status)
            cache.write(rk, v, table, start=held, cu_seqlens=cu, status=status)
            out, lse = cache.attend(rq, table, after, most, cu_seqlens=cu, max_new=new,
                                    weights=weights, workspace=scratch, status=status)
            kept = cache.evict(weights, table, after, to, max_len=most, keep=keep, sinks=2, recent=8,
                               workspace=room, status=status)
            return (out, lse, weights, *kept, cache.k_codes, cache.v_codes, cache.k_scale,
                    cache.v_scale)
        return step

    want = [t.clone() for t in prepare()()]
    step = prepare()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    graph.replay()
    torch.cuda.synchronize()
    assert int(status.item()) == 0
    for a, b in zip(got, want):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
