"""One workspace for calls of several sizes and forms (kvx_attend8): requests and
queries that grow and shrink, fp32 and bf16 queries, with and without weights.
Outputs hold a sentinel before each call: what nobody wrote shows.  Tolerances
as in test_gpu_attend8.py."""
import numpy as np
import pytest
import torch

import decode_reference as ref
from cross_model_kv_transfer_gb300 import kvx
from test_gpu_attend8 import compare, dev, make

pytestmark = pytest.mark.gpu

# R, new: a batch that grows and shrinks, chunks between single tokens
STEPS = [(2, 1), (16, 1), (64, 1), (3, 5), (64, 1), (1, 40), (16, 5), (64, 1), (2, 70), (40, 3)]


def inputs(R, new, H, G, d, bs, dtype, seed):
    lens = [new + (37 * r + 11) % 500 for r in range(R)]
    c = make(H, G, d, bs, lens, [new] * R, dtype, seed)
    want = ref.attend(c["q"].double().numpy(), c["rk"], c["rv"], c["table"], lens, c["cu"], d ** -0.5)
    return c, lens, want


def call(c, lens, want, R, new, H, G, dtype, ws, weights):
    most = max(lens)
    q = c["q"].cuda()
    out = torch.full_like(q, 1e30)
    lse = torch.full((R * new, H * G), 1e30, device="cuda")
    w = torch.zeros((R, H, most), device="cuda") if weights else None
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    c["cache"].attend(q, dev(c["table"]), dev(lens), most, cu_seqlens=dev(c["cu"]), max_new=new, out=out, lse=lse,
                      weights=w, workspace=ws, status=status)
    assert int(status.item()) == 0
    compare(out, lse, w, want, dtype == torch.bfloat16, most, new * G)


@pytest.mark.parametrize("d,bs,dtypes", [(64, 16, [torch.float32]), (64, 16, [torch.float32, torch.bfloat16]),
                                         (128, 24, [torch.float32]), (64, 7, [torch.bfloat16, torch.float32]),
                                         (256, 16, [torch.bfloat16])])
@pytest.mark.parametrize("weights", [False, True])
def test_one_workspace_for_calls_that_grow_and_shrink(d, bs, dtypes, weights):
    H, G = 8, 2
    made = [(R, new, dt, *inputs(R, new, H, G, d, bs, dt, 3 + i))
            for i, (R, new) in enumerate(STEPS) for dt in dtypes]
    spaces = [c["cache"].attend_workspace(ntok=R * new, num_requests=R, q_heads=H * G, max_len=max(lens), max_new=new,
                                          dtype=dt, weights=weights) for R, new, dt, c, lens, _ in made]
    ws = torch.zeros(max(s.numel() for s in spaces), dtype=torch.uint8, device="cuda")
    for turn in range(2):
        for R, new, dt, c, lens, want in made:
            call(c, lens, want, R, new, H, G, dt, ws, weights)


@pytest.mark.parametrize("G,max_new", [(2, 2 ** 31 - 1), (8, 2 ** 29)])
@pytest.mark.parametrize("new", [1, 130, 420])
def test_any_bound_on_a_requests_queries(G, max_new, new):
    H, lens, news = 2, [500, 60], [new, 1]
    c = make(H, G, 128, 16, lens, news, torch.bfloat16, 53)
    want = ref.attend(c["q"].double().numpy(), c["rk"], c["rv"], c["table"], lens, c["cu"], 128 ** -0.5)
    w = torch.zeros((2, H, 500), device="cuda")
    out = torch.full(c["q"].shape, 1e30, dtype=torch.bfloat16, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    _, lse = c["cache"].attend(c["q"].cuda(), dev(c["table"]), dev(lens), 500, cu_seqlens=dev(c["cu"]), max_new=max_new,
                               out=out, weights=w, status=status)
    assert int(status.item()) == 0
    compare(out, lse, w, want, True, 500, new * G)


@pytest.mark.parametrize("d,bs,dtype", [(128, 16, torch.bfloat16), (64, 16, torch.float32)])
@pytest.mark.parametrize("room", ["of the window", "without weights", "of the window without weights"])
def test_a_window_and_then_single_tokens(d, bs, dtype, room):
    """A workspace of large bounds serves small calls; one without room for scores serves
    calls with weights."""
    H, G, R, bound = 8, 8, 16, 16384
    ws = None
    for new in (64, 1, 2, 5, 1):
        lens = [new + (53 * r + 7) % 400 for r in range(R)]
        c = make(H, G, d, bs, lens, [new] * R, dtype, 61 + new)
        want = ref.attend(c["q"].double().numpy(), c["rk"], c["rv"], c["table"], lens, c["cu"], d ** -0.5)
        if ws is None or room == "without weights":
            ws = c["cache"].attend_workspace(ntok=R * new, num_requests=R, q_heads=H * G, max_len=bound, max_new=new,
                                             dtype=dtype, weights="without" not in room)
        w = torch.zeros((R, H, bound), device="cuda")
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        out, lse = c["cache"].attend(c["q"].cuda(), dev(c["table"]), dev(lens), bound, cu_seqlens=dev(c["cu"]),
                                     max_new=new, weights=w, workspace=ws, status=status)
        assert int(status.item()) == 0
        compare(out, lse, w[..., :max(lens)].contiguous(), want, dtype == torch.bfloat16, max(lens), new * G)
        assert not w[..., max(lens):].any()


@pytest.mark.parametrize("G,new,d,dtype", [(8, 1, 128, torch.bfloat16), (4, 10, 128, torch.bfloat16),
                                           (4, 70, 64, torch.bfloat16), (4, 3, 64, torch.float32),
                                           (2, 20, 256, torch.bfloat16)])
def test_only_the_first_1024_bytes_have_to_be_zero(G, new, d, dtype):
    H, lens = 2, [900, 77]
    c = make(H, G, d, 16, lens, [new, new], dtype, 71)
    want = ref.attend(c["q"].double().numpy(), c["rk"], c["rv"], c["table"], lens, c["cu"], d ** -0.5)
    ws = c["cache"].attend_workspace(ntok=2 * new, num_requests=2, q_heads=H * G, max_len=900, max_new=new,
                                     dtype=dtype, weights=True)
    assert not ws[:1024].any()
    ws[1024:] = 0xFF
    for _ in range(2):
        call(c, lens, want, 2, new, H, G, dtype, ws, True)


def test_the_rest_of_a_workspace_is_not_filled():
    """It may be gigabytes: a call without a workspace would spend its time there."""
    cache = kvx.Cache8.empty(4, 2, 128, 16)
    make_ws = lambda: cache.attend_workspace(ntok=1, num_requests=1, q_heads=16, max_len=1 << 22, weights=True)
    ws = make_ws()
    at, size = ws.data_ptr(), ws.numel()
    assert size > 1 << 28
    ws.fill_(0xFF)
    del ws
    ws = make_ws()                        # the allocator gives the same memory again
    assert (ws.data_ptr(), ws.numel()) == (at, size)
    assert not ws[:1024].any() and (ws[1024:] == 0xFF).all()


def test_a_call_without_a_workspace_takes_a_gigabyte_for_scores_at_most():
    c = make(1, 8, 128, 16, [300], [1], torch.bfloat16, 73)
    q, table, lens = c["q"].cuda(), dev(c["table"]), dev([300])
    want = ref.attend(c["q"].double().numpy(), c["rk"], c["rv"], c["table"], [300], c["cu"], 128 ** -0.5)
    taken = []
    for bound in (1 << 20, 1 << 24, 1 << 26, 1 << 28):      # scores of 32 MB, 512 MB, 2 GB, 8 GB
        w = torch.zeros((1, 1, bound), device="cuda")
        torch.cuda.synchronize()
        held = torch.cuda.memory_allocated()
        torch.cuda.reset_peak_memory_stats()
        out, lse = c["cache"].attend(q, table, lens, bound, weights=w)
        taken.append(torch.cuda.max_memory_allocated() - held)
        compare(out, lse, w[..., :300].contiguous(), want, True, 300, 8)
        del w
    assert taken[0] < 1 << 26 and 1 << 29 <= taken[1] < 1 << 30 and max(taken[2:]) < 1 << 26


@pytest.mark.parametrize("G,new,d,dtype", [(8, 1, 128, torch.bfloat16), (4, 10, 128, torch.bfloat16),
                                           (4, 140, 128, torch.bfloat16), (4, 3, 64, torch.float32),
                                           (2, 40, 256, torch.bfloat16)])
def test_outputs_over_the_queries(G, new, d, dtype):
    H, R = 2, 30
    lens = [new + (61 * r) % 700 for r in range(R)]
    c = make(H, G, d, 16, lens, [new] * R, dtype, 79)
    want = ref.attend(c["q"].double().numpy(), c["rk"], c["rv"], c["table"], lens, c["cu"], d ** -0.5)
    q = c["q"].cuda()
    out, lse = c["cache"].attend(q, dev(c["table"]), dev(lens), max(lens), cu_seqlens=dev(c["cu"]), max_new=new, out=q)
    assert out is q
    compare(out, lse, None, want, dtype == torch.bfloat16, max(lens), new * G)
