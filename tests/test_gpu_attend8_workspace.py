"""One workspace for calls of several sizes and forms (kvx_attend8): requests and
queries that grow and shrink, fp32 and bf16 queries, with and without weights.
Outputs hold a sentinel before each call: what nobody wrote shows.  Tolerances
as in test_gpu_attend8.py."""
import numpy as np
import pytest
import torch

import decode_reference as ref
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
