"""Workspaces that the decoding calls cannot use are refused before anything is
enqueued: other devices, views with gaps, too few bytes; bytes are counted as
such whatever the tensor's type."""
import pytest
import torch

from cross_model_kv_transfer_gb300 import kvx
from test_gpu_evict8 import dev, make

pytestmark = pytest.mark.gpu


def calls():
    c = make(1, 64, 16, [90], 32, 41)
    cache, table, lens = c["cache"], dev(c["table"]), dev([90])
    q = torch.randn((1, 2, 64), device="cuda")
    w = torch.tensor(c["w"]).cuda()
    attend_ws = cache.attend_workspace(ntok=1, num_requests=1, q_heads=2, max_len=90, dtype=q.dtype)
    evict_ws = cache.evict_workspace(num_requests=1, max_len=90, keep=32)
    return [(attend_ws, lambda ws: cache.attend(q, table, lens, 90, workspace=ws)[0]),
            (evict_ws, lambda ws: cache.evict(w, table, lens, dev(c["to"]), max_len=90, keep=32, workspace=ws)[0])]


@pytest.mark.parametrize("which", [0, 1])
def test_workspaces(which):
    ws, call = calls()[which]
    want = call(ws)
    n = ws.numel()
    for bad in (ws.cpu(), torch.zeros((2, 2 * n), dtype=torch.uint8, device="cuda")[:, ::2],
                torch.zeros((n, 2), dtype=torch.uint8, device="cuda")[:, 0]):
        with pytest.raises(ValueError, match="workspace"):
            call(bad)
    for few in (ws[:-256] if n > 256 else ws[:0], torch.zeros(n // 4 - 64, device="cuda")):
        with pytest.raises(kvx.KvxError):
            call(few)
    assert torch.equal(call(torch.zeros(n // 4, device="cuda")), want)
