"""Shared attention whose tables are refused: a call behind it on the same stream and in
the same workspace gives what it gives alone."""
import pytest
import torch

from cross_model_kv_transfer_gb300 import kvx
from test_gpu_attend8_shared import call, check, dev, make

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("news,cu,kw", [
    ([3], [0, 2], dict(groups=None, max_new=3, max_group=1)),     # does not end at the last query
    ([2, 0], [0, 2, 2], dict(max_new=1, max_group=2)),            # a request above max_new beside an empty one
    ([0, 4, 0], [0, 0, 4, 4], dict(max_new=2, max_group=3)),
])
def test_a_good_call_behind_a_refused_one(news, cu, kw, dtype):
    """No CTA of the refused call's own slots has a query, while its prefix, which is good,
    is worked on in full."""
    bad = make(1, 8, 128, 16, [6000], [len(news)], [20] * len(news), news, dtype, 41)
    good = make(1, 8, 128, 16, [3000], [2], [9, 33], [1, 1], dtype, 43)
    ws = bad["cache"].attend_shared_workspace(ntok=8, num_requests=3, q_heads=8, max_prefix=6000, max_len=33,
                                              max_group=3, max_new=4, dtype=dtype)
    want = check(good)
    n = sum(news)
    for _ in range(20):
        out = torch.full((n, 8, 128), 7.0, dtype=dtype, device="cuda")
        lse = torch.full((n, 8), 7.0, device="cuda")
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        call(bad, out=out, lse=lse, status=status, cu_seqlens=dev(cu), workspace=ws, **kw)
        got = call(good, workspace=ws)
        assert all(torch.equal(a, b) for a, b in zip(got, want))
        assert (out == 7).all() and (lse == 7).all() and int(status.item()) == kvx.KVX_FLAG_BAD_SEQLENS
