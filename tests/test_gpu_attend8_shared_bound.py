"""Shared attention of one prefix for all requests, given without a group table: a bound
on the group that its queries exceed is refused as one of a table's groups is."""
import pytest
import torch

from cross_model_kv_transfer_gb300 import kvx
from test_gpu_attend8_shared import call, check, dev, make

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("H,G,d,bs,prefix,lens,news", [
    (1, 4, 64, 16, 50, [4, 5, 6, 7, 8], [1] * 5),           # few rows: prefix in parts
    (1, 4, 64, 16, 0, [4, 5, 6, 7, 8], [1] * 5),            # no slots before: one result
    (1, 8, 128, 16, 9000, [3] * 64, [1] * 64),              # a prefix of much work
    (1, 2, 64, 16, 300, [2100, 5], [1, 1]),                 # more own slots than an item's CTA takes
    (2, 13, 128, 16, 90, [100, 30], [5, 4]),                # more rows than it takes
    (1, 12, 64, 7, 50, [20, 9], [1, 2]),
])
def test_a_group_above_its_bound_writes_nothing(H, G, d, bs, prefix, lens, news, dtype):
    c = make(H, G, d, bs, [prefix], [len(lens)], lens, news, dtype, 47)
    n, most, R = sum(news), max(news), len(lens)
    one_token = most == 1
    for few in {1, R - 1}:
        if few * most >= n:
            continue
        for cu in ((dev(c["cu"]), None) if one_token else (dev(c["cu"]),)):
            out = torch.full((n, H * G, d), 7.0, dtype=dtype, device="cuda")
            lse = torch.full((n, H * G), 7.0, device="cuda")
            status = torch.zeros(1, dtype=torch.int32, device="cuda")
            call(c, groups=None, cu_seqlens=cu, max_group=few, out=out, lse=lse, status=status)
            assert (out == 7).all() and (lse == 7).all(), few
            assert int(status.item()) == kvx.KVX_FLAG_BAD_SEQLENS, few
    check(c, groups=None, max_group=R)
