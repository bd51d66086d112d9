"""Eviction of rows of zero codes that shared a block with large values: their new
block's scale is as small as scales get, and zeros they stay."""
import numpy as np
import pytest
import torch

import decode_reference as ref
from test_gpu_evict8 import check, dev, make

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("scale", [2.0 ** -126, 1.0, 4.0, 2.0 ** 20, 2.0 ** 118])
@pytest.mark.parametrize("d,bs,keep", [(64, 16, 1), (64, 16, 20), (128, 128, 100), (16, 7, 3)])
def test_zero_rows_stay_zero(d, bs, keep, scale):
    """Every row that stays is zero in K, and in V's odd heads; `scale` is that of all blocks."""
    H, n = 2, 300
    c = make(H, d, bs, [n], keep, 21)
    for m, codes, scales, cache_codes, cache_scale in ((0, c["kc"], c["ks"], c["cache"].k_codes, c["cache"].k_scale),
                                                       (1, c["vc"], c["vs"], c["cache"].v_codes, c["cache"].v_scale)):
        scales[c["table"][0]] = scale
        kept = ref.evict(c["w"], [n], keep, 0, 0)
        for h in range(H):
            if m and h % 2 == 0:
                continue
            for j in kept[0, h]:
                codes[c["table"][0][j // bs], h, j % bs] = 0x80 if j % 3 == 0 else 0
        cache_codes.copy_(torch.tensor(codes))
        cache_scale.copy_(torch.tensor(scales))
    check(c, keep, 0, 0)
    page = int(c["to"][0][0])
    assert (c["cache"].k_scale[page] == 2.0 ** -126).all()
    # attention over them: zeros, not NaN
    q = torch.ones((1, H, d), dtype=torch.bfloat16, device="cuda")
    if bs % 8 == 0:
        out, lse = c["cache"].attend(q, dev(c["to"]), dev([keep]), keep)
        assert torch.isfinite(lse).all() and (out[:, 1] == 0).all()


@pytest.mark.parametrize("bs", [16, 128])
def test_zero_rows_beside_small_ones(bs):
    """A block that takes zeros from under a large scale and tiny values from under a
    small one."""
    H, d, n, keep = 1, 128, 4 * bs, bs
    c = make(H, d, bs, [n], keep, 22)
    t = c["table"][0]
    for codes, scales, cc, cs in ((c["kc"], c["ks"], c["cache"].k_codes, c["cache"].k_scale),
                                  (c["vc"], c["vs"], c["cache"].v_codes, c["cache"].v_scale)):
        scales[t[0]], codes[t[0], 0, :bs // 2] = 2.0 ** 40, 0
        scales[t[1]] = 2.0 ** -122
        cc.copy_(torch.tensor(codes))
        cs.copy_(torch.tensor(scales))
    c["w"][:] = 0
    c["w"][0, 0, :bs // 2] = 2
    c["w"][0, 0, bs:bs + bs // 2] = 1
    check(c, keep, 0, 0)
    got = c["cache"].v_codes[int(c["to"][0][0]), 0].cpu().numpy()
    assert not np.isnan(ref.E4M3[got]).any()
