"""fp32 rotary positions to fp32's own precision.

(1, 0) turned gives the cosine and the sine themselves.  The phase is exact to
2^-32 of a turn (1.5e-9 rad) and rounded to fp32 after whole quarter turns (half
an ulp of a quarter's half: 2.4e-8 rad); CUDA's sincospif is within 1 ulp of its
value, 6e-8 up to 1.  Together 8.6e-8; the frequency itself is off by a few
2^-64 of a turn a position.  A general pair adds three roundings of 2^-24, of
values up to |x0| + |x1|."""
import numpy as np
import pytest
import torch

import decode_reference as ref
from cross_model_kv_transfer_gb300 import kvx

pytestmark = pytest.mark.gpu


def phases(pos, w):
    """pos * w mod 2 pi in fp64, good to 1e-11 for positions below 2^18."""
    turns = w / (2 * np.pi)
    return 2 * np.pi * ((pos[:, None] * turns) % 1.0)


@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("d,theta", [(128, 1e4), (64, 5e5), (18, 1e4)])      # the last: one pair a thread
def test_cosines_and_sines(d, theta, layout):
    n = 20000
    pos = torch.arange(n, dtype=torch.int32) * 11 + 3
    x = torch.zeros((n, 1, d))
    even = np.arange(d // 2) if layout == "half" else 2 * np.arange(d // 2)
    odd = even + (d // 2 if layout == "half" else 1)
    x[..., even] = 1.0
    y = kvx.Rope(d, theta, layout=layout).apply(x.cuda(), positions=pos.cuda())[0].double().cpu().numpy()[:, 0]
    w, _ = ref.frequencies(d, theta)
    a = phases(pos.double().numpy(), w)
    assert np.abs(y[:, even] - np.cos(a)).max() <= 9e-8
    assert np.abs(y[:, odd] - np.sin(a)).max() <= 9e-8


@pytest.mark.parametrize("transpose", [False, True])
def test_rows_of_any_values(transpose):
    n, h, d = 4000, 3, 128
    g = torch.Generator().manual_seed(2)
    x = torch.randn((n, h, d), generator=g)
    pos = torch.randint(0, 131072, (n,), generator=g, dtype=torch.int32)
    y = kvx.Rope(d, 1e4).apply(x.cuda(), positions=pos.cuda(), transpose=transpose)[0].double().cpu().numpy()
    w, amp = ref.frequencies(d, 1e4)
    want = ref.rope(x.double().numpy(), pos.double().numpy(), d, "half", w, amp, transpose)
    x = np.abs(x.double().numpy())
    sums = np.concatenate([x[..., :64] + x[..., 64:]] * 2, -1)
    assert (np.abs(y - want) <= (9e-8 + 3 * 2.0 ** -24) * sums).all()
