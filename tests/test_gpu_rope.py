"""Rotary positions (kvx_rope_apply) against the formula in fp64: layouts, part
of the head, scaled frequencies, strides, in place, the gradient, flags.

Tolerance: the angle is off by at most ~4e-7 rad (32-bit phase and its fp32
form) and __sincosf by ~4e-7 more, two products and a sum round three times
(2^-24 each): |error| <= 1.5e-6 a (|x0| + |x1|); twice that is allowed.  bf16
output adds half an ulp, 2^-9 |y|, allowed as 2^-8 |y|."""
import numpy as np
import pytest
import torch

import decode_reference as ref
from cross_model_kv_transfer_gb300 import kvx

pytestmark = pytest.mark.gpu

SCALINGS = {
    "none": {},
    "linear": dict(scaling="linear", factor=4.0),
    "bands": dict(scaling="bands", factor=8.0, low_band=1.0, high_band=4.0, original_context=8192),
    "yarn": dict(scaling="yarn", factor=4.0, beta_fast=32.0, beta_slow=1.0, original_context=4096),
}


def pairs_sum(x, rot, layout):
    """|x0| + |x1| of each element's pair (0 for copied dims)."""
    i = np.arange(rot // 2)
    i0, i1 = (i, i + rot // 2) if layout == "half" else (2 * i, 2 * i + 1)
    s = np.zeros_like(x)
    s[..., i0] = s[..., i1] = np.abs(x[..., i0]) + np.abs(x[..., i1])
    return s


def check(x, y, pos, rot, layout, theta, scaling, transpose, bf16):
    w, amp = ref.frequencies(rot, theta, **scaling)
    want = ref.rope(x, pos, rot, layout, w, amp, transpose)
    tol = 3e-6 * amp * pairs_sum(x, rot, layout) + (2.0 ** -8 * np.abs(want) if bf16 else 0)
    assert (np.abs(y - want) <= tol).all(), np.abs(y - want).max()
    assert np.array_equal(y[..., rot:], x[..., rot:])


@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("n,hq,hk,d,rot,scaling", [
    (1, 1, 1, 128, 128, "none"), (16, 64, 8, 128, 128, "bands"), (37, 5, 1, 64, 32, "yarn"),
    (300, 7, 3, 96, 48, "linear"), (3, 2, 2, 80, 80, "none"), (5, 3, 1, 18, 6, "yarn"),
    (2, 2, 1, 256, 256, "bands"), (9, 71, 1, 64, 64, "none"), (4, 1, 1, 2, 2, "none"),
    (2500, 16, 8, 128, 64, "bands")])
def test_matches_the_formula(n, hq, hk, d, rot, scaling, dtype, layout):
    g = torch.Generator().manual_seed(n + d)
    q, k = (torch.randn((n, h, d), generator=g).to(dtype) for h in (hq, hk))
    pos = torch.randint(0, 131072, (n,), generator=g, dtype=torch.int32)
    kw = SCALINGS[scaling]
    rope = kvx.Rope(d, 5e5, rot_dim=rot, layout=layout, **kw)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    for transpose in (False, True):
        yq, yk = rope.apply(q.cuda(), k.cuda(), pos.cuda(), transpose=transpose, status=status)
        for x, y in ((q, yq), (k, yk)):
            check(x.double().numpy(), y.double().cpu().numpy(), pos.double().numpy(), rot, layout,
                  5e5, kw, transpose, dtype == torch.bfloat16)
    assert int(status.item()) == 0


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("width,off", [(0, 0), (3, 1), (8, 8)])
def test_views_in_place_and_one_of_the_two(dtype, width, off):
    n, hq, hk, d = 33, 6, 2, 64
    g = torch.Generator().manual_seed(3)
    flat = torch.randn((n, (hq + 2 * hk) * d + width), generator=g).to(dtype).cuda()
    view = flat[:, off:off + (hq + 2 * hk) * d].unflatten(1, (hq + 2 * hk, d))
    before = flat.clone()
    q, k = view[:, :hq], view[:, hq:hq + hk]
    x = view.double().cpu().numpy()
    rope = kvx.Rope(d, 1e4)
    got, none = rope.apply(q, first_position=70000)
    assert none is None
    pos = 70000.0 + np.arange(n)
    check(x[:, :hq], got.double().cpu().numpy(), pos, d, "half", 1e4, {}, False,
          dtype == torch.bfloat16)
    rope.apply(q, k, first_position=70000, q_out=q, k_out=k)
    y = view.double().cpu().numpy()
    check(x[:, :hq + hk], y[:, :hq + hk], pos, d, "half", 1e4, {}, False, dtype == torch.bfloat16)
    assert np.array_equal(y[:, hq + hk:], x[:, hq + hk:])
    outside = torch.ones_like(flat, dtype=torch.bool)
    outside[:, off:off + (hq + hk) * d] = False
    assert torch.equal(flat[outside], before[outside])
    # heads as the outer dimension
    t = torch.randn((hk, n, d), generator=g).to(dtype).cuda()
    _, got = rope.apply(None, t.transpose(0, 1), torch.arange(n, dtype=torch.int32, device="cuda"))
    check(t.transpose(0, 1).double().cpu().numpy(), got.double().cpu().numpy(), np.arange(n) * 1.0,
          d, "half", 1e4, {}, False, dtype == torch.bfloat16)


def test_the_gradient_is_the_transposed_rotation():
    """<R x, y> = <x, R^T y>, and the gradient of sum(y * R x) by differences:
    R is linear, so central differences carry only fp32 rounding."""
    n, h, d = 5, 3, 32
    g = torch.Generator().manual_seed(5)
    x, y = (torch.randn((n, h, d), generator=g).cuda() for _ in range(2))
    pos = torch.randint(0, 99999, (n,), generator=g, dtype=torch.int32).cuda()
    rope = kvx.Rope(d, 1e4, rot_dim=24, layout="interleaved", **SCALINGS["yarn"])
    f = lambda t: rope.apply(t, positions=pos)[0]
    grad = rope.apply(y, positions=pos, transpose=True)[0]
    lhs, rhs = (f(x).double() * y).sum(), (x.double() * grad).sum()
    # n h d products of size ~amp^1, each within 3e-6 (|x0| + |x1|) |y|
    assert abs(lhs - rhs) <= 2 * 3e-6 * 1.2 * 2 * (x.abs().double().sum() * y.abs().max())
    for i, j, e in ((0, 0, 0), (2, 1, 7), (4, 2, 23), (3, 0, 31)):
        step = torch.zeros_like(x)
        step[i, j, e] = 1.0
        num = ((f(x + step).double() - f(x - step).double()) / 2 * y).sum()
        # |x| + 1 below 6: each of the two forwards within 3e-6 * 1.2 * 12 on two elements
        assert abs(num - grad[i, j, e]) <= 2e-4


def test_positions_out_of_range_are_skipped_and_flagged():
    rope = kvx.Rope(64, 1e4)
    q = torch.ones((3, 2, 64), device="cuda")
    out = torch.full_like(q, 7.0)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    rope.apply(q, positions=torch.tensor([0, -1, 5], dtype=torch.int32, device="cuda"), q_out=out,
               status=status)
    assert int(status.item()) == kvx.KVX_FLAG_BAD_POSITION
    assert torch.equal(out[1], torch.full_like(out[1], 7.0))
    assert torch.equal(out[0], q[0]) and not torch.equal(out[2], q[2])


def test_no_tokens_and_another_stream():
    rope = kvx.Rope(128, 1e6)
    out, _ = rope.apply(torch.empty((0, 4, 128), device="cuda"))
    assert out.shape == (0, 4, 128)
    s = torch.cuda.Stream()
    x = torch.randn((1000, 8, 128), device="cuda")
    s.wait_stream(torch.cuda.current_stream())
    y, _ = rope.apply(x, stream=s)
    torch.cuda.current_stream().wait_stream(s)
    check(x.double().cpu().numpy(), y.double().cpu().numpy(), np.arange(1000.0), 128, "half", 1e6,
          {}, False, False)
