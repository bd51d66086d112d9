"""Attention over the 8-bit cache where scores are far larger than any healthy
model's: queries that nobody wrote (padding of a captured batch) or a finite
outlier.  Such a row has to end and give the softmax of its scores, and the
ordinary rows beside it must not notice.

Scores of size S are known to about 2^-16 S (test_gpu_attend8.py), so what is
asked for is what that leaves certain: a slot whose score is a quarter or more
above all others takes all of the weight, slots with the same key share it.
Then p is 1 or 1 / n to 2^-20 (sums of a few equal terms), and an output is off
by its own rounding (bf16: 2^-8 |o|) and 2^-20 of sum p |v|; bf16 forms round p
to 2^-10 of itself before its product with v where it is no power of two."""
import numpy as np
import pytest
import torch

import decode_reference as ref
from cross_model_kv_transfer_gb300 import kvx
from test_gpu_attend8 import compare, dev, make

pytestmark = pytest.mark.gpu

SIZES = [2.0 ** 17, 2.0 ** 24, 2.0 ** 27, 1e9, 2.0 ** 36, 1e20, 1e30]
# few rows of each (request, KV head) to many: H, G, new
FEW8, FEW16, NARROW, WIDE = (2, 8, 1), (2, 4, 4), (2, 4, 12), (2, 4, 70)


def attend(c, lens, new, G, scale, weights=None):
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    out, lse = c["cache"].attend(c["q"].cuda(), dev(c["table"]), dev(lens), max(lens), cu_seqlens=dev(c["cu"]),
                                 max_new=new, scale=scale, weights=weights, status=status)
    want = ref.attend(c["q"].double().numpy(), c["rk"], c["rv"], c["table"], lens, c["cu"], scale)
    assert int(status.item()) == 0
    return out, lse, want


def certain(out, lse, want, rows, bf16):
    """Rows whose weights are 1 or 1 / n."""
    o, ls, _, mass, reach = (t[rows] if i != 2 else t for i, t in enumerate(want))
    got, l = out.double().cpu().numpy()[rows], lse.double().cpu().numpy()[rows]
    tol = (2.0 ** -8 * np.abs(o) + 2.0 ** -10 * mass if bf16 else 0) + 2.0 ** -20 * mass + 1e-30
    assert np.isfinite(got).all() and (np.abs(got - o) <= tol).all(), (np.abs(got - o) / tol).max()
    assert (np.abs(l - ls) <= 2.0 ** -16 * reach).all()


def ordinary(out, lse, want, rows, bf16, n):
    rest = tuple(t[rows] if i != 2 else t for i, t in enumerate(want))
    compare(out[torch.tensor(rows).cuda()], lse[torch.tensor(rows).cuda()], None, rest, bf16, n, 1)


def planted(H, G, new, d, bs, lens, dtype, size, seed):
    """Every third row is a multiple of one of its keys, with a score of about `size`."""
    c = make(H, G, d, bs, lens, [new] * len(lens), dtype, seed, qscale=1.0)
    q, scale = c["q"].double(), d ** -0.5
    big = np.zeros(q.shape[:2], dtype=bool)
    rng = np.random.default_rng(seed)
    for t in range(q.shape[0]):
        r, i = divmod(t, new)
        for hq in range(H * G):
            see = lens[r] - new + i + 1
            if see <= 0 or (t * H * G + hq) % 3:
                continue
            keys = c["rk"].rows(c["table"][r], range(see), hq // G)
            j = int(rng.integers(0, see))
            row = torch.tensor(keys[j] * (size / (scale * (keys[j] @ keys[j])))).to(dtype).double()
            x = np.sort(scale * (keys @ row.numpy()))
            if see > 1 and x[-2] > 0.75 * x[-1]:
                continue                 # another key lies too near
            q[t, hq] = row
            big[t, hq] = True
    c["q"] = q.to(dtype)
    assert big.any() and not big.all()
    return c, big, scale


@pytest.mark.parametrize("size", SIZES)
@pytest.mark.parametrize("H,G,new", [FEW8, FEW16, NARROW, WIDE])
def test_huge_scores_beside_ordinary_ones(H, G, new, size):
    lens = [700, 150]
    c, big, scale = planted(H, G, new, 128, 16, lens, torch.bfloat16, size, 3)
    out, lse, want = attend(c, lens, new, G, scale)
    certain(out, lse, want, big, True)
    ordinary(out, lse, want, ~big, True, 700)


def rising(H, G, new, n, dtype, size):
    """Keys along one direction, larger slot by slot (several share each of e4m3's
    magnitudes): every tile brings a new maximum.  Every other head looks along the
    direction, the rest against it (the first slots are the largest then)."""
    d, bs = 128, 16
    c = make(H, G, d, bs, [n], [new], dtype, 11, qscale=1.0)
    sign = np.where(np.arange(d) % 3 == 0, -1.0, 1.0)
    code = (1 + np.arange(n) * 125 // (n - 1)).astype(np.uint8)
    kc = c["cache"].k_codes
    for j in range(n):
        kc[int(c["table"][0][j // bs]), :, j % bs] = torch.tensor(
            np.where(sign < 0, code[j] | 0x80, code[j]).astype(np.uint8)).cuda()
    c["cache"].k_scale.fill_(1.0)
    c["cache"].v_scale.fill_(0.25)
    c["rk"] = ref.RefCache(kc.cpu().numpy(), c["cache"].k_scale.cpu().numpy())
    c["rv"] = ref.RefCache(c["cache"].v_codes.cpu().numpy(), c["cache"].v_scale.cpu().numpy())
    scale = d ** -0.5
    a = 2.0 ** np.round(np.log2(size / (scale * d * 448)))
    q = torch.tensor(np.tile(a * sign, (new, H * G, 1)))
    q[:, 1::2] *= -1
    c["q"] = q.to(dtype)
    return c, scale


@pytest.mark.parametrize("size", SIZES)
@pytest.mark.parametrize("H,G,new", [FEW8, FEW16, NARROW, WIDE])
def test_scores_that_rise_from_tile_to_tile(H, G, new, size):
    c, scale = rising(H, G, new, 900, torch.bfloat16, size)
    out, lse, want = attend(c, [900], new, G, scale)
    certain(out, lse, want, np.ones((new, H * G), dtype=bool), True)


def equal_keys(H, G, new, n, dtype, size):
    """Two far slots with one key, which every query is a multiple of."""
    d, bs = 128, 16
    c = make(H, G, d, bs, [n], [new], dtype, 13, qscale=1.0)
    c["cache"].k_scale.fill_(2.0 ** -5)
    c["cache"].v_scale.fill_(2.0 ** -5)
    kc, t = c["cache"].k_codes, c["table"][0]
    j0, j1 = 3, n - new
    kc[int(t[j1 // bs]), :, j1 % bs] = kc[int(t[j0 // bs]), :, j0 % bs]
    c["rk"] = ref.RefCache(kc.cpu().numpy(), c["cache"].k_scale.cpu().numpy())
    c["rv"] = ref.RefCache(c["cache"].v_codes.cpu().numpy(), c["cache"].v_scale.cpu().numpy())
    scale = d ** -0.5
    q = np.empty((new, H * G, d))
    for h in range(H * G):
        key = c["rk"].rows(t, [j0], h // G)[0]
        q[:, h] = key * (size / (scale * (key @ key)))
    c["q"] = torch.tensor(q).to(dtype)
    return c, scale


@pytest.mark.parametrize("size", SIZES)
@pytest.mark.parametrize("H,G,new", [FEW8, FEW16, NARROW, WIDE])
def test_equal_keys_share_the_weight(H, G, new, size):
    c, scale = equal_keys(H, G, new, 3000, torch.bfloat16, size)
    out, lse, want = attend(c, [3000], new, G, scale)
    assert abs(want[2].max() - 0.5 * G * new) < 1e-9
    certain(out, lse, want, np.ones((new, H * G), dtype=bool), True)


# the form of fp32 queries, large head dims and odd blocks: few columns to many
SPLIT = [(2, 4, 1, 128, 16, torch.float32), (2, 8, 2, 64, 16, torch.float32), (1, 4, 20, 128, 24, torch.float32),
         (2, 2, 3, 256, 16, torch.bfloat16), (2, 2, 20, 256, 32, torch.float32), (1, 4, 9, 128, 7, torch.bfloat16)]


@pytest.mark.parametrize("size", SIZES)
@pytest.mark.parametrize("H,G,new,d,bs,dtype", SPLIT)
def test_huge_scores_in_the_split_form(H, G, new, d, bs, dtype, size):
    lens = [1500, 150]
    c, big, scale = planted(H, G, new, d, bs, lens, dtype, size, 3)
    bf16 = dtype == torch.bfloat16
    out, lse, want = attend(c, lens, new, G, scale)
    certain(out, lse, want, big, bf16)
    ordinary(out, lse, want, ~big, bf16, 1500)


@pytest.mark.parametrize("H,G,new", [FEW8, FEW16, NARROW, WIDE])
def test_rows_of_infinities_and_nan_end_and_stay_alone(H, G, new):
    lens = [300]
    c = make(H, G, 128, 16, lens, [new], torch.bfloat16, 17)
    odd = np.zeros((new, H * G), dtype=bool)
    odd[::3, ::2] = True
    q = c["q"].clone()
    for k, (t, h) in enumerate(zip(*np.nonzero(odd))):
        q[t, h, k % 128] = [float("inf"), float("nan"), -float("inf")][k % 3]
    good = c["q"].clone()
    c["q"] = q
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    out, lse = c["cache"].attend(q.cuda(), dev(c["table"]), dev(lens), 300, cu_seqlens=dev(c["cu"]), max_new=new,
                                 status=status)
    want = ref.attend(good.double().numpy(), c["rk"], c["rv"], c["table"], lens, c["cu"], 128 ** -0.5)
    assert int(status.item()) == 0 and torch.isnan(out[torch.tensor(odd).cuda()]).all()
    ordinary(out, lse, want, ~odd, True, 300)


# Weights: kept scores of 8 and 16 columns, of narrow rows and of the split form; scores
# formed again by the wide form, and by every other one where the bound on the lengths is
# too large to keep them.
WEIGHED = [(*FEW8, 128, 16, torch.bfloat16), (*FEW16, 128, 16, torch.bfloat16), (*NARROW, 128, 16, torch.bfloat16),
           (*WIDE, 128, 16, torch.bfloat16), (2, 4, 3, 64, 16, torch.float32), (1, 4, 20, 128, 24, torch.float32),
           (2, 2, 20, 256, 16, torch.bfloat16)]


def check_weights(w, out, lse, want, c, lens, new, G, sure, n):
    """Each weight is the sum of its sure rows' probabilities, off by 2^-20 of themselves,
    and of its ordinary ones', off as in test_gpu_attend8.py."""
    H = w.shape[1]
    xe = np.where(sure, 0, 2.0 ** -16 * want[4]).max()
    tol = (2 * xe + n * 2.0 ** -23 + (new * G + 16) * 2.0 ** -23 + 2.0 ** -20) * want[2] + 1e-30
    got = w[..., :max(lens)].double().cpu().numpy()
    assert np.isfinite(got).all() and (np.abs(got - want[2]) <= tol).all(), (np.abs(got - want[2]) / tol).max()
    assert not w[..., max(lens):].any()


@pytest.mark.parametrize("size", [2.0 ** 13, 2.0 ** 17, 1e9, 1e30])
@pytest.mark.parametrize("bound", [0, 1 << 26])
@pytest.mark.parametrize("H,G,new,d,bs,dtype", WEIGHED)
def test_weights_of_huge_scores(H, G, new, d, bs, dtype, bound, size):
    lens = [1100, 150]
    c, big, scale = planted(H, G, new, d, bs, lens, dtype, size, 5)
    bound = bound or max(lens)
    w = torch.zeros((2, H, bound), device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    out, lse = c["cache"].attend(c["q"].cuda(), dev(c["table"]), dev(lens), bound, cu_seqlens=dev(c["cu"]),
                                 max_new=new, scale=scale, weights=w, status=status)
    assert int(status.item()) == 0
    want = ref.attend(c["q"].double().numpy(), c["rk"], c["rv"], c["table"], lens, c["cu"], scale)
    certain(out, lse, want, big, dtype == torch.bfloat16)
    check_weights(w, out, lse, want, c, lens, new, G, big, 1100)


@pytest.mark.parametrize("bound", [0, 1 << 26])
@pytest.mark.parametrize("H,G,new,d,bs,dtype", WEIGHED[:4] + [(2, 4, 3, 128, 16, torch.float32)])
def test_weights_of_equal_keys(H, G, new, d, bs, dtype, bound):
    c, scale = equal_keys(H, G, new, 1500, dtype, 1e9)
    bound = bound or 1500
    w = torch.zeros((1, H, bound), device="cuda")
    out, lse = c["cache"].attend(c["q"].cuda(), dev(c["table"]), dev([1500]), bound, cu_seqlens=dev(c["cu"]),
                                 max_new=new, scale=scale, weights=w)
    want = ref.attend(c["q"].double().numpy(), c["rk"], c["rv"], c["table"], [1500], c["cu"], scale)
    check_weights(w, out, lse, want, c, [1500], new, G, np.ones((new, H * G), dtype=bool), 1500)


@pytest.mark.parametrize("lens,new,G,d,bs,dtype", [([400, 33, 0, 257], [70, 33, 2, 1], 4, 64, 16, torch.float32),
                                                   ([90, 700], [90, 9], 2, 256, 32, torch.bfloat16),
                                                   ([300], [300], 8, 128, 24, torch.float32)])
def test_split_weights_without_kept_scores(lens, new, G, d, bs, dtype):
    c = make(2, G, d, bs, lens, new, dtype, 43)
    bound = 1 << 26
    w = torch.full((len(lens), 2, bound), 0.25, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    out, lse = c["cache"].attend(c["q"].cuda(), dev(c["table"]), dev(lens), bound, cu_seqlens=dev(c["cu"]),
                                 max_new=max(new), weights=w, status=status)
    want = ref.attend(c["q"].double().numpy(), c["rk"], c["rv"], c["table"], lens, c["cu"], d ** -0.5)
    assert int(status.item()) == 0
    n = max(lens)
    compare(out, lse, None, want, dtype == torch.bfloat16, n, max(new) * G)
    for r, L in enumerate(lens):
        assert (w[r, :, L:] == 0.25).all()
        ws = want[2][r, :, :L]
        got = w[r, :, :L].double().cpu().numpy() - 0.25
        tol = (2 * 2.0 ** -16 * want[4].max() + (n + max(new) * G + 16) * 2.0 ** -23) * (ws + 0.25)
        assert (np.abs(got - ws) <= tol).all()


def test_more_columns_than_shared_memory_holds_log_sum_exps_for():
    """Kept scores of more than 12,288 columns."""
    H, G, new, n = 1, 16, 900, 900
    c = make(H, G, 64, 16, [n], [new], torch.float32, 47)
    w = torch.zeros((1, H, n), device="cuda")
    out, lse = c["cache"].attend(c["q"].cuda(), dev(c["table"]), dev([n]), n, cu_seqlens=dev(c["cu"]), max_new=new,
                                 weights=w)
    want = ref.attend(c["q"].double().numpy(), c["rk"], c["rv"], c["table"], [n], c["cu"], 0.125)
    compare(out, lse, w, want, False, n, new * G)


@pytest.mark.parametrize("exp", [-90, 100, 126, 127])
@pytest.mark.parametrize("H,G,new,d,bs,dtype", WEIGHED)
def test_value_scales_at_the_ends_of_their_range(H, G, new, d, bs, dtype, exp):
    """Values up to 2^127 (codes up to 1 under the largest scales) and down to 2^-96."""
    lens = [300, 90]
    c = make(H, G, d, bs, lens, [new, new], dtype, 19)
    v = c["cache"].v_codes
    small = (v & 0x80) | (v & 0x7F).clamp(max=0x38)
    v.copy_(torch.where((v & 0x7F) == 0x7F, v, small))            # slots that nobody holds keep their NaN
    c["cache"].v_scale.fill_(2.0 ** exp)
    c["rv"] = ref.RefCache(v.cpu().numpy(), c["cache"].v_scale.cpu().numpy())
    out, lse, want = attend(c, lens, new, G, d ** -0.5)
    compare(out, lse, None, want, dtype == torch.bfloat16, 300, 1)
