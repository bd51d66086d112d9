"""The 8-bit paged cache's write (kvx_cache8_write) against fp64: scales and
codes are exact (a power-of-two scale makes x / scale exact, and the nearest
code with ties to even is then unique), so everything is compared for equality."""
import numpy as np
import pytest
import torch

import decode_reference as ref
from cross_model_kv_transfer_gb300 import kvx

pytestmark = pytest.mark.gpu


def gpu_cache(kc, ks, vc, vs):
    return kvx.Cache8(*(torch.tensor(t).cuda() for t in (kc, vc, ks, vs)))


def same(cache, rk, rv):
    for codes, scale, r in ((cache.k_codes, cache.k_scale, rk), (cache.v_codes, cache.v_scale, rv)):
        assert np.array_equal(scale.double().cpu().numpy(), r.scale)
        assert np.array_equal(ref.E4M3[codes.cpu().numpy()], r.values)


def setup(H, d, bs, num_blocks, seed, scales="pow2"):
    kc, ks = ref.random_cache(num_blocks, H, bs, d, seed, scales)
    vc, vs = ref.random_cache(num_blocks, H, bs, d, seed + 1, scales)
    return gpu_cache(kc, ks, vc, vs), ref.RefCache(kc, ks), ref.RefCache(vc, vs)


def fresh(n, H, d, dtype, seed):
    rng = np.random.default_rng(seed)
    x = rng.standard_normal((n, H, d)) * np.exp(2.0 * rng.standard_normal((n, 1, 1)))
    return torch.tensor(x).to(dtype)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("H,d,bs,lens,starts", [
    (2, 128, 16, [1, 1, 1], [0, 15, 16]), (8, 128, 16, [40, 0, 3, 17], [0, 5, 14, 31]),
    (1, 64, 24, [100, 7], [23, 0]), (3, 96, 1, [5, 2], [0, 3]), (2, 256, 7, [20, 9], [6, 7]),
    (1, 16, 64, [63, 65], [1, 63]), (5, 80, 128, [1, 200], [127, 100]),
    (2, 128, 300, [700], [299])])
def test_write_matches_fp64(H, d, bs, lens, starts, dtype):
    total = [a + n for a, n in zip(starts, lens)]
    nb = sum(-(-t // bs) for t in total) + 3
    cache, rk, rv = setup(H, d, bs, nb, 11)
    table = ref.block_table(total, bs, nb, 5)
    cu = np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)
    k, v = fresh(cu[-1], H, d, dtype, 1), fresh(cu[-1], H, d, dtype, 2)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    cache.write(k.cuda(), v.cuda(), torch.tensor(table).cuda(),
                torch.tensor(starts, dtype=torch.int32).cuda(),
                cu_seqlens=torch.tensor(cu).cuda(), status=status)
    rk.write(k.double().numpy(), table, starts, cu)
    rv.write(v.double().numpy(), table, starts, cu)
    same(cache, rk, rv)
    assert int(status.item()) == 0


@pytest.mark.parametrize("scales", ["pow2", "any"])
def test_token_by_token_equals_its_reference(scales):
    """Appends one token at a time, of growing and shrinking size, past block
    ends; older codes are re-scaled when the scale grows."""
    H, d, bs, R = 2, 64, 8, 3
    cache, rk, rv = setup(H, d, bs, 12, 3, scales)
    table = ref.block_table([30] * R, bs, 12, 1)
    rng = np.random.default_rng(0)
    at = [0, 7, 3]
    for step in range(18):
        x = torch.tensor(rng.standard_normal((2, R, H, d)) * 4.0 ** rng.integers(-3, 4, (2, R, 1, 1)))
        x = x.float()
        cache.write(x[0].cuda(), x[1].cuda(), torch.tensor(table).cuda(),
                    torch.tensor(at, dtype=torch.int32).cuda())
        rk.write(x[0].double().numpy(), table, at, list(range(R + 1)))
        rv.write(x[1].double().numpy(), table, at, list(range(R + 1)))
        if scales == "pow2":
            same(cache, rk, rv)
        at = [a + 1 for a in at]
    if scales == "any":   # old / new is rounded to fp32: a tie may fall the other way
        got = ref.E4M3[cache.k_codes.cpu().numpy()]
        assert np.mean(got != rk.values) < 1e-3
        assert np.allclose(cache.k_scale.double().cpu().numpy(), rk.scale, rtol=1e-7)


def test_extreme_values_infinities_and_nan():
    H, d, bs = 1, 16, 4
    cache, rk, rv = setup(H, d, bs, 6, 9)
    table = np.array([[0, 1, 2, 3, 4]], dtype=np.int32)
    x = torch.zeros((20, H, d))
    x[0:4] = 0.0                                     # a block of zeros
    x[4, 0, :4] = torch.tensor([1e-45, -1e-40, 2e-38, 1e-38])   # below the smallest scale
    x[8, 0, :3] = torch.tensor([3.4028235e38, -1.7e38, 1.0])
    x[12, 0, :3] = torch.tensor([448.0, 448.00003, -447.0])     # either side of 1.75 * 2^8
    x[16, 0, :5] = torch.tensor([float("inf"), float("-inf"), float("nan"), 2.0, -3.0])
    v = x.clone()
    v[16] = 1.0
    v[12, 0, 1] = 447.9
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    cache.write(x.cuda(), v.cuda(), torch.tensor(table).cuda(),
                cu_seqlens=torch.tensor([0, 20], dtype=torch.int32).cuda(), status=status)
    rk.write(x.double().numpy(), table, [0], [0, 20])
    rv.write(v.double().numpy(), table, [0], [0, 20])
    same(cache, rk, rv)
    assert int(status.item()) == kvx.KVX_FLAG_NOT_FINITE
    assert rk.scale[0, 0] == 2.0 ** -126 and rk.scale[3, 0] == 2.0 and rv.scale[3, 0] == 1.0


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_strided_rows_and_a_paged_source(dtype):
    """k and v as views of one projection, and the rows of a paged cache read
    through src_rows (a row outside it is stored as zeros and flagged)."""
    H, d, bs, n = 2, 64, 16, 45
    cache, rk, rv = setup(H, d, bs, 8, 21)
    table = ref.block_table([n], bs, 8, 2)
    cu = torch.tensor([0, n], dtype=torch.int32).cuda()
    fused = torch.tensor(np.random.default_rng(1).standard_normal((60, 3 * H, d + 8))).to(dtype)
    k, v = fused[:, H:2 * H, 3:3 + d], fused[:, 2 * H:, :d]
    rows = np.random.default_rng(2).permutation(60)[:n].astype(np.int32)
    dev = fused.cuda()
    cache.write(dev[:, H:2 * H, 3:3 + d], dev[:, 2 * H:, :d], torch.tensor(table).cuda(),
                cu_seqlens=cu, src_rows=torch.tensor(rows).cuda())
    rk.write(k.double().numpy(), table, [0], [0, n], rows)
    rv.write(v.double().numpy(), table, [0], [0, n], rows)
    same(cache, rk, rv)
    bad = rows.copy()
    bad[3], bad[40] = -1, 60
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    cache.write(dev[:, H:2 * H, :d], dev[:, 2 * H:, :d], torch.tensor(table).cuda(), cu_seqlens=cu,
                src_rows=torch.tensor(bad).cuda(), status=status)
    assert int(status.item()) == kvx.KVX_FLAG_BAD_SRC_BLOCK
    for j in (3, 40):
        assert not cache.k_codes[table[0][j // bs], :, j % bs].any()


def test_flags_skip_only_what_they_name():
    H, d, bs = 1, 16, 4
    cache, rk, rv = setup(H, d, bs, 6, 4)
    dev = lambda t: torch.tensor(t, dtype=torch.int32).cuda()
    x = fresh(12, H, d, torch.float32, 7)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    before = cache.k_codes.clone()
    for cu in ([0, 5, 4, 12], [1, 4, 8, 12], [0, 4, 8, 11]):
        status.zero_()
        cache.write(x.cuda(), x.cuda(), dev([[0, 1], [2, 3], [4, 5]]), cu_seqlens=dev(cu),
                    status=status)
        assert int(status.item()) == kvx.KVX_FLAG_BAD_SEQLENS
        assert torch.equal(cache.k_codes, before)
    status.zero_()     # a block id outside the pool, and tokens past the table
    cache.write(x.cuda(), x.cuda(), dev([[0, 6], [-1, 3], [4, 5]]), dev([0, 0, 6]),
                cu_seqlens=dev([0, 4, 8, 12]), status=status)
    table = [[0, 0], [0, 0], [4, 5]]
    rk.write(x.double().numpy(), table, [0], [0, 4])
    rk.write(x.double().numpy()[8:], [[4, 5]], [6], [0, 2])
    assert np.array_equal(ref.E4M3[cache.k_codes.cpu().numpy()], rk.values)
    assert int(status.item()) == kvx.KVX_FLAG_BAD_BLOCK | kvx.KVX_FLAG_BAD_LENGTH
    status.zero_()
    before = cache.k_codes.clone()
    cache.write(x[:1].cuda(), x[:1].cuda(), dev([[0, 1]]), dev([-1]), status=status)
    assert int(status.item()) == kvx.KVX_FLAG_BAD_LENGTH and torch.equal(cache.k_codes, before)


def test_blocks_past_32_bit_offsets_and_another_stream():
    H, d, bs = 2, 128, 64
    nb = 2 ** 32 // (H * bs * d) + 8
    cache = kvx.Cache8.empty(nb, H, d, bs)
    table = torch.tensor([[nb - 1, 3]], dtype=torch.int32, device="cuda")
    x = fresh(70, H, d, torch.bfloat16, 1).cuda()
    s = torch.cuda.Stream()
    y = 2 * x
    cu = torch.tensor([0, 70], dtype=torch.int32, device="cuda")
    s.wait_stream(torch.cuda.current_stream())
    cache.write(x, y, table, cu_seqlens=cu, stream=s)
    s.synchronize()
    z = np.zeros((2, H, bs, d), dtype=np.uint8)
    rk, rv = (ref.RefCache(z, np.ones((2, H))) for _ in range(2))
    rk.write(x.double().cpu().numpy(), [[1, 0]], [0], [0, 70])
    rv.write(y.double().cpu().numpy(), [[1, 0]], [0], [0, 70])
    for codes, r in ((cache.k_codes, rk), (cache.v_codes, rv)):
        got = codes[torch.tensor([3, nb - 1], device="cuda")].cpu().numpy()
        assert np.array_equal(ref.E4M3[got], r.values)
