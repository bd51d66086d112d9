"""Bounds of the decoding calls that the host alone can check: loose bounds on a
request's queries, sizes of workspaces (no GPU needed: nothing is enqueued)."""
import pytest

from cross_model_kv_transfer_gb300 import kvx
from test_decode_abi import P, attend_args, cache_desc, evict_args


@pytest.mark.parametrize("dtype", [kvx.KVX_BF16, kvx.KVX_F32])
@pytest.mark.parametrize("q_heads,max_new", [(4, 2 ** 31 - 1), (16, 2 ** 29), (2, 2 ** 31 - 1)])
def test_a_bound_on_queries_beyond_all_queries_counts_as_all(dtype, q_heads, max_new):
    tight = attend_args(q_heads=q_heads, max_new=10, dtype=dtype)
    loose = attend_args(q_heads=q_heads, max_new=max_new, dtype=dtype)
    assert tight.workspace_bytes == loose.workspace_bytes > 0


def test_rows_that_32_bits_cannot_count_are_refused():
    wide = cache_desc(heads=1)
    for dtype in (kvx.KVX_BF16, kvx.KVX_F32):
        a = attend_args(wide, q_heads=32768, ntok=2 ** 16, max_new=2 ** 16, dtype=dtype)
        assert a.workspace_bytes == 0 and kvx.kvx_attend8(a, None) == kvx.KVX_ERR_UNSUPPORTED


BOUNDS = {"num_requests": [1, 2, 7, 16, 64, 1000, 65535], "ntok": [1, 2, 64, 500, 5000, 2 ** 20],
          "max_new": [1, 2, 4, 8, 9, 16, 17, 33, 64, 65, 128, 1000, 5000, 2 ** 31 - 1],
          "max_len": [0, 1, 255, 4096, 16384, 131071, 2 ** 24, 2 ** 27, 2 ** 31 - 1025],
          "q_heads": [8, 16, 40, 64, 512, 1024]}


@pytest.mark.parametrize("weights", [None, P])
@pytest.mark.parametrize("d,bs,dtype", [(128, 16, kvx.KVX_BF16), (64, 16, kvx.KVX_BF16), (64, 16, kvx.KVX_F32),
                                        (128, 24, kvx.KVX_F32), (256, 16, kvx.KVX_BF16), (128, 7, kvx.KVX_BF16)])
def test_workspaces_never_fall_as_a_bound_rises(d, bs, dtype, weights):
    cache = cache_desc(heads=8, head_dim=d, block_size=bs)
    at = dict(num_requests=16, ntok=2000, max_new=8, max_len=16384, q_heads=64)

    def size(**sizes):
        return attend_args(cache, weights=weights, weights_stride=2 ** 31, dtype=dtype, **sizes).workspace_bytes

    for base in (at, dict(at, max_new=1), dict(at, max_new=100), dict(at, max_len=2 ** 20, num_requests=200)):
        for name, values in BOUNDS.items():
            got = [size(**dict(base, **{name: v})) for v in values]
            assert all(x > 0 for x in got) and got == sorted(got), (name, got)


def test_a_workspace_of_larger_calls_is_large_enough_for_every_smaller_one():
    """The window of a prompt, then decoding: the sizes at which a wide call keeps no
    scores and a narrow one does."""
    cache = cache_desc(heads=8, head_dim=128)
    sizes = dict(num_requests=16, max_len=16384, q_heads=64, weights=P, weights_stride=16384)
    window = attend_args(cache, ntok=16 * 64, max_new=64, **sizes).workspace_bytes
    for new in (1, 2, 8, 16):
        assert attend_args(cache, ntok=16 * new, max_new=new, **sizes).workspace_bytes <= window


def test_evictions_in_place_are_refused():
    """Other CTAs still read the lengths and weights when the results are written."""
    Q = P + (1 << 20)
    ok = dict(lens=P, new_lens=P + 8, weights=Q, kept_weights=Q + 4 * (3 * 64 + 64), weights_stride=64, max_len=64)
    for over in (dict(new_lens=P), dict(new_lens=P + 4), dict(new_lens=P - 4), dict(kept_weights=Q),
                 dict(kept_weights=Q + 4 * 64), dict(kept_weights=Q + 4 * (3 * 64 + 63)),
                 dict(kept_weights=Q - 4 * (4 * 32 - 1))):
        a = evict_args(**dict(ok, **over))
        assert a.workspace_bytes > 0 and kvx.kvx_evict8(a, None) == kvx.KVX_ERR_INVALID_ARG, over


def test_attention_in_place_is_refused_with_weights():
    """Weights may need the queries again when the outputs are written already."""
    sizes = dict(q=P, out=P, weights=P, weights_stride=64)
    for dtype in (kvx.KVX_BF16, kvx.KVX_F32):
        assert kvx.kvx_attend8(attend_args(dtype=dtype, **sizes), None) == kvx.KVX_ERR_INVALID_ARG
