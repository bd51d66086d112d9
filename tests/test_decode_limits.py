"""Bounds of the decoding calls that the host alone can check: loose bounds on a
request's queries, sizes of workspaces (no GPU needed: nothing is enqueued)."""
import pytest

from cross_model_kv_transfer_gb300 import kvx
from test_decode_abi import P, attend_args, cache_desc


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
