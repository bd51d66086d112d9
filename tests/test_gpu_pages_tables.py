"""Pages in narrow places: several tables of a compaction, entries outside the pool where
pages are short."""
import numpy as np
import pytest
import torch

from cross_model_kv_transfer_gb300 import kvx

pytestmark = pytest.mark.gpu


def dev(t):
    return torch.tensor(np.asarray(t, dtype=np.int32), device="cuda")


def test_overlapping_tables_are_refused_and_rows_apart_are_not():
    refs = [0, 0, 0, 1, 1, 2]
    pages = kvx.Pages(dev(refs), 4)
    table = dev([[3, -1], [4, 5], [5, -1]])
    for tables in ([table, table], [table, table[1:]], [table[:2], table[1:]], [table[2:], table]):
        with pytest.raises(kvx.KvxError) as e:
            pages.compact(tables)
        assert e.value.status == kvx.KVX_ERR_INVALID_ARG
    assert table.tolist() == [[3, -1], [4, 5], [5, -1]] and pages.refs.tolist() == refs
    # rows of one tensor, and a table without entries anywhere
    used, moved = pages.compact([table[:1], table[:0], table[1:], table[3:]])
    assert table.tolist() == [[0, -1], [1, 2], [2, -1]] and pages.refs.tolist() == [1, 1, 2, 0, 0, 0]
    assert int(used.item()) == 3 and moved.tolist() == [-1, -1, -1, 0, 1, 2]
