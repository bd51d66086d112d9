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


@pytest.mark.parametrize("rows,new", [(3, 4), (1500, 4), (3, 400)])
def test_entries_outside_the_pool_where_pages_are_short(rows, new):
    """They become -1, as they count; all else stays, whether a warp takes its rows in one turn
    or in several."""
    bs, width = 4, 120
    table = np.full((rows, width), -1)
    table[:, 0] = 0                                  # all rows share a page
    table[0, 1], table[1, 0], table[2, 1] = 99, -7, -2147483648
    refs = [rows - 1, 1, 0, 0]
    pages, t, status = kvx.Pages(dev(refs), bs), dev(table), torch.zeros(1, dtype=torch.int32, device="cuda")
    copies = torch.full((rows, 2), 7, dtype=torch.int32, device="cuda")
    pages.reserve(t, dev([2] * rows), new, copies=copies, status=status)
    assert int(status.item()) == kvx.KVX_FLAG_NO_PAGES | kvx.KVX_FLAG_BAD_BLOCK
    table[0, 1] = table[1, 0] = table[2, 1] = -1
    assert t.tolist() == table.tolist() and pages.refs.tolist() == refs and (copies == -1).all()
    # beside the new slots they stay
    t = dev([[50, -1, 60]])
    status.zero_()
    pages.reserve(t, dev([4]), 4, status=status)
    assert t.tolist() == [[50, 2, 60]] and int(status.item()) == 0
