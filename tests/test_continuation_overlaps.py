"""Buffers that a call reads and writes do not overlap: tables of one compaction, a fork's old
and new rows, a selection's old and new scores are refused (no GPU needed: nothing is enqueued)."""
import ctypes

import pytest

from cross_model_kv_transfer_gb300 import kvx
from test_continuation_abi import beam_args, pages_args
from test_decode_abi import P


@pytest.mark.parametrize("tables", [
    [(P, 8), (P, 8)],                          # one table twice
    [(P, 8), (P + 16, 2)],                     # a table and rows of it
    [(P + 28, 1), (P, 8)],
    [(P, 2), (P + 4096, 8), (P + 4, 1)],
    [(P, 4), (P + 12, 4)],
    [(P, 2 ** 62)],                            # entries that no memory holds
    [(P + 4096, 8), (P, 2 ** 61 + 1)],
])
def test_tables_of_a_compaction_do_not_overlap(tables):
    n = len(tables)
    at = (ctypes.c_void_p * n)(*[t for t, _ in tables])
    entries = (ctypes.c_int64 * n)(*[e for _, e in tables])
    a = pages_args(kvx.PagesCompactArgs, used=P + 65536, moved=P + 69632, tables=ctypes.addressof(at),
                   entries=ctypes.addressof(entries), num_tables=n)
    assert kvx.kvx_pages_compact(a, None) == kvx.KVX_ERR_INVALID_ARG


@pytest.mark.parametrize("over", [
    # 2 old rows of 4 at P, their lengths 4096 bytes behind; 2 new rows 8192 bytes behind them
    dict(new_table=P + 16), dict(new_table=P + 28), dict(new_table=P - 28), dict(num_new=3, new_table=P - 36),
    dict(new_lens=P + 4096 + 4), dict(new_lens=P + 4096 - 4), dict(parents=P + 8192), dict(parents=P + 8192 + 28),
    dict(parents=P + 12288), dict(parents=P + 12288 + 4), dict(parents=P + 12288 - 4)])
def test_new_rows_overlap_nothing_that_a_fork_reads(over):
    a = pages_args(kvx.PagesForkArgs, **{**dict(lens=P + 4096, parents=P + 16384, new_table=P + 8192,
                                                new_lens=P + 12288), **over})
    assert kvx.kvx_pages_fork(a, None) == kvx.KVX_ERR_INVALID_ARG


@pytest.mark.parametrize("over", [
    # scores and done of 2 x 3, new ones of 2 x 4
    dict(new_scores=P + 20), dict(new_scores=P - 28), dict(new_done=P + 65536 + 5), dict(new_done=P + 65536 - 7)])
def test_new_scores_overlap_no_old_ones(over):
    a = beam_args(**{**dict(eos=1, done=P + 65536, new_done=P + 69632), **over})
    assert kvx.kvx_beam_select(a, None) == kvx.KVX_ERR_INVALID_ARG
