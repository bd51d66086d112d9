"""Host-side refusals of the calls that continue one prompt in several ways, and the
Python checks in front of them (no GPU needed: nothing is enqueued)."""
import ctypes
import os
import subprocess

import pytest
import torch

from cross_model_kv_transfer_gb300 import kvx
from test_decode_abi import BAD_CACHES, P, cache_desc

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
BIG = 1 << 40


def test_structs_match_the_c_layout(tmp_path):
    fields = {"kvx_attend8_shared_args": kvx.Attend8SharedArgs, "kvx_pages_fork_args": kvx.PagesForkArgs,
              "kvx_pages_free_args": kvx.PagesFreeArgs, "kvx_pages_reserve_args": kvx.PagesReserveArgs,
              "kvx_pages_compact_args": kvx.PagesCompactArgs, "kvx_cache8_copy_args": kvx.Cache8CopyArgs,
              "kvx_beam_args": kvx.BeamArgs}
    lines = ['#include <stdio.h>', '#include <stddef.h>', '#include "kvx.h"', "int main(void){"]
    for cname, cls in fields.items():
        lines.append(f'printf("{cname} %zu\\n", sizeof({cname}));')
        for f, _ in cls._fields_:
            lines.append(f'printf("{cname}.{f} %zu\\n", offsetof({cname}, {f}));')
    lines += ['printf("flag %u\\n", KVX_FLAG_NO_PAGES);', "return 0;}"]
    src, exe = tmp_path / "probe.c", tmp_path / "probe"
    src.write_text("\n".join(lines))
    subprocess.run(["gcc", "-I", os.path.join(ROOT, "include"), str(src), "-o", str(exe)], check=True)
    got = dict(ln.split() for ln in subprocess.run([str(exe)], capture_output=True, text=True,
                                                    check=True).stdout.splitlines())
    for cname, cls in fields.items():
        assert int(got[cname]) == ctypes.sizeof(cls), cname
        for f, _ in cls._fields_:
            assert int(got[f"{cname}.{f}"]) == getattr(cls, f).offset, f"{cname}.{f}"
    assert int(got["flag"]) == kvx.KVX_FLAG_NO_PAGES


def set_all(a, over):
    for n, v in over.items():
        target = a.own if hasattr(a, "own") and hasattr(a.own, n) else a
        setattr(target, n, v)
    return a


def shared_args(cache=None, **over):
    own = kvx.Attend8Args(cache=cache_desc() if cache is None else cache, q=P, out=P, q_token_stride=256,
                          q_head_stride=64, out_token_stride=256, out_head_stride=64,
                          dtype=kvx.KVX_BF16, q_heads=4, ntok=10, num_requests=3, max_new=8,
                          cu_seqlens=P, lens=P, max_len=64, scale=0.125, workspace=P)
    a = kvx.Attend8SharedArgs(own=own, prefix_table=P, prefix_lens=P, groups=P, max_prefix_blocks=4,
                              num_prefixes=2, max_prefix=64, max_group=2)
    set_all(a, over)
    if "workspace_bytes" not in over:
        a.own.workspace_bytes = kvx.kvx_attend8_shared_workspace_bytes(a)
    return a


def test_shared_attention_refuses():
    bad = kvx.KVX_ERR_INVALID_ARG
    call = lambda **over: kvx.kvx_attend8_shared(shared_args(**over), None)
    for over in BAD_CACHES:
        assert kvx.kvx_attend8_shared(shared_args(cache_desc(**over)), None) == bad
    for over in (dict(prefix_table=None), dict(prefix_table=P + 2), dict(prefix_lens=None), dict(prefix_lens=P + 1), dict(groups=P + 2),
                 dict(groups=None), dict(max_prefix_blocks=0), dict(num_prefixes=0), dict(max_prefix=-1),
                 dict(max_group=0), dict(weights=P, weights_stride=64), dict(q=None), dict(out=P + 1),
                 dict(workspace=None), dict(workspace=P + 128), dict(q_heads=3), dict(max_new=0),
                 dict(ntok=-1), dict(lens=None), dict(scale=float("nan")), dict(dtype=2), dict(cu_seqlens=None)):
        assert call(**over) == bad, over
    need = kvx.kvx_attend8_shared_workspace_bytes(shared_args())
    assert need > 0 and call(workspace_bytes=need - 1) == bad
    assert call(max_prefix=2 ** 31 - 1) != kvx.KVX_OK
    # a group's rows are counted in 32 bits
    assert call(ntok=2 ** 30, num_requests=2 ** 20, max_group=2 ** 20, max_new=2 ** 10) == kvx.KVX_ERR_UNSUPPORTED
    assert call(ntok=0) == kvx.KVX_OK
    assert call(ntok=0, groups=None, num_prefixes=1) == kvx.KVX_OK
    assert kvx.load().kvx_attend8_shared(None, None) == bad
    assert kvx.load().kvx_attend8_shared_workspace_bytes(None) == 0


def test_shared_workspaces_never_fall():
    need = lambda **over: kvx.kvx_attend8_shared_workspace_bytes(shared_args(**over))
    for dtype in (kvx.KVX_F32, kvx.KVX_BF16):
        for name, values in (("ntok", (1, 10, 100, 5000)), ("max_group", (1, 2, 3, 9)), ("max_new", (1, 2, 9, 70, 700)),
                             ("max_prefix", (0, 64, 5000)), ("q_heads", (2, 4, 16, 64)), ("max_len", (0, 5, 900))):
            sizes = [need(dtype=dtype, **{name: v}) for v in values]
            assert sizes == sorted(sizes) and sizes[0] > 0, (name, sizes)


def pages_args(cls, **over):
    common = dict(refs=P, num_blocks=8, block_size=16, num_rows=2, width=4, table=P, lens=P)
    more = {kvx.PagesForkArgs: dict(parents=P, num_new=2, new_table=P + 4096, new_lens=P + 4096),
            kvx.PagesFreeArgs: {}, kvx.PagesReserveArgs: dict(add_all=1, copies=P, workspace=P),
            kvx.PagesCompactArgs: dict(used=P, moved=P, workspace=P)}[cls]
    names = {n for n, _ in cls._fields_}
    a = cls(**{k: v for k, v in {**common, **more}.items() if k in names})
    for n, v in over.items():
        setattr(a, n, v)
    if "workspace_bytes" in names and "workspace_bytes" not in over:
        a.workspace_bytes = kvx.kvx_pages_workspace_bytes(a.num_blocks)
    return a


def test_pages_refuse():
    bad, no = kvx.KVX_ERR_INVALID_ARG, kvx.KVX_ERR_UNSUPPORTED
    pool = [dict(refs=None), dict(refs=P + 2), dict(num_blocks=0), dict(num_blocks=2 ** 31 - 1024)]
    shape = [dict(num_rows=-1), dict(width=0), dict(table=None)]
    for cls, call, more in (
            (kvx.PagesForkArgs, kvx.kvx_pages_fork,
             shape + [dict(block_size=0), dict(block_size=1025), dict(lens=None), dict(parents=None), dict(num_new=-1),
                      dict(new_table=None), dict(new_lens=None), dict(new_table=P), dict(new_lens=P), dict(table=P + 2),
                      dict(lens=P + 1), dict(parents=P + 3), dict(new_table=P + 2), dict(new_lens=P + 2),
                      dict(width=2 ** 27)]),
            (kvx.PagesFreeArgs, kvx.kvx_pages_free, shape),
            (kvx.PagesReserveArgs, kvx.kvx_pages_reserve,
             shape + [dict(block_size=0), dict(lens=None), dict(add_all=-1), dict(add=P + 2), dict(copies=P + 2),
                      dict(table=P + 1), dict(workspace=None),
                      dict(workspace=P + 4), dict(workspace_bytes=100), dict(num_caches=-1), dict(num_caches=1),
                      dict(width=2 ** 27)]),
            (kvx.PagesCompactArgs, kvx.kvx_pages_compact,
             [dict(block_size=0), dict(used=None), dict(moved=None), dict(used=P + 2), dict(moved=P + 1), dict(num_tables=-1), dict(num_tables=9),
              dict(num_tables=1), dict(workspace=None), dict(workspace_bytes=0), dict(num_caches=2)])):
        for over in pool + more:
            assert call(pages_args(cls, **over), None) == bad, (cls, over)
        assert getattr(kvx.load(), call.__name__)(None, None) == bad
    assert kvx.kvx_pages_reserve(pages_args(kvx.PagesReserveArgs, num_rows=2 ** 20, width=2 ** 12), None) == no
    # nothing to do
    assert kvx.kvx_pages_fork(pages_args(kvx.PagesForkArgs, num_rows=0, num_new=0), None) == kvx.KVX_OK
    assert kvx.kvx_pages_free(pages_args(kvx.PagesFreeArgs, num_rows=0), None) == kvx.KVX_OK
    assert kvx.kvx_pages_reserve(pages_args(kvx.PagesReserveArgs, num_rows=0), None) == kvx.KVX_OK
    for n in (0, -1, 2 ** 31 - 1024):
        assert kvx.kvx_pages_workspace_bytes(n) == 0


def test_caches_of_pages_are_checked():
    bad = kvx.KVX_ERR_INVALID_ARG

    def with_caches(cls, call, *descs):
        array = (kvx.Cache8Desc * len(descs))(*descs)
        a = pages_args(cls) if cls is not kvx.Cache8CopyArgs else kvx.Cache8CopyArgs(pairs=P, num_pairs=3)
        a.caches, a.num_caches = ctypes.addressof(array), len(descs)
        return call(a, None)
    good = cache_desc()
    for cls, call in ((kvx.PagesReserveArgs, kvx.kvx_pages_reserve), (kvx.PagesCompactArgs, kvx.kvx_pages_compact),
                      (kvx.Cache8CopyArgs, kvx.kvx_cache8_copy)):
        for over in BAD_CACHES:
            if not {"max_blocks_per_req", "block_table"} & set(over):
                assert with_caches(cls, call, good, cache_desc(**over)) != kvx.KVX_OK, (cls, over)
        assert with_caches(cls, call, good, cache_desc(num_blocks=9)) == bad
        if cls is not kvx.Cache8CopyArgs:
            assert with_caches(cls, call, good, cache_desc(block_size=8)) == bad
    copy = lambda **kw: kvx.kvx_cache8_copy(kvx.Cache8CopyArgs(**kw), None)
    assert copy(num_caches=1, num_pairs=0) == bad and copy(num_caches=-1) == bad
    assert copy(num_pairs=-1) == bad and copy(num_pairs=1) == bad and copy() == kvx.KVX_OK


def beam_args(**over):
    a = kvx.BeamArgs(logits=P, row_stride=100, dtype=kvx.KVX_F32, num_requests=2, beams=3, out_beams=4, vocab=100,
                     eos=-1, scores=P, tokens=P, parents=P, new_scores=P + 4096, workspace=P)
    for n, v in over.items():
        setattr(a, n, v)
    if "workspace_bytes" not in over:
        a.workspace_bytes = kvx.kvx_beam_workspace_bytes(a)
    return a


def test_beam_selection_refuses():
    for over in (dict(logits=None), dict(logits=P + 2), dict(dtype=2), dict(num_requests=-1), dict(beams=0),
                 dict(beams=33), dict(out_beams=0), dict(out_beams=33), dict(vocab=0), dict(eos=-2), dict(eos=100),
                 dict(scores=None), dict(scores=P + 2), dict(tokens=P + 1), dict(tokens=None), dict(parents=None), dict(new_scores=None),
                 dict(new_scores=P), dict(done=P), dict(done=P, new_done=P, eos=1), dict(workspace=None),
                 dict(workspace=P + 8), dict(workspace_bytes=10), dict(vocab=2 ** 31 - 1), dict(num_requests=2 ** 30)):
        assert kvx.kvx_beam_select(beam_args(**over), None) == kvx.KVX_ERR_INVALID_ARG, over
    assert kvx.kvx_beam_select(beam_args(num_requests=0), None) == kvx.KVX_OK
    assert kvx.load().kvx_beam_select(None, None) == kvx.KVX_ERR_INVALID_ARG
    assert kvx.load().kvx_beam_workspace_bytes(None) == 0


def test_python_refuses_tensors_on_the_cpu_and_bad_shapes():
    i32 = lambda *s: torch.zeros(s, dtype=torch.int32)
    pages = kvx.Pages(i32(8), 16)
    for call in (lambda: pages.fork(i32(2, 3), i32(2), i32(2)), lambda: pages.free(i32(2, 3)),
                 lambda: pages.reserve(i32(2, 3), i32(2)), lambda: pages.compact([i32(2, 3)]),
                 lambda: kvx.beam_select(torch.zeros(4, 9), torch.zeros(2, 2)),
                 lambda: kvx.Pages(torch.zeros(8), 16), lambda: kvx.Pages(i32(2, 4), 16),
                 lambda: kvx.Pages(i32(16)[::2], 16)):
        with pytest.raises(ValueError):
            call()
    cache = kvx.Cache8.empty(4, 1, 16, 16, device="cpu")
    with pytest.raises(ValueError):
        cache.attend_shared(torch.zeros(1, 1, 16), i32(1, 1), i32(1), i32(1, 1), i32(1), max_prefix=1, max_len=1)
    with pytest.raises(ValueError):
        kvx.copy_pages([cache], i32(1, 2))
    with pytest.raises(kvx.KvxError):
        kvx.beam_workspace(requests=1, beams=33, vocab=10, device="cpu")
    with pytest.raises(kvx.KvxError):
        cache.attend_shared_workspace(ntok=1, num_requests=1, q_heads=1, max_prefix=-1, max_len=1)
