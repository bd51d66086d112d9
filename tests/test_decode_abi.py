"""Host-side refusals of the decoding calls, and the Python checks in front of
them (no GPU needed: nothing is enqueued)."""
import ctypes

import numpy as np
import pytest

import decode_reference as ref
from cross_model_kv_transfer_gb300 import kvx

P = 1 << 20   # an aligned address that no refused call reads


def rope_desc(**over):
    d = dict(head_dim=128, rot_dim=128, layout=0, scaling=0, theta=1e4, factor=1.0, low_band=1.0,
             high_band=4.0, beta_fast=32.0, beta_slow=1.0, amplitude=0.0, original_context=8192)
    d.update(over)
    return kvx.RopeDesc(**d)


@pytest.mark.parametrize("over", [
    dict(head_dim=127), dict(head_dim=258, rot_dim=2), dict(rot_dim=0), dict(rot_dim=130),
    dict(rot_dim=3), dict(layout=2), dict(scaling=4), dict(scaling=-1), dict(theta=1.0),
    dict(theta=float("inf")), dict(amplitude=float("nan")), dict(scaling=1, factor=0.5),
    dict(scaling=1, factor=float("nan")), dict(scaling=2, factor=2.0, original_context=0),
    dict(scaling=2, factor=2.0, low_band=4.0), dict(scaling=3, factor=2.0, beta_slow=0.0),
    dict(scaling=3, factor=2.0, beta_fast=1.0)])
def test_rope_init_refuses(over):
    assert kvx.kvx_rope_init(rope_desc(**over))[0] == kvx.KVX_ERR_INVALID_ARG


@pytest.mark.parametrize("kw", [
    dict(), dict(scaling="linear", factor=4.0), dict(scaling="yarn", factor=8.0,
                                                     original_context=4096),
    dict(scaling="bands", factor=8.0, low_band=1.0, high_band=4.0, original_context=8192)])
@pytest.mark.parametrize("d,rot,theta", [(128, 128, 5e5), (64, 16, 1e4), (256, 256, 1e6), (6, 2, 1e4)])
def test_rope_init_frequencies(d, rot, theta, kw):
    r = kvx.Rope(d, theta, rot_dim=rot, **kw)
    w, amp = ref.frequencies(rot, theta, **kw)
    turns = np.array(list(r.state.turns), dtype=np.float64) / 2.0 ** 64
    # fp64 pow and product: a few ulps of the frequency
    assert np.allclose(turns[:rot // 2], (w / (2 * np.pi)) % 1.0, rtol=1e-12, atol=1e-18)
    assert (turns[rot // 2:] == 0).all()
    assert abs(r.state.amplitude - amp) <= 2.0 ** -23 * amp
    assert kvx.Rope(d, theta, rot_dim=rot, amplitude=0.5, **kw).state.amplitude == 0.5


def test_rope_apply_refuses():
    st, rope = kvx.kvx_rope_init(rope_desc())
    assert st == kvx.KVX_OK

    def call(**over):
        a = kvx.RopeArgs(q=P, k=P, q_out=P, k_out=P, q_token_stride=1024, q_head_stride=128,
                         k_token_stride=1024, k_head_stride=128, q_out_token_stride=1024,
                         q_out_head_stride=128, k_out_token_stride=1024, k_out_head_stride=128,
                         ntok=4, q_heads=8, k_heads=8, dtype=kvx.KVX_BF16)
        for n, v in over.items():
            setattr(a, n, v)
        return kvx.kvx_rope_apply(rope, a, None)

    assert call(ntok=0) == kvx.KVX_OK
    for over in (dict(ntok=-1), dict(q_heads=0), dict(k_heads=65536), dict(q_out=None), dict(dtype=2),
                 dict(transpose=2), dict(first_position=-1), dict(q=None, k=None), dict(q=P + 1),
                 dict(k_out=P + 1)):
        assert call(**over) == kvx.KVX_ERR_INVALID_ARG, over
    assert kvx.load().kvx_rope_apply(None, None, None) == kvx.KVX_ERR_INVALID_ARG


def cache_desc(**over):
    c = dict(k_codes=P, v_codes=P, k_scale=P, v_scale=P, num_blocks=8, heads=2, head_dim=64,
             block_size=16, max_blocks_per_req=4, block_table=P)
    c.update(over)
    return kvx.Cache8Desc(**c)


BAD_CACHES = [dict(k_codes=None), dict(v_codes=P + 8), dict(k_scale=None), dict(v_scale=P + 2),
              dict(num_blocks=0), dict(num_blocks=2 ** 31), dict(heads=0), dict(head_dim=0),
              dict(head_dim=24), dict(head_dim=272), dict(block_size=0), dict(block_size=1025),
              dict(max_blocks_per_req=0), dict(block_table=None)]


def write_args(cache=None, **over):
    a = kvx.Cache8WriteArgs(cache=cache_desc() if cache is None else cache, k=P, v=P,
                            k_token_stride=128, k_head_stride=64, v_token_stride=128,
                            v_head_stride=64, dtype=kvx.KVX_BF16, num_requests=2, ntok=10,
                            cu_seqlens=P)
    for n, v in over.items():
        setattr(a, n, v)
    return a


def attend_args(cache=None, **over):
    a = kvx.Attend8Args(cache=cache_desc() if cache is None else cache, q=P, out=P,
                        q_token_stride=256, q_head_stride=64, out_token_stride=256,
                        out_head_stride=64, dtype=kvx.KVX_BF16, q_heads=4, ntok=10, num_requests=2,
                        max_new=8, cu_seqlens=P, lens=P, max_len=64, scale=0.125, workspace=P)
    for n, v in over.items():
        setattr(a, n, v)
    if "workspace_bytes" not in over:
        a.workspace_bytes = kvx.kvx_attend8_workspace_bytes(a)
    return a


def evict_args(cache=None, **over):
    a = kvx.Evict8Args(cache=cache_desc() if cache is None else cache, dst_table=P, max_dst_blocks=2,
                       num_requests=2, lens=P, max_len=64, keep=32, sinks=4, recent=8, weights=P,
                       weights_stride=64, kept=P, kept_weights=P, new_lens=P, workspace=P)
    for n, v in over.items():
        setattr(a, n, v)
    if "workspace_bytes" not in over:
        a.workspace_bytes = kvx.kvx_evict8_workspace_bytes(a)
    return a


@pytest.mark.parametrize("over", BAD_CACHES)
def test_bad_caches_are_refused_by_every_call(over):
    c = cache_desc(**over)
    assert kvx.kvx_cache8_write(write_args(c), None) == kvx.KVX_ERR_INVALID_ARG
    assert kvx.kvx_attend8(attend_args(c), None) == kvx.KVX_ERR_INVALID_ARG
    assert kvx.kvx_evict8(evict_args(c), None) == kvx.KVX_ERR_INVALID_ARG
    assert kvx.kvx_attend8_workspace_bytes(attend_args(c)) == 0
    assert kvx.kvx_evict8_workspace_bytes(evict_args(c)) == 0


@pytest.mark.parametrize("over", [
    dict(dtype=3), dict(num_requests=0), dict(ntok=-1), dict(ntok=2 ** 31), dict(cu_seqlens=None),
    dict(k=None), dict(v=None), dict(k=P + 1), dict(src_rows=P, num_src_rows=0)])
def test_write_refuses(over):
    assert kvx.kvx_cache8_write(write_args(**over), None) == kvx.KVX_ERR_INVALID_ARG
    assert kvx.kvx_cache8_write(write_args(ntok=0), None) == kvx.KVX_OK


@pytest.mark.parametrize("over", [
    dict(dtype=3), dict(num_requests=0), dict(ntok=-1), dict(cu_seqlens=None), dict(max_new=0),
    dict(max_len=-1), dict(lens=None), dict(scale=float("nan")), dict(q_heads=5), dict(q_heads=0),
    dict(weights=P, weights_stride=63)])
def test_attend_refuses(over):
    assert kvx.kvx_attend8(attend_args(**over), None) == kvx.KVX_ERR_INVALID_ARG
    assert kvx.kvx_attend8_workspace_bytes(attend_args(**over)) == 0


def test_attend_refuses_pointers_and_small_workspaces():
    need = kvx.kvx_attend8_workspace_bytes(attend_args())
    assert need > 0
    for over in (dict(q=None), dict(out=None), dict(q=P + 1), dict(workspace=None),
                 dict(workspace=P + 16), dict(workspace_bytes=need - 1)):
        assert kvx.kvx_attend8(attend_args(**over), None) == kvx.KVX_ERR_INVALID_ARG
    assert kvx.kvx_attend8(attend_args(ntok=0), None) == kvx.KVX_OK


@pytest.mark.parametrize("over", [
    dict(dst_table=None), dict(max_dst_blocks=1), dict(num_requests=0), dict(num_requests=65536),
    dict(lens=None), dict(max_len=-1), dict(keep=0), dict(sinks=-1), dict(recent=-1),
    dict(sinks=20, recent=13), dict(weights=None), dict(weights_stride=63), dict(kept=None),
    dict(new_lens=None)])
def test_evict_refuses(over):
    assert kvx.kvx_evict8(evict_args(**over), None) == kvx.KVX_ERR_INVALID_ARG
    assert kvx.kvx_evict8_workspace_bytes(evict_args(**over)) == 0


def test_evict_refuses_small_workspaces():
    need = kvx.kvx_evict8_workspace_bytes(evict_args())
    for over in (dict(workspace=None), dict(workspace=P + 16), dict(workspace_bytes=need - 1)):
        assert kvx.kvx_evict8(evict_args(**over), None) == kvx.KVX_ERR_INVALID_ARG


def test_python_checks():
    torch = pytest.importorskip("torch")
    u8 = torch.zeros((4, 2, 16, 64), dtype=torch.uint8)
    f = torch.ones((4, 2))
    with pytest.raises(ValueError):
        kvx.Cache8(u8, u8[:3], f, f)
    with pytest.raises(ValueError):
        kvx.Cache8(u8, u8, f, f.double())
    with pytest.raises(ValueError):
        kvx.Cache8(u8.float(), u8, f, f)
    with pytest.raises(ValueError):
        kvx.Rope(64, 1e4, layout="both")
    with pytest.raises(kvx.KvxError):
        kvx.Rope(64, 1e4, rot_dim=65)
    cache = kvx.Cache8(u8, u8.clone(), f, f.clone())
    with pytest.raises(ValueError):       # the tensors are not on the current CUDA device
        cache.write(torch.zeros((1, 2, 64)), torch.zeros((1, 2, 64)),
                    torch.zeros((1, 1), dtype=torch.int32))


def test_structures_match_the_c_layout(tmp_path):
    import os
    import subprocess
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    fields = {"kvx_rope_desc": kvx.RopeDesc, "kvx_rope": kvx.RopeState, "kvx_rope_args": kvx.RopeArgs,
              "kvx_cache8": kvx.Cache8Desc, "kvx_cache8_write_args": kvx.Cache8WriteArgs,
              "kvx_attend8_args": kvx.Attend8Args, "kvx_evict8_args": kvx.Evict8Args}
    lines = ['#include <stdio.h>', '#include <stddef.h>', '#include "kvx.h"', "int main(void){"]
    for cname, cls in fields.items():
        lines.append(f'printf("{cname} %zu\\n", sizeof({cname}));')
        lines += [f'printf("{cname}.{f} %zu\\n", offsetof({cname}, {f}));' for f, _ in cls._fields_]
    lines.append("return 0;}")
    (tmp_path / "p.c").write_text("\n".join(lines))
    subprocess.run(["gcc", "-I", os.path.join(root, "include"), str(tmp_path / "p.c"), "-o",
                    str(tmp_path / "p")], check=True)
    got = dict(ln.split() for ln in subprocess.run([str(tmp_path / "p")], capture_output=True,
                                                    text=True, check=True).stdout.splitlines())
    for cname, cls in fields.items():
        assert int(got[cname]) == ctypes.sizeof(cls), cname
        for f, _ in cls._fields_:
            assert int(got[f"{cname}.{f}"]) == getattr(cls, f).offset, f"{cname}.{f}"


def test_the_reference_forms():
    """Worked examples of the fp64 forms that the GPU tests compare with."""
    assert ref.E4M3[0x7E] == 448.0 and ref.E4M3[0x01] == 2.0 ** -9 and ref.E4M3[0x08] == 2.0 ** -6
    assert ref.e4m3_round(np.array([0.0, 1.0, 17.0, 19.0, 1e9, -1e9, 2.0 ** -10, 1.5 * 2.0 ** -9])
                          ).tolist() == [0.0, 1.0, 16.0, 20.0, 448.0, -448.0, 0.0, 2.0 ** -8]
    assert ref.pow2_scale(448.0) == 1.0 and ref.pow2_scale(449.0) == 2.0
    assert ref.pow2_scale(0.0) == 2.0 ** -126
    w = np.array([[[5.0, 1.0, 3.0, 3.0, 9.0, 0.0]]])
    assert ref.evict(w, [6], 3, 1, 1).tolist() == [[[0, 4, 5]]]
    assert ref.evict(w, [6], 4, 0, 1).tolist() == [[[0, 2, 4, 5]]]
    assert ref.evict(w, [2], 3, 1, 1).tolist() == [[[0, 1, -1]]]
    x = ref.rope(np.array([[[1.0, 2.0, 3.0, 4.0]]]), np.array([np.pi / 2]), 2, "half",
                 np.array([1.0]), 1.0)
    assert np.allclose(x, [[[-2.0, 1.0, 3.0, 4.0]]])
