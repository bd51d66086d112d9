"""The example that decodes after a transfer: every call of it against the plain
fp64 forms, on what that call read."""
import importlib.util
import os

import numpy as np
import pytest
import torch

import decode_reference as ref
from test_gpu_attend8 import compare

pytestmark = pytest.mark.gpu
PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples",
                    "decode_after_transfer.py")


def f64(t):
    return t.detach().double().cpu().numpy()


def test_every_step_of_it():
    spec = importlib.util.spec_from_file_location("decode_after_transfer", PATH)
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    seen = dict(write=0, attend=0, evict=0)

    def watch(stage, layer, **t):
        seen[stage] += 1
        cache = t["cache"]
        if stage == "write":
            # nearest of 4 significand bits at the block's scale, which brings the
            # largest magnitude to (224, 448]: within 2^-4 of it, and 2^-10 scales
            table, lens = t["table"].cpu().numpy(), t["lens"].tolist()
            for codes, scale, x in ((cache.k_codes, cache.k_scale, t["k"]),
                                    (cache.v_codes, cache.v_scale, t["v"])):
                got = ref.RefCache(codes.cpu().numpy(), scale.cpu().numpy())
                want, at = f64(x)[t["rows"].cpu().numpy()], 0
                for r, n in enumerate(lens):
                    for h in range(cache.heads):
                        y, w = got.rows(table[r], range(n), h), want[at:at + n, h]
                        s = np.array([got.scale[table[r][j // 16], h] for j in range(n)])[:, None]
                        assert (np.abs(y - w) <= 2.0 ** -4 * np.abs(w) + 2.0 ** -10 * s).all()
                    at += n
        elif stage == "attend" and (seen["attend"] % 7 == 0 or t["cu"] is not None):
            k = ref.RefCache(cache.k_codes.cpu().numpy(), cache.k_scale.cpu().numpy())
            v = ref.RefCache(cache.v_codes.cpu().numpy(), cache.v_scale.cpu().numpy())
            lens = t["lens"].tolist()
            cu = np.arange(len(lens) + 1) if t["cu"] is None else t["cu"].cpu().numpy()
            want = ref.attend(f64(t["q"]), k, v, t["table"].cpu().numpy(), lens, cu,
                              cache.head_dim ** -0.5)
            compare(t["out"], t["lse"], None, want, True, max(lens), 8 * int(np.diff(cu).max()))
        elif stage == "evict":
            want = ref.evict(t["weights"].cpu().numpy(), t["lens"].tolist(), 64, 4, 16)
            assert np.array_equal(t["kept"].cpu().numpy(), want)
            # each query of each head of the group gave a weight of one in all
            given = t["weights"].sum(-1).cpu().numpy()
            assert np.abs(given - 8 * (16 + 24)).max() <= 8 * 40 * 2.0 ** -12

    lens, flags = example.run(watch=watch)
    torch.cuda.synchronize()
    assert flags == 0 and lens == [64 + 24, 64 + 24]
    assert seen == dict(write=2, attend=2 * (1 + 48), evict=2)
