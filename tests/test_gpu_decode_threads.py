"""Decoding calls from several host threads at once, each with its own cache,
stream and sizes: what one thread's call sets for a kernel must serve the other's."""
import ctypes
import threading

import pytest
import torch

from cross_model_kv_transfer_gb300 import kvx
from test_gpu_evict8 import dev, make

pytestmark = pytest.mark.gpu


def test_evictions_of_different_lengths_from_several_threads():
    jobs, errors = [], []
    keep = 64
    for i, n in enumerate((90000, 170000, 64000, 120000)):
        c = make(1, 16, 16, [n], keep, 30 + i)
        cache, w, table, lens, to = (c["cache"], torch.tensor(c["w"]).cuda(), dev(c["table"]), dev([n]),
                                     dev(c["to"]))
        want = cache.evict(w, table, lens, to, max_len=n, keep=keep, sinks=4, recent=8)
        got = [torch.zeros_like(t) for t in want]
        ws = cache.evict_workspace(num_requests=1, max_len=n, keep=keep)
        desc = kvx.Cache8Desc(cache.k_codes.data_ptr(), cache.v_codes.data_ptr(), cache.k_scale.data_ptr(),
                              cache.v_scale.data_ptr(), cache.num_blocks, 1, 16, 16, table.shape[1], table.data_ptr())
        a = kvx.Evict8Args(cache=desc, dst_table=to.data_ptr(), max_dst_blocks=to.shape[1], num_requests=1,
                           lens=lens.data_ptr(), max_len=n, keep=keep, sinks=4, recent=8, weights=w.data_ptr(),
                           weights_stride=w.shape[2], kept=got[0].data_ptr(), kept_weights=got[1].data_ptr(),
                           new_lens=got[2].data_ptr(), workspace=ws.data_ptr(), workspace_bytes=ws.numel())
        jobs.append((a, n, want, got, torch.cuda.Stream(), (cache, w, table, lens, to, ws)))
    torch.cuda.synchronize()
    start = threading.Barrier(len(jobs))
    evict = kvx.load().kvx_evict8

    def work(a, n, want, got, stream, held):
        try:
            torch.cuda.set_device(0)
            args, raw = ctypes.byref(a), stream.cuda_stream
            start.wait(30)
            for _ in range(4000):
                st = evict(args, raw)
                if st != kvx.KVX_OK:
                    errors.append(f"{n}: status {st}")
                    break
            stream.synchronize()
            if not all(torch.equal(x, y) for x, y in zip(want, got)):
                errors.append(f"{n}: other results")
        except Exception as e:     # noqa: BLE001 -- a thread's exception would be lost
            errors.append(f"{n}: {e!r}")

    threads = [threading.Thread(target=work, args=j) for j in jobs]
    for t in threads:
        t.start()
    for t in threads:
        t.join(120)
    assert not errors, errors
    assert all(not t.is_alive() for t in threads)
