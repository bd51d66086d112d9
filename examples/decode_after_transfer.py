"""Answer from a transferred cache: transfer, 8-bit cache, decoding, eviction.

A target model's cache is filled from a pilot's by one transfer (bf16, paged);
each layer's part is quantised into an 8-bit paged cache, the prompts' last
tokens and every decoded token attend to it and add up the attention weight of
its slots, and when the requests hold more than the budget the slots that
attention used least are evicted.  Weights, pilot caches and the target's
queries, keys and values are synthetic.

    python examples/decode_after_transfer.py
"""
import dataclasses
import os
import sys

import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)

from cross_model_kv_transfer_gb300 import kvx
from cross_model_kv_transfer_gb300.workloads import WORKLOADS, make_inputs


def transfer(wl):
    """The pilot's caches mapped into a paged bf16 cache of the target."""
    inp = {k: v.cuda() if torch.is_tensor(v) else v for k, v in make_inputs(wl, "cpu").items()}
    plan = kvx.Plan(src_layers=wl.src_layers, tgt_layers=wl.tgt_layers, kv_heads=wl.kv_heads,
                    head_dim=wl.head_dim, k=wl.k, rope_theta_src=wl.theta_src,
                    rope_theta_tgt=wl.theta_tgt, max_position=wl.max_position,
                    kv_dtype=wl.kv_dtype, w_dtype=torch.float32, b_dtype=wl.b_dtype,
                    layout=wl.layout, block_size=wl.block_size)
    shape = (wl.tgt_layers, wl.num_blocks * wl.block_size, wl.kv_heads, wl.head_dim)
    dst_k, dst_v = (torch.zeros(shape, dtype=wl.kv_dtype, device="cuda") for _ in range(2))
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    plan.transfer(src_k=inp["src_k"], src_v=inp["src_v"], layer_idx=inp["layer_idx"], w=inp["w"],
                  b=inp["b"], dst_k=dst_k, dst_v=dst_v, cu_seqlens=inp["cu_seqlens"],
                  block_table=inp["block_table"], num_blocks=wl.num_blocks, status=status)
    return dst_k, dst_v, inp["block_table"], inp["cu_seqlens"], status


def run(prompts=(70, 200), layers=2, window=16, steps=(24, 24), keep=64, sinks=4, recent=16,
        group=8, seed=11, watch=None):
    """Two stretches of decoding with an eviction between them; ``watch(stage,
    layer, **tensors)`` sees what each call read and wrote.  Returns the
    requests' final lengths and the status flags (0: none)."""
    wl = dataclasses.replace(WORKLOADS["llama31_8b_70b_paged"].with_tokens(prompts, [0] * len(prompts)),
                             tgt_layers=layers)
    watch = watch or (lambda stage, layer, **tensors: None)
    R, H, d, bs = len(prompts), wl.kv_heads, wl.head_dim, wl.block_size
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")
    g = torch.Generator().manual_seed(seed)
    draw = lambda n, heads: torch.randn((n, heads, d), generator=g).to(torch.bfloat16).cuda()

    dst_k, dst_v, paged, cu, status = transfer(wl)
    # where the transfer put each token, as rows of its pool
    rows = torch.cat([(paged[r, torch.arange(n, device="cuda") // bs] * bs
                       + torch.arange(n, device="cuda") % bs) for r, n in enumerate(prompts)]).int()

    # blocks of the 8-bit pool: for the prompts and what is decoded, then for what eviction keeps
    most = [n + sum(steps) for n in prompts]
    per, per_kept = -(-max(most) // bs), -(-(keep + steps[1]) // bs)
    order = torch.randperm(R * (per + per_kept), generator=g).int().cuda()
    table, fresh = order[:R * per].view(R, per), order[R * per:].view(R, per_kept)
    caches = [kvx.Cache8.empty(R * (per + per_kept), H, d, bs) for _ in range(layers)]
    rope = kvx.Rope(d, wl.theta_tgt)
    weights = [torch.zeros((R, H, max(most)), device="cuda") for _ in range(layers)]
    max_len = max(most)
    scratch = caches[0].attend_workspace(ntok=R * window, num_requests=R, q_heads=H * group,
                                         max_len=max_len, max_new=window, weights=True)

    # the transferred tokens, quantised; the prompts' last tokens vote for slots
    ends = [min(window, n) for n in prompts]
    cu_w = i32([0] + torch.tensor(ends).cumsum(0).tolist())
    positions = torch.cat([torch.arange(n - e, n) for n, e in zip(prompts, ends)]).int().cuda()
    lens = i32(list(prompts))
    for l, cache in enumerate(caches):
        cache.write(dst_k[l], dst_v[l], table, cu_seqlens=cu, src_rows=rows, status=status)
        watch("write", l, cache=cache, table=table, lens=lens, k=dst_k[l], v=dst_v[l], rows=rows)
        q, _ = rope.apply(draw(sum(ends), H * group), positions=positions, status=status)
        out, lse = cache.attend(q, table, lens, max_len, cu_seqlens=cu_w, max_new=window,
                                weights=weights[l], workspace=scratch, status=status)
        watch("attend", l, cache=cache, table=table, lens=lens, q=q, out=out, lse=lse, cu=cu_w)

    position = lens.clone()      # of the next token: evicted slots do not move it back
    for stretch in range(2):
        for _ in range(steps[stretch]):
            after = lens + 1
            for l, cache in enumerate(caches):
                q, k = rope.apply(draw(R, H * group), draw(R, H), position, status=status)
                cache.write(k, draw(R, H), table, start=lens, status=status)
                out, lse = cache.attend(q, table, after, max_len, weights=weights[l],
                                        workspace=scratch, status=status)
                watch("attend", l, cache=cache, table=table, lens=after, q=q, out=out, lse=lse,
                      cu=None)
            lens, position = after, position + 1
        if stretch == 0:
            for l, cache in enumerate(caches):
                kept, kept_weights, left = cache.evict(weights[l], table, lens, fresh, max_len=max_len,
                                                       keep=keep, sinks=sinks, recent=recent,
                                                       status=status)
                watch("evict", l, cache=cache, weights=weights[l], lens=lens, kept=kept,
                      kept_weights=kept_weights, new_lens=left)
                weights[l].zero_()
                weights[l][:, :, :keep] = kept_weights
            table, lens = fresh, left
    return lens.tolist(), int(status.item())


if __name__ == "__main__":
    def report(stage, layer, **t):
        if stage == "evict":
            share = t["kept_weights"].sum().item() / t["weights"].sum().item()
            print(f"layer {layer}: slots {t['lens'].tolist()} -> {t['new_lens'].tolist()}, "
                  f"{100 * share:.1f} % of the attention weight stays")

    final, flags = run(watch=report)
    print(f"slots at the end {final}, flags {flags}")
