"""Beam search on transferred prompts: one copy of each prompt, many continuations.

The target's cache of each prompt is filled by one transfer and quantised into
pages of an 8-bit pool; the beams of a prompt share those pages and hold pages of
their own for what they decode.  In every step the beams' next slots are reserved
(a page that several beams share is copied before one of them writes to it), the
new tokens attend to the shared prompt and to their own slots, the best candidates
are chosen, and the block table's rows are forked to them.  Half-way the first
prompt is dropped and the pool compacted.  The target is synthetic: two small
matrices a layer around the attention, random embeddings and a random vocabulary.

    python examples/beams_after_transfer.py
"""
import dataclasses
import os
import sys

import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
for path in (ROOT, os.path.dirname(os.path.abspath(__file__))):
    if path not in sys.path:
        sys.path.insert(0, path)

from cross_model_kv_transfer_gb300 import kvx
from cross_model_kv_transfer_gb300.workloads import WORKLOADS
from decode_after_transfer import transfer


class Target:
    """What the example needs of a model: from tokens to queries, keys and values of a
    layer, and from the last hidden state to logits."""

    def __init__(self, layers, heads, group, d, vocab, seed, hidden=64):
        g = torch.Generator().manual_seed(seed)
        draw = lambda *s: (torch.randn(s, generator=g) / s[-2] ** 0.5).cuda()
        self.embed = draw(vocab, hidden) * vocab ** 0.5
        self.layers = [(draw(hidden, (group + 2) * heads * d), draw(group * heads * d, hidden))
                       for _ in range(layers)]
        self.head = 3 * draw(hidden, vocab)
        self.shape = (heads, group, d)

    def qkv(self, l, x):
        H, G, d = self.shape
        y = (x @ self.layers[l][0]).to(torch.bfloat16).view(x.shape[0], (G + 2) * H, d)
        return y[:, :G * H], y[:, G * H:(G + 1) * H], y[:, (G + 1) * H:]

    def after(self, l, x, out):
        return x + out.flatten(1).float() @ self.layers[l][1]

    def logits(self, x):
        return (x @ self.head).to(torch.bfloat16)


def run(prompts=(70, 200), layers=2, beams=4, steps=(10, 10), vocab=1000, group=8, eos=1, seed=5,
        watch=None):
    """Two stretches of beam search; the first prompt is dropped between them and the
    pool compacted.  ``watch(stage, **tensors)`` sees what the calls read and wrote.
    Returns (token histories of the prompts that are left, scores, flags); a row without a
    beam has a history of -1 and a score of -inf."""
    wl = dataclasses.replace(WORKLOADS["llama31_8b_70b_paged"].with_tokens(prompts, [0] * len(prompts)),
                             tgt_layers=layers)
    watch = watch or (lambda stage, **tensors: None)
    P, H, d, bs = len(prompts), wl.kv_heads, wl.head_dim, wl.block_size
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")
    target = Target(layers, H, group, d, vocab, seed)
    rope = kvx.Rope(d, wl.theta_tgt)
    dst_k, dst_v, paged, cu, status = transfer(wl)
    rows = torch.cat([(paged[r, torch.arange(n, device="cuda") // bs] * bs
                       + torch.arange(n, device="cuda") % bs) for r, n in enumerate(prompts)]).int()

    # one pool for prompts and continuations
    width, own_width = -(-max(prompts) // bs), -(-sum(steps) // bs) + 1
    blocks = sum(-(-n // bs) for n in prompts) + 2 * P * beams * own_width
    pages = kvx.Pages.empty(blocks, bs)
    scratch = pages.workspace()
    caches = [kvx.Cache8.empty(blocks, H, d, bs) for _ in range(layers)]
    prefix = torch.full((P, width), -1, dtype=torch.int32, device="cuda")
    before = i32(list(prompts))
    pages.reserve(prefix, torch.zeros_like(before), before, max_new=max(prompts), workspace=scratch,
                  status=status)
    for l, cache in enumerate(caches):
        cache.write(dst_k[l], dst_v[l], prefix, cu_seqlens=cu, src_rows=rows, status=status)
    table = torch.full((P * beams, own_width), -1, dtype=torch.int32, device="cuda")
    lens = torch.zeros(P * beams, dtype=torch.int32, device="cuda")
    # at first one beam of each prompt counts, so that it goes on in several ways
    scores = torch.full((P, beams), float("-inf"), device="cuda")
    scores[:, 0] = 0.0
    done = torch.zeros((P, beams), dtype=torch.bool, device="cuda")
    tokens = torch.zeros(P * beams, dtype=torch.int32, device="cuda")
    history = torch.zeros((P * beams, 0), dtype=torch.int32, device="cuda")
    attend = caches[0].attend_shared_workspace(
        ntok=P * beams, num_requests=P * beams, q_heads=H * group, max_prefix=max(prompts),
        max_len=sum(steps), num_prefixes=P, max_group=beams)
    choose = kvx.beam_workspace(requests=P, beams=beams, vocab=vocab)

    for stretch in range(2):
        groups = i32([beams * p for p in range(prefix.shape[0] + 1)])
        for _ in range(steps[stretch]):
            pages.reserve(table, lens, 1, caches=caches, workspace=scratch, status=status)
            x = target.embed[tokens.long().clamp(min=0)]     # rows without a beam go along
            position = (before.repeat_interleave(beams) + lens).int()
            after = lens + 1
            for l, cache in enumerate(caches):
                q, k, v = target.qkv(l, x)
                q, k = rope.apply(q, k, position, status=status)
                cache.write(k, v, table, start=lens, status=status)
                out, lse = cache.attend_shared(q, prefix, before, table, after, groups=groups,
                                               max_prefix=max(prompts), max_len=sum(steps),
                                               max_group=beams, workspace=attend, status=status)
                watch("attend", layer=l, cache=cache, q=q, k=k, v=v, out=out, lse=lse, prefix=prefix,
                      before=before, table=table, lens=after, groups=groups)
                x = target.after(l, x, out)
            logits = target.logits(x)
            chosen, parents, new_scores, new_done = kvx.beam_select(
                logits, scores, eos=eos, done=done, workspace=choose, status=status)
            watch("select", logits=logits, scores=scores, done=done, tokens=chosen, parents=parents,
                  new_scores=new_scores, new_done=new_done)
            parents, tokens = parents.view(-1), chosen.view(-1)
            new_table, new_lens = pages.fork(table, after, parents, status=status)
            watch("fork", pages=pages, old=table, old_lens=after, parents=parents, table=new_table,
                  lens=new_lens, prefix=prefix)
            table, lens, scores, done = new_table, new_lens, new_scores, new_done
            # a prompt with fewer candidates than beams has rows without one: parents and tokens of -1
            kept = torch.where(parents[:, None] < 0, parents[:, None], history[parents.long().clamp(min=0)])
            history = torch.cat([kept, tokens[:, None]], 1)
        if stretch == 0 and P > 1:
            # the first prompt is answered: its pages go, the others move together
            pages.free(prefix[:1], status=status)
            pages.free(table[:beams], status=status)
            prefix, before, table, lens = prefix[1:], before[1:], table[beams:], lens[beams:]
            scores, done, tokens, history = scores[1:], done[1:], tokens[beams:], history[beams:]
            used, moved = pages.compact([prefix, table], caches, workspace=scratch, status=status)
            watch("compact", pages=pages, used=used, moved=moved, table=table, prefix=prefix)
    return history, scores, int(status.item())


if __name__ == "__main__":
    def report(stage, **t):
        if stage == "compact":
            print(f"{int(t['used'].item())} of {t['pages'].num_blocks} pages are held after the first prompt")

    history, scores, flags = run(watch=report)
    for row, s in zip(history.tolist(), scores.view(-1).tolist()):
        print(f"score {s:8.3f}  tokens {row}")
    print(f"flags {flags}")
