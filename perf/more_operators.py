"""Measured cases of the operators with which a target model continues one
transferred prompt in several ways at once: attention of a batch over a shared
prefix, the references to a cache's pages (rows forked, pages reserved, copied
and compacted) and beam search's selection.

``run`` computes each operator either in plain torch operations (``own`` false)
or through the library's entry points (``own`` true); ``exact`` computes it in
fp64, written apart from both.

The 8-bit cache: e4m3 codes [blocks][H][block][d] and one fp32 scale for each
(block, head) of the keys and of the values.  A block table names a row's pages,
-1 where it has none; refs[b] counts the rows that hold page b.
"""
import math

import torch

own = False

DEV = "cuda"
DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16}


def listed():
    return [
        # eight beams of one prompt, one token each: latency
        dict(name="shared_beams", op="shared", prefixes=1, members=8, shortest=4096, longest=4096,
             own_len=48, new=1, q_heads=64, kv_heads=8, head_dim=128, block=16, dtype="bf16"),
        # a small model in fp32, two odd prompts with five samples each
        dict(name="shared_f32", op="shared", prefixes=2, members=5, shortest=333, longest=777,
             own_len=29, new=1, q_heads=8, kv_heads=2, head_dim=64, block=16, dtype="f32"),
        # ragged prompts with sixteen samples each
        dict(name="shared_samples", op="shared", prefixes=4, members=16, shortest=1024,
             longest=16384, own_len=500, new=1, q_heads=64, kv_heads=8, head_dim=128, block=16,
             dtype="bf16"),
        # one long document asked by 64 requests, three tokens each at a time
        dict(name="shared_document", op="shared", prefixes=1, members=64, shortest=65535,
             longest=65535, own_len=1024, new=3, q_heads=64, kv_heads=8, head_dim=128, block=64,
             dtype="bf16"),
        # four beams of one short request, one layer's cache: latency
        dict(name="reorder_one", op="reorder", requests=1, beams=4, longest=100, new=1, blocks=64,
             layers=1, heads=8, head_dim=128, block=16),
        # a beam step of 16 requests with 8 beams: rows forked, last pages copied for 8 layers
        dict(name="reorder_batch", op="reorder", requests=16, beams=8, longest=2000, new=1,
             blocks=16384, layers=8, heads=2, head_dim=128, block=16),
        # the same in a pool of many small pages, rows of whole conversations, draft tokens
        dict(name="reorder_long", op="reorder", requests=64, beams=4, longest=16384, new=7,
             blocks=131072, layers=2, heads=1, head_dim=64, block=16),
        # a small pool with holes
        dict(name="compact_small", op="compact", rows=16, longest=300, blocks=512, held=0.5,
             layers=1, heads=8, head_dim=128, block=16),
        # a large pool of which half is free, four layers
        dict(name="compact_large", op="compact", rows=64, longest=1000, blocks=4096, held=0.5,
             layers=4, heads=8, head_dim=128, block=16),
        # one request of four beams
        dict(name="beam_one", op="beam", requests=1, beams=4, out=4, vocab=32000, dtype="f32",
             ended=False),
        # sixteen requests of eight beams, some of which have ended
        dict(name="beam_batch", op="beam", requests=16, beams=8, out=8, vocab=128256,
             dtype="bf16", ended=True),
        # many beams over a large vocabulary
        dict(name="beam_wide", op="beam", requests=8, beams=32, out=32, vocab=151936, dtype="f32",
             ended=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["shared", "shared", "reorder", "compact", "beam"])
    heads, d = rng.choice([1, 2, 4, 8]), rng.choice([64, 128])
    block = rng.choice([8, 16, 24, 32, 64])
    if op == "shared":
        P = _log(rng, 1, 8)
        members = _log(rng, 1, 64)
        hi = _log(rng, 16, max(16, 65536 // P))
        new = min(rng.choice([1, 1, 1, 2, 5]), max(1, 192 // members))
        return dict(op="shared", prefixes=P, members=members, shortest=rng.randint(1, hi),
                    longest=hi, own_len=max(new, _log(rng, 1, max(1, min(1024, 65536 // (P * members))))),
                    new=new, q_heads=heads * rng.choice([1, 2, 4, 5, 8]), kv_heads=heads,
                    head_dim=d, block=block, dtype=rng.choice(["bf16", "bf16", "f32"]))
    if op == "reorder":
        R, K = _log(rng, 1, 32), rng.choice([1, 2, 3, 4, 8])
        hi = _log(rng, 16, min(4096, 65536 // R))
        new = rng.choice([1, 1, 1, 2, 9, 40])
        most = R * (-(-hi // block) + K * (3 + -(-new // block)))
        return dict(op="reorder", requests=R, beams=K, longest=hi, new=new,
                    blocks=most + rng.randint(1, most),
                    layers=rng.randint(1, max(1, min(8, 2 ** 28 // (most * heads * block * d)))),
                    heads=heads, head_dim=d, block=block)
    if op == "compact":
        blocks = _log(rng, 64, 4096)
        return dict(op="compact", rows=_log(rng, 1, 64), longest=_log(rng, block, 2000),
                    blocks=blocks, held=rng.uniform(0.1, 0.9),
                    layers=rng.randint(1, max(1, min(6, 2 ** 28 // (blocks * heads * block * d)))),
                    heads=heads, head_dim=d, block=block)
    R, K = _log(rng, 1, 32), _log(rng, 1, 32)
    return dict(op="beam", requests=R, beams=K, out=rng.choice([K, K, rng.randint(1, 32)]),
                vocab=_log(rng, 50, max(2000, min(262144, 2 ** 25 // (R * K)))),
                dtype=rng.choice(["bf16", "f32"]), ended=rng.random() < 0.5)


# --- what a program has in hand ----------------------------------------------

def _ints(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def _prefix_lengths(case):
    P, lo, hi = case["prefixes"], case["shortest"], case["longest"]
    return [hi if P == 1 else lo + (hi - lo) * r // (P - 1) for r in range(P)]


def _own_lengths(case):
    """Slots of the requests' own, from their new tokens up to the most, spread."""
    R, lo, hi = case["prefixes"] * case["members"], case["new"], case["own_len"]
    return [lo + (hi - lo) * (r * 7 % R + 1) // R for r in range(R)]


def _table(pages, order):
    """A block table of rows with these many pages, taken from `order`, and how many."""
    most = max(1, max(pages))
    table = torch.full((len(pages), most), -1, dtype=torch.int32, device=DEV)
    at = 0
    for r, n in enumerate(pages):
        table[r, :n] = order[at:at + n]
        at += n
    return table, at


def _filled_cache(blocks, H, bs, d, g):
    """Codes and scales of a cache that earlier writes filled."""
    x = torch.randn((blocks, H, bs, d), generator=g, device=DEV)
    x *= torch.exp(0.5 * torch.randn((H, 1, d), generator=g, device=DEV))
    m, e = torch.frexp(x.abs().amax((2, 3)))
    scale = torch.ldexp(torch.ones_like(m), e - 9 + (m > 0.875).to(e.dtype))
    x /= scale[:, :, None, None]
    return x.to(torch.float8_e4m3fn).view(torch.uint8), scale


def prepare(case, seed):
    g = _gen(seed)
    s = {"case": case}
    op = case["op"]
    if op == "shared":
        H, Hq, d, bs, new = (case[k] for k in ("kv_heads", "q_heads", "head_dim", "block", "new"))
        P, M = case["prefixes"], case["members"]
        before, lens = _prefix_lengths(case), _own_lengths(case)
        pages, own_pages = [-(-n // bs) for n in before], [-(-n // bs) for n in lens]
        blocks = sum(pages) + sum(own_pages) + 1
        order = torch.randperm(blocks, generator=g, device=DEV).to(torch.int32)
        s["prefix_table"], at = _table(pages, order)
        s["table"], _ = _table(own_pages, order[at:])
        s["prefix_lens"], s["lens"] = _ints(before), _ints(lens)
        s["groups"] = _ints([M * p for p in range(P + 1)])
        s["cu"] = _ints([new * r for r in range(P * M + 1)])
        s["max_prefix"], s["max_len"] = max(before), max(lens)
        for m in "kv":
            s[m + "_codes"], s[m + "_scale"] = _filled_cache(blocks, H, bs, d, g)
        s["q"] = (1.5 * torch.randn((P * M * new, Hq, d), generator=g, device=DEV)).to(
            DTYPES[case["dtype"]])
        s["scale"] = 1.0 / math.sqrt(d)
    elif op == "reorder":
        R, K, bs, hi = (case[k] for k in ("requests", "beams", "block", "longest"))
        lens = [max(1, hi - (hi - 1) * r // R // 2) for r in range(R) for _ in range(K)]
        held = [-(-n // bs) for n in lens]
        # beams of one request share all pages but their last one or two
        own_pages = [min(n, 1 + (k + r) % 2) for r, n in enumerate(held[::K]) for k in range(K)]
        order = torch.randperm(case["blocks"], generator=g, device=DEV).to(torch.int32)
        s["table"] = torch.full((R * K, -(-(hi + case["new"]) // bs)), -1, dtype=torch.int32,
                                device=DEV)
        at = 0
        for r in range(R):
            n = held[r * K]
            for k in range(K):
                row = s["table"][r * K + k]
                if k == 0:
                    row[:n] = order[at:at + n]
                    at += n
                else:
                    row[:n] = s["table"][r * K, :n]
                    mine = own_pages[r * K + k]
                    row[n - mine:n] = order[at:at + mine]
                    at += mine
        s["lens"] = _ints(lens)
        s["refs"] = torch.bincount(s["table"][s["table"] >= 0].long(),
                                   minlength=case["blocks"]).to(torch.int32)
        pick = torch.randint(0, K, (R, K), generator=g, device=DEV).sort(1)[0]
        s["parents"] = (pick + K * torch.arange(R, device=DEV)[:, None]).reshape(-1).to(torch.int32)
        s["caches"] = [(*_filled_cache(case["blocks"], case["heads"], bs, case["head_dim"], g),
                        *_filled_cache(case["blocks"], case["heads"], bs, case["head_dim"], g))
                       for _ in range(case["layers"])]
    elif op == "compact":
        bs, blocks = case["block"], case["blocks"]
        n, width = case["rows"], -(-case["longest"] // bs)
        used = max(1, min(blocks - 1, int(blocks * case["held"])))
        order = torch.randperm(blocks, generator=g, device=DEV)[:used]
        # the first pages are shared by rows, the others held by one row each
        pick = torch.randint(0, used, (n, width), generator=g, device=DEV)
        table = order[pick].to(torch.int32)
        width_of = torch.randint(1, width + 1, (n, 1), generator=g, device=DEV)
        s["table0"] = torch.where(torch.arange(width, device=DEV) < width_of, table,
                                  torch.full_like(table, -1))
        s["refs0"] = torch.bincount(s["table0"][s["table0"] >= 0].long(), minlength=blocks).to(torch.int32)
        s["refs0"][order] += (s["refs0"][order] == 0).to(torch.int32)      # held by other tables
        s["caches"] = [(*_filled_cache(blocks, case["heads"], bs, case["head_dim"], g),
                        *_filled_cache(blocks, case["heads"], bs, case["head_dim"], g))
                       for _ in range(case["layers"])]
    else:
        R, K, V = case["requests"], case["beams"], case["vocab"]
        s["logits"] = (2.5 * torch.randn((R * K, V), generator=g, device=DEV)).to(
            DTYPES[case["dtype"]])
        s["scores"] = -20.0 + 4.0 * torch.randn((R, K), generator=g, device=DEV)
        s["done"] = (torch.rand((R, K), generator=g, device=DEV) < 0.2) if case["ended"] else None
    if own:
        _handles(s)
    return s


def _handles(s):
    """The library's objects that a program keeps beside its tensors."""
    from cross_model_kv_transfer_gb300 import kvx
    case = s["case"]
    op = case["op"]
    if op == "shared":
        c = s["cache"] = kvx.Cache8(s["k_codes"], s["v_codes"], s["k_scale"], s["v_scale"])
        s["workspace"] = c.attend_shared_workspace(
            ntok=s["q"].shape[0], num_requests=s["lens"].shape[0], num_prefixes=case["prefixes"],
            q_heads=case["q_heads"], max_prefix=s["max_prefix"], max_len=s["max_len"],
            max_group=case["members"], max_new=case["new"], dtype=s["q"].dtype)
    elif op in ("reorder", "compact"):
        s["handles"] = [kvx.Cache8(kc, vc, ks, vs) for kc, ks, vc, vs in s["caches"]]
        if op == "reorder":
            s["pages"] = kvx.Pages(s["refs"], case["block"])
        s["workspace"] = kvx.Pages(s["refs" if op == "reorder" else "refs0"], case["block"]).workspace()
    else:
        s["workspace"] = kvx.beam_workspace(requests=case["requests"], beams=case["beams"],
                                            vocab=case["vocab"], out=case["out"])


# --- the operators --------------------------------------------------------------

def run(state):
    if own:
        return _run_own(state)
    return {"shared": _shared, "reorder": _reorder, "compact": _compact, "beam": _beam}[
        state["case"]["op"]](state)


def _run_own(s):
    from cross_model_kv_transfer_gb300 import kvx
    case = s["case"]
    op = case["op"]
    if op == "shared":
        return list(s["cache"].attend_shared(
            s["q"], s["prefix_table"], s["prefix_lens"], s["table"], s["lens"],
            max_prefix=s["max_prefix"], max_len=s["max_len"], groups=s["groups"],
            max_group=case["members"], cu_seqlens=s["cu"], max_new=case["new"], scale=s["scale"],
            workspace=s["workspace"]))
    if op == "reorder":
        s["table"], s["lens"] = s["pages"].fork(s["table"], s["lens"], s["parents"])
        s["pages"].reserve(s["table"], s["lens"], case["new"], caches=s["handles"],
                           workspace=s["workspace"])
        return [s["table"], s["lens"], s["refs"]] + _cache_values(s)
    if op == "compact":
        table, refs = s["table0"].clone(), s["refs0"].clone()
        used, moved = kvx.Pages(refs, case["block"]).compact([table], s["handles"],
                                                             workspace=s["workspace"])
        return [table, refs, used, moved] + _cache_values(s)
    return list(kvx.beam_select(s["logits"], s["scores"], beams=case["out"],
                                eos=2 if case["ended"] else None, done=s["done"],
                                workspace=s["workspace"]))


def _cache_values(s):
    """The caches' own buffers: the codes as the 8-bit numbers they are, and the scales."""
    return [x.view(torch.float8_e4m3fn) if x.dtype == torch.uint8 else x
            for layer in s["caches"] for x in layer]


def _gather(codes, scale, table):
    """A padded batch of a paged cache's values, fp32 [R][H][slots][d]."""
    t = table.long().clamp(min=0)
    x = codes[t].view(torch.float8_e4m3fn).float() * scale[t][..., None, None]
    R, P, H, bs, d = x.shape
    return x.permute(0, 2, 1, 3, 4).reshape(R, H, P * bs, d)


def _shared(s):
    case = s["case"]
    P, M, new, H, Hq, d = (case[k] for k in ("prefixes", "members", "new", "kv_heads", "q_heads",
                                            "head_dim"))
    G, R, lens = Hq // H, P * M, s["lens"].long()
    q = s["q"].float() * s["scale"]
    # the requests' own slots
    k = _gather(s["k_codes"], s["k_scale"], s["table"])
    qo = q.reshape(R, new, H, G, d).permute(0, 2, 3, 1, 4).reshape(R, H, G * new, d)
    xo = (qo @ k.transpose(-1, -2)).reshape(R, H, G, new, -1)
    j, i = torch.arange(xo.shape[-1], device=DEV), torch.arange(new, device=DEV)
    seen = j[None, None] <= (lens[:, None] - new + i)[:, :, None]
    xo = xo.masked_fill_(~seen[:, None, None], float("-inf"))
    v = _gather(s["v_codes"], s["v_scale"], s["table"])
    v = v.masked_fill_((j[None] >= lens[:, None])[:, None, :, None], 0.0)
    top = xo.amax(-1)
    # the prefixes, each against all of its requests' queries at once
    out = torch.empty((P, M, H, G, new, d), device=DEV)
    lse = torch.empty((P, M, H, G, new), device=DEV)
    xo = xo.reshape(P, M, H, G, new, -1)
    v = v.reshape(P, M, H, -1, d)
    top = top.reshape(P, M, H, G, new)
    for p, n in enumerate(_prefix_lengths(case)):
        table = s["prefix_table"][p:p + 1, :-(-n // case["block"])]
        kp = _gather(s["k_codes"], s["k_scale"], table)[0, :, :n]
        qp = q.reshape(P, M, new, H, G, d)[p].permute(2, 0, 3, 1, 4).reshape(H, M * G * new, d)
        x = qp @ kp.transpose(-1, -2)
        del kp
        t = torch.maximum(x.amax(-1).reshape(H, M, G, new).transpose(0, 1), top[p])
        rows = t.transpose(0, 1).reshape(H, M * G * new, 1)
        x = x.sub_(rows).exp_()
        vp = _gather(s["v_codes"], s["v_scale"], table)[0, :, :n]
        o = (x @ vp).reshape(H, M, G, new, d).transpose(0, 1)
        total = x.sum(-1).reshape(H, M, G, new).transpose(0, 1)
        po = (xo[p] - t[..., None]).exp()
        o = o + (po.reshape(M, H, G * new, -1) @ v[p]).reshape(M, H, G, new, d)
        total = total + po.sum(-1)
        out[p] = o / total[..., None]
        lse[p] = t + total.log()
        del x, vp
    out = out.permute(0, 1, 4, 2, 3, 5).reshape(R * new, Hq, d).to(s["q"].dtype)
    return [out, lse.permute(0, 1, 4, 2, 3).reshape(R * new, Hq).contiguous()]


def _reorder(s):
    case = s["case"]
    bs, new, refs = case["block"], case["new"], s["refs"]
    parents, old, blocks = s["parents"].long(), s["table"], case["blocks"]
    lens, W = s["lens"][parents], old.shape[1]
    # fork: rows hold their parents' pages
    held = torch.arange(W, device=DEV) < ((lens + bs - 1) // bs)[:, None]
    table = torch.where(held, old[parents], torch.full_like(old, -1))
    one = lambda t: torch.where(t >= 0, 1, 0).to(torch.int32).reshape(-1)
    refs.index_add_(0, table.long().clamp(min=0).reshape(-1), one(table))
    refs.index_add_(0, old.long().clamp(min=0).reshape(-1), -one(old))
    # reserve: pages that the next tokens are written to, a row's own
    n = table.shape[0]
    row = torch.arange(n, device=DEV)[:, None]
    first, last = lens.long() // bs, (lens.long() + new - 1) // bs
    col = first[:, None] + torch.arange(-(-new // bs) + 1, device=DEV)
    asked = col <= last[:, None]
    col = col.clamp(max=W - 1)
    page = table.gather(1, col)
    at = page.long().clamp(min=0)
    shared = asked & (page >= 0) & (refs[at] > 1)
    users = torch.zeros_like(refs).index_add_(0, at.reshape(-1), shared.to(torch.int32).reshape(-1))
    mark = torch.where(shared, row.expand_as(at), torch.full_like(at, -1)).to(torch.int32)
    latest = torch.full_like(refs, -1).scatter_reduce_(0, at.reshape(-1), mark.reshape(-1), "amax")
    stays = shared & (refs[at] == users[at]) & (latest[at] == row)
    need = asked & ((page < 0) | (shared & ~stays))
    rank = need.reshape(-1).long().cumsum(0).reshape(need.shape) - 1
    free = torch.argsort((refs != 0).to(torch.int8), stable=True)
    fresh = free[rank.clamp(min=0)]
    table.scatter_reduce_(1, col, torch.where(need, fresh, torch.full_like(fresh, -1)).to(torch.int32),
                          "amax")
    moved = need & (page >= 0)
    table.scatter_(1, col[:, :1], torch.where(need, fresh, page.long())[:, :1].to(torch.int32))
    refs.index_add_(0, at.reshape(-1), -moved.to(torch.int32).reshape(-1))
    refs.index_add_(0, fresh.reshape(-1), need.to(torch.int32).reshape(-1))
    # copies of pages that hold tokens and were shared; the others copy onto themselves
    copy = moved[:, 0] & (lens % bs > 0)
    src = torch.where(page < 0, fresh, at)[:, 0]
    dst = torch.where(copy, fresh[:, 0], src)
    for layer in s["caches"]:
        for x in layer:
            x[dst] = x[src]
    s["table"], s["lens"] = table, lens
    return [table, lens, refs] + _cache_values(s)


def _compact(s):
    blocks = s["case"]["blocks"]
    refs = s["refs0"].clone()
    held = refs != 0
    used = held.sum()
    b = torch.arange(blocks, device=DEV)
    hole, mover = ~held & (b < used), held & (b >= used)
    # the i-th page to move goes to the i-th hole
    src, dst = torch.nonzero(mover)[:, 0], torch.nonzero(hole)[:, 0]
    moved = torch.where(held, b, torch.full_like(b, -1))
    moved[src] = dst
    old = s["table0"].long()
    table = torch.where(old >= 0, moved[old.clamp(min=0)], old).to(torch.int32)
    fresh = torch.zeros_like(refs).index_add_(0, moved.clamp(min=0), refs)
    for layer in s["caches"]:
        for x in layer:
            x[dst] = x[src]
    return [table, fresh, used.to(torch.int32).reshape(1), moved.to(torch.int32)] + _cache_values(s)


def _beam(s):
    case = s["case"]
    R, K, V, N = (case[k] for k in ("requests", "beams", "vocab", "out"))
    # scores are ranked: in 64 bits, so that neighbours do not change places
    x = s["logits"].double()
    top = x.amax(-1, keepdim=True)
    x = x - (top + (x - top).exp().sum(-1, keepdim=True).log()) + s["scores"].double().reshape(-1, 1)
    if s["done"] is not None:
        over = s["done"].reshape(-1, 1)
        x = torch.where(over, torch.full_like(x, float("-inf")), x)
        x[:, 2:3] = torch.where(over, s["scores"].double().reshape(-1, 1), x[:, 2:3])
    x = x.reshape(R, K * V)
    M = min(N, K * V)
    best, at = x.topk(M, -1)
    least = best[:, -1:]
    # of those equal to the least the lowest places, which topk does not promise
    place = torch.arange(K * V, device=DEV)
    equal = torch.where(x == least, place, torch.full_like(place, K * V)).topk(M, -1, largest=False)[0]
    at = torch.cat([torch.where(best > least, at, torch.full_like(at, K * V)), equal], 1).sort(1)[0]
    got = torch.where(at < K * V, x.gather(1, at.clamp(max=K * V - 1)),
                      torch.full((), float("-inf"), dtype=x.dtype, device=DEV))
    got, order = got.sort(dim=-1, descending=True, stable=True)
    at = at.gather(1, order)[:, :M]
    got = got[:, :M]
    if M < N:
        got = torch.nn.functional.pad(got, (0, N - M), value=float("-inf"))
        at = torch.nn.functional.pad(at, (0, N - M))
    there = got > float("-inf")
    none = torch.full_like(at, -1)
    tokens = torch.where(there, at % V, none)
    parents = torch.where(there, at // V + K * torch.arange(R, device=DEV)[:, None], none)
    done = None
    if s["done"] is not None:
        done = (tokens == 2) & there
    return [tokens.to(torch.int32), parents.to(torch.int32), got.float(), done]


# --- what a pass cannot do without -----------------------------------------------

def work(case):
    op = case["op"]
    if op == "shared":
        new, Hq, H, d, bs = (case[k] for k in ("new", "q_heads", "kv_heads", "head_dim", "block"))
        before, lens = _prefix_lengths(case), _own_lengths(case)
        slots = sum(before) + sum(lens)
        pages = sum(-(-n // bs) for n in before + lens)
        pairs = sum(n * case["members"] * new for n in before) + \
            sum(new * n - new * (new - 1) // 2 for n in lens)
        rows = len(lens) * new * Hq
        size = 4 if case["dtype"] == "f32" else 2
        return {"bytes": slots * H * 2 * d + 8 * H * pages + rows * (2 * d * size + 4),
                "flops": 4 * Hq * d * pairs}
    if op == "beam":
        rows = case["requests"] * case["beams"]
        n = rows * case["vocab"]
        return {"bytes": n * (4 if case["dtype"] == "f32" else 2) + 4 * rows
                + 13 * case["requests"] * case["out"], "flops": 4 * n}
    page = 2 * case["heads"] * (case["block"] * case["head_dim"] + 4) * case["layers"]
    if op == "reorder":
        R, K, bs, hi = (case[k] for k in ("requests", "beams", "block", "longest"))
        rows = R * K
        width = -(-(hi + case["new"]) // bs)
        # of a request's beams about 0.37 have no child; as many rows need a copy of a last page
        copies = int(R * K * (1 - 1 / K) ** K) if K > 1 else 0
        return {"bytes": 8 * rows * width + 4 * case["blocks"] + 16 * rows + 2 * copies * page,
                "flops": rows * width}
    used = int(case["blocks"] * case["held"])
    moves = int(used * (1 - case["held"]))
    entries = case["rows"] * -(-case["longest"] // case["block"])
    return {"bytes": 12 * case["blocks"] + 8 * entries + 2 * moves * page,
            "flops": case["blocks"] + entries}


# --- the definition in 64 bits ------------------------------------------------------

def exact(case, seed):
    global own
    if case["op"] in ("reorder", "compact") and 2 * case["blocks"] * case["layers"] * case["heads"] * \
            case["block"] * case["head_dim"] > 3e8:
        return None
    was, own = own, False
    try:
        s = prepare(case, seed)
    finally:
        own = was
    return {"shared": _exact_shared, "beam": _exact_beam, "reorder": _exact_reorder,
            "compact": _exact_compact}[case["op"]](s)


def _exact_shared(s):
    """Each request alone: its prefix and its own slots as one sequence."""
    case = s["case"]
    bs, new, H, Hq, d, M = (case[k] for k in ("block", "new", "kv_heads", "q_heads", "head_dim",
                                             "members"))
    before, lens = s["prefix_lens"].tolist(), s["lens"].tolist()
    R = len(lens)
    if sum(before) * M * new * Hq > 2e9:
        return None
    G = Hq // H
    out = torch.zeros((R * new, Hq, d), dtype=torch.float64, device=DEV)
    lse = torch.zeros((R * new, Hq), dtype=torch.float64, device=DEV)

    def values(m, table, n, h):
        ids = table[:-(-n // bs)].long()
        x = s[m + "_codes"][ids, h].view(torch.float8_e4m3fn).double()
        return (x * s[m + "_scale"][ids, h].double()[:, None, None]).reshape(-1, d)[:n]

    for p, n in enumerate(before):
        for h in range(H):
            kp, vp = (values(m, s["prefix_table"][p], n, h) for m in "kv")
            for r in range(p * M, (p + 1) * M):
                k, v = (torch.cat([x, values(m, s["table"][r], lens[r], h)])
                        for x, m in ((kp, "k"), (vp, "v")))
                q = s["q"][r * new:(r + 1) * new, h * G:(h + 1) * G].double()
                x = torch.einsum("igd,jd->igj", q, k) * s["scale"]
                last = n + lens[r] - new + torch.arange(new, device=DEV)
                x.masked_fill_(torch.arange(n + lens[r], device=DEV)[None, None] > last[:, None, None],
                               -math.inf)
                total = torch.logsumexp(x, -1)
                out[r * new:(r + 1) * new, h * G:(h + 1) * G] = torch.exp(x - total[..., None]) @ v
                lse[r * new:(r + 1) * new, h * G:(h + 1) * G] = total
    return [out, lse]


def _exact_pages(s, moves):
    """The caches' values after the pages' moves (source, destination)."""
    src, dst = (torch.tensor([m[i] for m in moves], dtype=torch.long, device=DEV) for i in (0, 1))
    got = []
    for layer in s["caches"]:
        for x in layer:
            y = (x.view(torch.float8_e4m3fn) if x.dtype == torch.uint8 else x).double()
            y[dst] = y[src]
            got.append(y)
    return got


def _exact_reorder(s):
    """Row after row, page after page."""
    case = s["case"]
    bs, new = case["block"], case["new"]
    old, lens, refs = s["table"].tolist(), s["lens"].tolist(), s["refs"].tolist()
    parents = s["parents"].tolist()
    rows = [old[p][:-(-lens[p] // bs)] for p in parents]
    rows = [row + [-1] * (len(old[0]) - len(row)) for row in rows]
    for table, by in ((rows, 1), (old, -1)):
        for row in table:
            for page in row:
                if page >= 0:
                    refs[page] += by
    free = iter([b for b, n in enumerate(refs) if n == 0])
    moves = []
    for row, p in zip(rows, parents):
        n = lens[p]
        for b in range(n // bs, (n + new - 1) // bs + 1):
            page = row[b]
            if page >= 0 and refs[page] == 1:
                continue
            row[b] = next(free)
            refs[row[b]] = 1
            if page >= 0:
                refs[page] -= 1
                if b * bs < n:
                    moves.append((page, row[b]))
    return [None, None, None] + _exact_pages(s, moves)


def _exact_compact(s):
    refs = s["refs0"].tolist()
    used = sum(n != 0 for n in refs)
    holes = [b for b in range(used) if refs[b] == 0]
    movers = [b for b in range(used, len(refs)) if refs[b] != 0]
    return [None, None, None, None] + _exact_pages(s, list(zip(movers, holes)))


def _exact_beam(s):
    case = s["case"]
    R, K, V, N = (case[k] for k in ("requests", "beams", "vocab", "out"))
    best = torch.full((R, N), -math.inf, dtype=torch.float64, device=DEV)
    for r in range(R):
        got = []
        for k in range(K):
            if s["done"] is not None and bool(s["done"][r, k]):
                got.append(s["scores"][r, k:k + 1].double())
                continue
            x = torch.log_softmax(s["logits"][r * K + k].double(), -1) + s["scores"][r, k].double()
            got.append(x.sort(descending=True)[0][:N])
        got = torch.cat(got).sort(descending=True)[0][:N]
        best[r, :got.numel()] = got
    return [None, None, best, None]
