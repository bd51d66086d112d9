"""Measured cases of the operators with which a target model decodes on a
transferred cache: rotary positions, the 8-bit paged cache's write, attention
over that cache, and eviction by accumulated attention weight.

``run`` computes each operator either in plain torch operations in fp32
(``own`` false) or through the library's entry points (``own`` true);
``exact`` computes it in fp64, written apart from both.

The 8-bit cache: e4m3 codes [blocks][H][block][d], one fp32 scale for each
(block, head) of the keys and of the values.  The writer's scales are powers
of two, the smallest with amax / scale <= 448 and at least 2^-126.
"""
import math

import torch

own = False

DEV = "cuda"
DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16}


def listed():
    return [
        # one new token for each of 16 running requests: queries and keys of one layer, latency
        dict(name="rope_step", op="rope", tokens=16, q_heads=64, k_heads=8, head_dim=128,
             rot_dim=128, layout="half", scaling="none", theta=1e6, dtype="bf16",
             transpose=False, fused=True, far=16384),
        # a prompt's queries and keys, views of one fused projection, frequencies
        # scaled by wavelength bands for a long context
        dict(name="rope_prompt", op="rope", tokens=32768, q_heads=64, k_heads=8, head_dim=128,
             rot_dim=128, layout="half", scaling="bands", theta=5e5, dtype="bf16",
             transpose=False, fused=True, far=131072),
        # the gradient of a partial, interleaved rotation in fp32, an odd length
        dict(name="rope_grad", op="rope", tokens=2047, q_heads=16, k_heads=8, head_dim=128,
             rot_dim=64, layout="interleaved", scaling="yarn", theta=1e4, dtype="f32",
             transpose=True, fused=False, far=32768),
        # one token appended for each of 16 requests, mostly into started blocks
        dict(name="write_step", op="write", requests=16, shortest=1, longest=1, filled=4111,
             heads=8, head_dim=128, block=16, dtype="bf16"),
        # 16 ragged transferred prompts quantised into a paged cache, one layer
        dict(name="write_prompts", op="write", requests=16, shortest=1024, longest=16384,
             filled=0, heads=8, head_dim=128, block=16, dtype="bf16"),
        # a short conversation of a small model in fp32: one token, latency
        dict(name="attend_one", op="attend", requests=1, shortest=512, longest=512, new=1,
             q_heads=4, kv_heads=2, head_dim=64, block=16, dtype="f32", weights=False),
        # one decoding step of a ragged batch that also keeps score for the eviction
        dict(name="attend_step", op="attend", requests=16, shortest=1024, longest=16384, new=1,
             q_heads=64, kv_heads=8, head_dim=128, block=16, dtype="bf16", weights=True),
        # one decoding step of a single long request: few rows, a long axis
        dict(name="attend_long", op="attend", requests=1, shortest=131071, longest=131071, new=1,
             q_heads=64, kv_heads=8, head_dim=128, block=64, dtype="bf16", weights=False),
        # the last tokens of a prompt vote on what the cache keeps
        dict(name="attend_window", op="attend", requests=2, shortest=8191, longest=8192, new=61,
             q_heads=32, kv_heads=8, head_dim=128, block=16, dtype="bf16", weights=True),
        # a whole prompt attends to itself
        dict(name="attend_prompt", op="attend", requests=1, shortest=8192, longest=8192, new=8192,
             q_heads=64, kv_heads=8, head_dim=128, block=16, dtype="bf16", weights=False),
        # one request over its budget
        dict(name="evict_one", op="evict", requests=1, shortest=2048, longest=2048, keep=512,
             sinks=4, recent=64, heads=8, head_dim=128, block=16),
        # a ragged batch brought under one budget after its prompts
        dict(name="evict_batch", op="evict", requests=16, shortest=1024, longest=16384, keep=4096,
             sinks=4, recent=512, heads=8, head_dim=128, block=16),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rope", "write", "attend", "attend", "evict"])
    if op == "rope":
        hk = rng.choice([1, 2, 4, 8])
        d = rng.choice([64, 80, 96, 128, 256])
        return dict(op="rope", tokens=_log(rng, 1, 16384), q_heads=hk * rng.choice([1, 2, 4, 5, 8]),
                    k_heads=hk, head_dim=d, rot_dim=rng.choice([d, d // 2]),
                    layout=rng.choice(["half", "interleaved"]),
                    scaling=rng.choice(["none", "linear", "bands", "yarn"]),
                    theta=rng.choice([1e4, 5e5, 1e6]), dtype=rng.choice(["bf16", "f32"]),
                    transpose=rng.random() < 0.3, fused=rng.random() < 0.5,
                    far=_log(rng, 1024, 131072))
    heads, d = rng.choice([1, 2, 4, 8]), rng.choice([64, 128])
    block = rng.choice([8, 16, 24, 32, 64, 128])
    if op == "write":
        R = _log(rng, 1, 64)
        hi = _log(rng, 1, max(1, 131072 // R))
        return dict(op="write", requests=R, shortest=rng.randint(1, hi), longest=hi,
                    filled=rng.choice([0, rng.randint(1, 300)]), heads=heads, head_dim=d,
                    block=block, dtype=rng.choice(["bf16", "f32"]))
    if op == "attend":
        dtype = rng.choice(["bf16", "bf16", "f32"])
        G = rng.choice([1, 2, 4, 5, 8])
        if rng.random() < 0.6:
            R = _log(rng, 1, 64)
            hi = _log(rng, 16, max(16, 131072 // R))
            new = rng.choice([1, 1, 1, 2, 5])
        else:
            R = _log(rng, 1, 4)
            hi = _log(rng, 64, 4096)
            new = _log(rng, 8, hi)
        lo = rng.randint(min(hi, new), hi)
        return dict(op="attend", requests=R, shortest=max(lo, new), longest=max(hi, new), new=new,
                    q_heads=heads * G, kv_heads=heads, head_dim=d, block=block, dtype=dtype,
                    weights=rng.random() < 0.4)
    R = _log(rng, 1, 32)
    hi = _log(rng, 64, max(64, 131072 // R))
    keep = rng.randint(max(2, hi // 16), max(2, hi // 2))
    recent = rng.randint(0, keep // 4)
    return dict(op="evict", requests=R, shortest=rng.randint(hi // 2, hi), longest=hi, keep=keep,
                sinks=min(4, keep - recent), recent=recent, heads=heads, head_dim=d, block=block)


# --- what a program has in hand ----------------------------------------------

def _lengths(case):
    """The requests' lengths, spread evenly between the shortest and the longest."""
    R, lo, hi = case["requests"], case["shortest"], case["longest"]
    return [hi if R == 1 else lo + (hi - lo) * r // (R - 1) for r in range(R)]


def _ints(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def _table(pages, g, extra=0):
    """A block table over a shuffled pool, [R][most], and the pool's size."""
    R, most = len(pages), max(1, max(pages))
    total = sum(pages) + extra + 1
    order = torch.randperm(total, generator=g, device=DEV).to(torch.int32)
    table = torch.zeros((R, most), dtype=torch.int32, device=DEV)
    at = 0
    for r, n in enumerate(pages):
        table[r, :n] = order[at:at + n]
        at += n
    return table, total, order[at:]


def _channel_scale(H, d, g):
    return torch.exp(0.5 * torch.randn((H, 1, d), generator=g, device=DEV))


def _filled_cache(blocks, H, bs, d, g):
    """Codes and scales of a cache that earlier writes filled."""
    x = torch.randn((blocks, H, bs, d), generator=g, device=DEV) * _channel_scale(H, d, g)
    scale = _scale_of(x.abs().amax((2, 3)))
    return _encode(x, scale[:, :, None, None]), scale


def prepare(case, seed):
    g = _gen(seed)
    s = {"case": case}
    op = case["op"]
    if op == "rope":
        n, hq, hk, d = (case[k] for k in ("tokens", "q_heads", "k_heads", "head_dim"))
        dt = DTYPES[case["dtype"]]
        heads = hq + 2 * hk if case["fused"] else hq + hk
        x = torch.randn((n, heads, d), generator=g, device=DEV).to(dt)
        s["q"], s["k"] = x[:, :hq], x[:, hq:hq + hk]
        s["positions"] = torch.randint(0, case["far"], (n,), generator=g, device=DEV,
                                       dtype=torch.int32)
        # the model's table of angles, made once in fp64
        w, amp = _frequencies(case)
        ang = torch.arange(case["far"], dtype=torch.float64, device=DEV)[:, None] * w
        s["cos"], s["sin"] = (torch.cos(ang) * amp).float(), (torch.sin(ang) * amp).float()
    elif op == "write":
        H, d, bs, dt = case["heads"], case["head_dim"], case["block"], DTYPES[case["dtype"]]
        lens = _lengths(case)
        start = [0 if not case["filled"] else (case["filled"] + 7 * r) % (case["filled"] + 1)
                 for r in range(len(lens))]
        pages = [-(-(a + n) // bs) for a, n in zip(start, lens)]
        s["table"], blocks, _ = _table(pages, g)
        cu = [0]
        for n in lens:
            cu.append(cu[-1] + n)
        s["cu"], s["start"], s["ntok"] = _ints(cu), _ints(start), cu[-1]
        for m in "kv":
            s[m + "_codes"], s[m + "_scale"] = _filled_cache(blocks, H, bs, d, g)
            s[m] = (torch.randn((cu[-1], H, d), generator=g, device=DEV)
                    * _channel_scale(H, d, g).reshape(H, d)).to(dt)
    elif op == "attend":
        H, Hq, d, bs = case["kv_heads"], case["q_heads"], case["head_dim"], case["block"]
        R, new, dt = case["requests"], case["new"], DTYPES[case["dtype"]]
        lens = _lengths(case)
        s["table"], blocks, _ = _table([-(-n // bs) for n in lens], g)
        s["lens"], s["max_len"] = _ints(lens), max(lens)
        s["cu"] = _ints([new * r for r in range(R + 1)])
        for m in "kv":
            s[m + "_codes"], s[m + "_scale"] = _filled_cache(blocks, H, bs, d, g)
        s["q"] = (1.5 * torch.randn((R * new, Hq, d), generator=g, device=DEV)).to(dt)
        s["scale"] = 1.0 / math.sqrt(d)
        s["weights"] = torch.zeros((R, H, s["table"].shape[1] * bs), device=DEV) \
            if case["weights"] else None
    else:
        H, d, bs, keep = case["heads"], case["head_dim"], case["block"], case["keep"]
        lens = _lengths(case)
        R = case["requests"]
        dst = [-(-min(n, keep) // bs) for n in lens]
        s["table"], blocks, rest = _table([-(-n // bs) for n in lens], g, extra=R * max(dst))
        s["dst_table"] = rest[:R * max(dst)].reshape(R, max(dst)).contiguous()
        s["lens"], s["max_len"] = _ints(lens), max(lens)
        for m in "kv":
            s[m + "_codes"], s[m + "_scale"] = _filled_cache(blocks, H, bs, d, g)
        # accumulated attention weight: a few slots hold most of it
        s["weights"] = torch.exp(2.0 * torch.randn((R, H, s["table"].shape[1] * bs), generator=g,
                                                   device=DEV))
    if own:
        _handles(s)
    return s


def _handles(s):
    """The library's objects that a program keeps beside its tensors."""
    from cross_model_kv_transfer_gb300 import kvx
    case = s["case"]
    if case["op"] == "rope":
        s["rope"] = kvx.Rope(case["head_dim"], case["theta"], rot_dim=case["rot_dim"],
                             layout=case["layout"], **_scaling(case))
        return
    s["cache"] = kvx.Cache8(s["k_codes"], s["v_codes"], s["k_scale"], s["v_scale"])
    if case["op"] == "attend":
        s["workspace"] = s["cache"].attend_workspace(
            ntok=s["q"].shape[0], num_requests=case["requests"], q_heads=case["q_heads"],
            max_len=s["max_len"], max_new=case["new"], dtype=s["q"].dtype,
            weights=case["weights"])
    elif case["op"] == "evict":
        s["workspace"] = s["cache"].evict_workspace(num_requests=case["requests"],
                                                    max_len=s["max_len"], keep=case["keep"])


# --- the operators --------------------------------------------------------------

def run(state):
    if own:
        return _run_own(state)
    return {"rope": _rope, "write": _write, "attend": _attend, "evict": _evict}[
        state["case"]["op"]](state)


def _run_own(s):
    case = s["case"]
    op = case["op"]
    if op == "rope":
        return s["rope"].apply(s["q"], s["k"], s["positions"], transpose=case["transpose"])
    c = s["cache"]
    if op == "write":
        c.write(s["k"], s["v"], s["table"], s["start"], cu_seqlens=s["cu"])
        return _cache_values(s)
    if op == "attend":
        out, lse = c.attend(s["q"], s["table"], s["lens"], s["max_len"], cu_seqlens=s["cu"],
                            max_new=case["new"], scale=s["scale"], weights=s["weights"],
                            workspace=s["workspace"])
        return [out, lse, s["weights"]]
    kept, kept_weights, new_lens = c.evict(
        s["weights"], s["table"], s["lens"], s["dst_table"], max_len=s["max_len"],
        keep=case["keep"], sinks=case["sinks"], recent=case["recent"], workspace=s["workspace"])
    return [kept, kept_weights, new_lens] + _cache_values(s)


def _cache_values(s):
    """The cache's own buffers: the codes as the 8-bit numbers they are, and the scales."""
    return [s["k_codes"].view(torch.float8_e4m3fn), s["v_codes"].view(torch.float8_e4m3fn),
            s["k_scale"], s["v_scale"]]


def _scaling(case):
    """A model's settings for contexts longer than the one it was trained on."""
    return {"none": {}, "linear": dict(scaling="linear", factor=4.0),
            "bands": dict(scaling="bands", factor=8.0, low_band=1.0, high_band=4.0,
                          original_context=8192),
            "yarn": dict(scaling="yarn", factor=4.0, beta_fast=32.0, beta_slow=1.0,
                         original_context=8192)}[case["scaling"]]


def _frequencies(case):
    """Radians a position for each pair, fp64, and the amplitude of the rotation."""
    rot, theta = case["rot_dim"], case["theta"]
    i = torch.arange(rot // 2, dtype=torch.float64, device=DEV)
    w = theta ** (-2.0 * i / rot)
    p = _scaling(case)
    if not p:
        return w, 1.0
    f = p["factor"]
    if p["scaling"] == "linear":
        return w / f, 1.0
    turns = p["original_context"] * w / (2 * math.pi)
    if p["scaling"] == "bands":
        # turns in the original context: few are stretched, many are kept
        keep = ((turns - p["low_band"]) / (p["high_band"] - p["low_band"])).clamp(0, 1)
        return w * (keep + (1 - keep) / f), 1.0
    pair = lambda beta: rot * math.log(p["original_context"] / (beta * 2 * math.pi)) / (
        2 * math.log(theta))
    lo = max(math.floor(pair(p["beta_fast"])), 0)
    hi = min(math.ceil(pair(p["beta_slow"])), rot - 1)
    keep = 1 - ((i - lo) / max(hi - lo, 0.001)).clamp(0, 1)
    return w * (keep + (1 - keep) / f), 0.1 * math.log(f) + 1.0


def _turn(x, c, s, case):
    rot, half = case["rot_dim"], case["rot_dim"] // 2
    x32 = x.float()
    r = x32[..., :rot]
    if case["layout"] == "half":
        a, b = r[..., :half], r[..., half:]
    else:
        a, b = r[..., 0::2], r[..., 1::2]
    u, v = a * c - b * s, b * c + a * s
    y = torch.cat([u, v], -1) if case["layout"] == "half" else torch.stack([u, v], -1).flatten(-2)
    return torch.cat([y, x32[..., rot:]], -1).to(x.dtype)


def _rope(s):
    case, p = s["case"], s["positions"].long()
    c, sn = s["cos"][p][:, None], s["sin"][p][:, None]
    if case["transpose"]:
        sn = -sn
    return _turn(s["q"], c, sn, case), _turn(s["k"], c, sn, case)


def _scale_of(amax):
    """The smallest power of two (at least 2^-126) that brings amax to 448 or less."""
    m, e = torch.frexp(amax)
    e = torch.where(amax > 0, (e - 9 + (m > 0.875).to(e.dtype)).clamp(min=-126),
                    torch.full_like(e, -126))
    return torch.ldexp(torch.ones_like(amax), e)


def _encode(x, scale):
    return (x * (1.0 / scale)).clamp(-448.0, 448.0).to(torch.float8_e4m3fn).view(torch.uint8)


def _decode(codes):
    return codes.view(torch.float8_e4m3fn).float()


def _write(s):
    case, bs = s["case"], s["case"]["block"]
    cu, start, table = s["cu"].long(), s["start"].long(), s["table"].long()
    n, R = s["ntok"], case["requests"]
    r = torch.repeat_interleave(torch.arange(R, device=DEV), cu[1:] - cu[:-1], output_size=n)
    slot = start[r] + torch.arange(n, device=DEV) - cu[r]
    page, off = table[r, slot // bs], slot % bs
    head = start % bs                        # slots of the first block that stay
    first = table[torch.arange(R, device=DEV), start // bs]
    where = (page, off, first, head)
    return [_write_one(s["k"], s["k_codes"], s["k_scale"], *where),
            _write_one(s["v"], s["v_codes"], s["v_scale"], *where), s["k_scale"], s["v_scale"]]


def _write_one(x, codes, scale, page, off, first, head):
    x = x.float()
    H, bs = codes.shape[1], codes.shape[2]
    most = torch.zeros_like(scale).scatter_reduce_(
        0, page[:, None].expand(-1, H), x.abs().amax(-1), "amax")
    touched = torch.zeros(scale.shape[0], dtype=torch.bool, device=DEV)
    touched[page] = True
    need = _scale_of(most)
    old = scale[first]
    grown = torch.where((head > 0)[:, None], torch.maximum(old, need[first]), need[first])
    new = torch.where(touched[:, None], need, scale)
    new[first] = grown
    before = codes[first]
    again = _encode(_decode(before), (grown / old)[:, :, None, None])
    stay = torch.arange(bs, device=DEV)[None, :] < head[:, None]
    codes[first] = torch.where(stay[:, None, :, None], again, before)
    codes[page, :, off] = _encode(x, new[page][:, :, None])
    scale.copy_(new)
    return codes.view(torch.float8_e4m3fn)


def _gather(codes, scale, table):
    """A padded batch of a paged cache's values, fp32 [R][H][slots][d]."""
    x = _decode(codes[table]) * scale[table][..., None, None]
    R, P, H, bs, d = x.shape
    return x.permute(0, 2, 1, 3, 4).reshape(R, H, P * bs, d)


def _attend(s):
    case = s["case"]
    R, new, H, Hq, d = (case[k] for k in ("requests", "new", "kv_heads", "q_heads", "head_dim"))
    G, table, lens = Hq // H, s["table"].long(), s["lens"].long()
    k = _gather(s["k_codes"], s["k_scale"], table)
    q = s["q"].float().reshape(R, new, H, G, d).permute(0, 2, 3, 1, 4).reshape(R, H, G * new, d)
    x = (q @ k.transpose(-1, -2) * s["scale"]).reshape(R, H, G, new, -1)
    del k
    j, i = torch.arange(x.shape[-1], device=DEV), torch.arange(new, device=DEV)
    seen = j[None, None] <= (lens[:, None] - new + i)[:, :, None]
    x = x.masked_fill_(~seen[:, None, None], float("-inf"))
    top = x.amax(-1, keepdim=True)
    p = x.sub_(top).exp_()
    total = p.sum(-1, keepdim=True)
    p = p.div_(total)
    v = _gather(s["v_codes"], s["v_scale"], table)
    v = v.masked_fill_((j[None] >= lens[:, None])[:, None, :, None], 0.0)
    o = (p.reshape(R, H, G * new, -1) @ v).reshape(R, H, G, new, d)
    lse = (top + total.log())[..., 0]
    if s["weights"] is not None:
        s["weights"] += p.sum((2, 3))
    out = o.permute(0, 3, 1, 2, 4).reshape(R * new, Hq, d).to(s["q"].dtype)
    return [out, lse.permute(0, 3, 1, 2).reshape(R * new, Hq).contiguous(), s["weights"]]


def _evict(s):
    case = s["case"]
    keep, sinks, recent, bs = (case[k] for k in ("keep", "sinks", "recent", "block"))
    lens, table, dst = s["lens"].long()[:, None, None], s["table"].long(), s["dst_table"].long()
    w = s["weights"]
    R, H, cap = w.shape
    j = torch.arange(cap, device=DEV)
    held = (j < sinks) | (j >= lens - recent)
    w_or = torch.where(held, torch.full_like(w, float("inf")), w)
    w_or = torch.where(j < lens, w_or, torch.full_like(w, float("-inf")))
    kept = torch.sort(w_or, dim=-1, descending=True, stable=True)[1][..., :keep]
    kept = torch.where(kept < lens, kept, torch.full_like(kept, cap)).sort(-1)[0]
    there = kept < cap
    at = kept.clamp(max=cap - 1)
    if kept.shape[-1] < keep:                # a budget beyond the table's width
        pad = keep - kept.shape[-1]
        at, there = (torch.nn.functional.pad(t, (0, pad)) for t in (at, there))
    kept_weights = torch.where(there, w.gather(-1, at), torch.zeros((), device=DEV))
    slots = dst.shape[1] * bs
    fill = max(0, slots - keep)
    src = torch.nn.functional.pad(at, (0, fill))[..., :slots]
    live = torch.nn.functional.pad(there, (0, fill))[..., :slots]
    page = table[torch.arange(R, device=DEV)[:, None, None], src // bs]
    head = torch.arange(H, device=DEV)[None, :, None]
    new_lens = torch.minimum(lens[:, 0, 0], torch.full_like(lens[:, 0, 0], keep)).to(torch.int32)
    for_k = _evict_one(s["k_codes"], s["k_scale"], page, head, src % bs, live, dst)
    for_v = _evict_one(s["v_codes"], s["v_scale"], page, head, src % bs, live, dst)
    return [torch.where(there, at, torch.full_like(at, -1)).to(torch.int32), kept_weights,
            new_lens, for_k, for_v, s["k_scale"], s["v_scale"]]


def _evict_one(codes, scale, page, head, off, live, dst):
    H, bs, d = codes.shape[1:]
    R, P = dst.shape
    x = _decode(codes[page, head, off]) * scale[page, head][..., None]
    x = torch.where(live[..., None], x, torch.zeros((), device=DEV)).reshape(R, H, P, bs, d)
    live = live.reshape(R, H, P, bs).transpose(1, 2)
    x = x.transpose(1, 2)
    new = _scale_of(x.abs().amax((3, 4)))
    got = _encode(x, new[..., None, None])
    codes[dst] = torch.where(live[..., None], got, codes[dst])
    scale[dst] = torch.where(live.any(-1), new, scale[dst])
    return codes.view(torch.float8_e4m3fn)


# --- what a pass cannot do without -----------------------------------------------

def work(case):
    op, size = case["op"], {"f32": 4, "bf16": 2}.get(case.get("dtype"), 1)
    d = case["head_dim"]
    if op == "rope":
        rows = case["tokens"] * (case["q_heads"] + case["k_heads"])
        return {"bytes": 2 * rows * d * size + 4 * case["tokens"], "flops": 3 * rows * case["rot_dim"]}
    lens, bs = _lengths(case), case["block"]
    if op == "write":
        n = 2 * sum(lens) * case["heads"] * d
        return {"bytes": n * (size + 1) + 8 * sum(-(-x // bs) for x in lens) * case["heads"],
                "flops": 2 * n}
    H = case.get("kv_heads") or case["heads"]
    if op == "attend":
        new, Hq = case["new"], case["q_heads"]
        pairs = sum(new * n - new * (new - 1) // 2 for n in lens)
        rows = len(lens) * new * Hq
        return {"bytes": sum(lens) * H * 2 * d + 8 * H * sum(-(-x // bs) for x in lens)
                + rows * (2 * d * size + 4) + (8 * H * sum(lens) if case["weights"] else 0),
                "flops": 4 * Hq * d * pairs}
    kept = sum(min(n, case["keep"]) for n in lens) * H
    return {"bytes": 4 * H * sum(lens) + kept * (4 * d + 8), "flops": H * sum(lens) + 4 * kept * d}


# --- the definition in 64 bits ------------------------------------------------------

def exact(case, seed):
    global own
    was, own = own, False
    try:
        s = prepare(case, seed)
    finally:
        own = was
    return {"rope": _exact_rope, "write": _exact_write, "attend": _exact_attend,
            "evict": _exact_evict}[case["op"]](s)


def _exact_rope(s):
    """Each pair as a complex number times e^(+-ipw)."""
    case = s["case"]
    w, amp = _frequencies(case)
    ang = s["positions"].double()[:, None, None] * w
    z = torch.polar(torch.full_like(ang, amp), -ang if case["transpose"] else ang)
    rot = case["rot_dim"]
    got = []
    for x in (s["q"], s["k"]):
        y = x.double().clone()
        first, second = ((slice(0, rot // 2), slice(rot // 2, rot)) if case["layout"] == "half"
                         else (slice(0, rot, 2), slice(1, rot, 2)))
        t = torch.complex(y[..., first].contiguous(), y[..., second].contiguous()) * z
        y[..., first], y[..., second] = t.real, t.imag
        got.append(y)
    return tuple(got)


def _e4m3_numbers():
    """The 127 non-negative finite numbers of the 8-bit format, ascending, by its definition."""
    v = [m * 2.0 ** -9 for m in range(8)]
    v += [(8 + m) * 2.0 ** (e - 10) for e in range(1, 16) for m in range(8)]
    return torch.tensor(v[:127], dtype=torch.float64, device=DEV)


def _exact_round(x):
    """The nearest 8-bit number, ties to the even code, clamped to +-448."""
    v = _e4m3_numbers()
    a = x.abs().clamp(max=448.0).contiguous()
    mid = (v[1:] + v[:-1]) / 2
    up = torch.searchsorted(mid, a, right=False)
    tie = (up < 126) & (a == mid[up.clamp(max=125)]) & (up % 2 == 1)
    return torch.copysign(v[up + tie.to(up.dtype)], x)


def _exact_scale(amax):
    e = torch.ceil(torch.log2((amax / 448.0).clamp(min=2.0 ** -126)))
    e = torch.where(torch.exp2(e) * 448.0 < amax, e + 1, e)
    return torch.where(torch.exp2(e - 1) * 448.0 >= amax, e - 1, e).clamp(min=-126).exp2()


def _exact_write(s):
    case, bs = s["case"], s["case"]["block"]
    cu, start, table = s["cu"].tolist(), s["start"].tolist(), s["table"].tolist()
    codes_out, scale_out = [], []
    for m in "kv":
        codes = _decode(s[m + "_codes"]).double()
        scale = s[m + "_scale"].double()
        for r in range(case["requests"]):
            x = s[m][cu[r]:cu[r + 1]].double()
            a, n = start[r], x.shape[0]
            if n == 0:
                continue
            P = -(-(a + n) // bs) - a // bs
            lead = a % bs
            x = torch.nn.functional.pad(x, (0, 0, 0, 0, lead, P * bs - lead - n))
            x = x.reshape(P, bs, *x.shape[1:]).transpose(1, 2)
            ids = torch.tensor(table[r][a // bs:a // bs + P], device=DEV)
            new = _exact_scale(x.abs().amax((2, 3)))
            if lead:
                old = scale[ids[0]].clone()
                new[0] = torch.maximum(new[0], old)
                codes[ids[0], :, :lead] = _exact_round(
                    codes[ids[0], :, :lead] * (old / new[0])[:, None, None])
            y = _exact_round(x / new[:, :, None, None])
            slot = torch.arange(P * bs, device=DEV).reshape(P, 1, bs, 1)
            codes[ids] = torch.where((slot >= lead) & (slot < lead + n), y, codes[ids])
            scale[ids] = new
        codes_out.append(codes)
        scale_out.append(scale)
    return codes_out + scale_out


def _exact_attend(s):
    case = s["case"]
    bs, new, H, Hq, d = (case[k] for k in ("block", "new", "kv_heads", "q_heads", "head_dim"))
    pairs = case["requests"] * new * Hq * case["longest"]
    if pairs > 6e9:
        return None
    G, lens = Hq // H, s["lens"].tolist()
    out = torch.zeros((case["requests"] * new, Hq, d), dtype=torch.float64, device=DEV)
    lse = torch.zeros((case["requests"] * new, Hq), dtype=torch.float64, device=DEV)
    weights = None if s["weights"] is None else s["weights"].double()
    for r, n in enumerate(lens):
        ids = s["table"][r, :-(-n // bs)].long()
        for h in range(H):
            k, v = ((_decode(s[m + "_codes"][ids, h]).double()
                     * s[m + "_scale"][ids, h].double()[:, None, None]).reshape(-1, d)[:n]
                    for m in "kv")
            limit = n - new + torch.arange(new, device=DEV)[:, None]
            mask = torch.arange(n, device=DEV)[None] > limit
            for g in range(G):
                q = s["q"][r * new:(r + 1) * new, h * G + g].double()
                x = ((q @ k.T) * s["scale"]).masked_fill_(mask, -math.inf)
                total = torch.logsumexp(x, -1)
                p = torch.exp_(x.sub_(total[:, None]))
                out[r * new:(r + 1) * new, h * G + g] = p @ v
                lse[r * new:(r + 1) * new, h * G + g] = total
                if weights is not None:
                    weights[r, h, :n] += p.sum(0)
    return [out, lse, weights]


def _exact_evict(s):
    case = s["case"]
    keep, sinks, recent, bs = (case[k] for k in ("keep", "sinks", "recent", "block"))
    lens, table, dst = s["lens"].tolist(), s["table"].long(), s["dst_table"].long()
    R, H = case["requests"], case["heads"]
    kept_weights = torch.zeros((R, H, keep), dtype=torch.float64, device=DEV)
    outs = [_decode(s["k_codes"]).double(), _decode(s["v_codes"]).double()]
    scales = [s["k_scale"].double(), s["v_scale"].double()]
    for r, n in enumerate(lens):
        m = min(n, keep)
        for h in range(H):
            w = s["weights"][r, h, :n].double()
            key = w.clone()
            key[:sinks] = math.inf
            key[max(0, n - recent):] = math.inf
            # a stable order by falling weight leaves the lower slot first
            at = torch.argsort(-key, stable=True)[:m].sort()[0]
            kept_weights[r, h, :m] = w[at]
            for codes, scale in zip(outs, scales):
                ids = table[r, at // bs]
                x = codes[ids, h, at % bs] * scale[ids, h][:, None]
                P = -(-m // bs)
                page = torch.nn.functional.pad(x, (0, 0, 0, P * bs - m)).reshape(P, bs, -1)
                new = _exact_scale(page.abs().amax((1, 2)))
                y = _exact_round(page / new[:, None, None]).reshape(P * bs, -1)[:m]
                j = torch.arange(m, device=DEV)
                codes[dst[r, j // bs], h, j % bs] = y
                scale[dst[r, :P], h] = new
    return [None, kept_weights, None] + outs + scales
