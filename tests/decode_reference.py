"""Plain fp64 numpy forms of the decoding operators (rotary positions, the 8-bit
paged cache, attention over it, eviction), and seeded caches for their tests.
They share nothing with the library."""
import math

import numpy as np
import torch


def e4m3_table():
    """Value of each of the 256 codes (1 sign, 4 exponent, 3 significand bits)."""
    v = np.empty(256)
    for c in range(256):
        e, m = (c >> 3) & 15, c & 7
        a = m * 2.0 ** -9 if e == 0 else (8 + m) * 2.0 ** (e - 10)
        v[c] = -a if c & 128 else a
    v[0x7F] = v[0xFF] = np.nan
    return v


E4M3 = e4m3_table()


def e4m3_round(x):
    """Value of the nearest code, ties to the even code, clamped to +-448."""
    a = np.minimum(np.abs(x), 448.0)
    pos = E4M3[:127]
    hi = np.searchsorted(pos, a)
    lo = np.maximum(hi - 1, 0)
    hi = np.minimum(hi, 126)
    dl, dh = a - pos[lo], pos[hi] - a
    pick = np.where((dh < dl) | ((dh == dl) & (hi % 2 == 0)), hi, lo)
    return np.copysign(pos[pick], x)


def pow2_scale(amax):
    e = -126
    while 448.0 * 2.0 ** e < amax:
        e += 1
    return 2.0 ** e


def frequencies(rot, theta, scaling=None, factor=1.0, low_band=0.0, high_band=0.0, beta_fast=32.0,
                beta_slow=1.0, original_context=0):
    w = np.array([theta ** (-2.0 * i / rot) for i in range(rot // 2)])
    if scaling is None:
        return w, 1.0
    if scaling == "linear":
        return w / factor, 1.0
    if scaling == "bands":
        n = original_context * w / (2 * math.pi)
        s = np.clip((n - low_band) / (high_band - low_band), 0, 1)
        return w * (s + (1 - s) / factor), 1.0
    pair = lambda b: rot * math.log(original_context / (b * 2 * math.pi)) / (2 * math.log(theta))
    lo = max(math.floor(pair(beta_fast)), 0)
    hi = max(min(math.ceil(pair(beta_slow)), rot - 1), lo + 0.001)
    s = 1 - np.clip((np.arange(rot // 2) - lo) / (hi - lo), 0, 1)
    return w * (s + (1 - s) / factor), 0.1 * math.log(factor) + 1


def rope(x, pos, rot, layout, w, amp, transpose=False):
    """x [tokens][heads][d] fp64."""
    y = x.copy()
    a = pos[:, None, None] * w
    c, s = amp * np.cos(a), amp * np.sin(a) * (-1 if transpose else 1)
    i = np.arange(rot // 2)
    i0, i1 = (i, i + rot // 2) if layout == "half" else (2 * i, 2 * i + 1)
    y[..., i0] = x[..., i0] * c - x[..., i1] * s
    y[..., i1] = x[..., i1] * c + x[..., i0] * s
    return y


class RefCache:
    """Codes as fp64 values [blocks][H][bs][d], scales fp64 [blocks][H]."""

    def __init__(self, codes, scale):
        self.values, self.scale = E4M3[codes], scale.astype(np.float64).copy()

    def write(self, x, table, start, cu, rows=None):
        bs = self.values.shape[2]
        for r in range(len(start)):
            i = cu[r]
            while i < cu[r + 1]:
                slot = start[r] + i - cu[r]
                s0, page = slot % bs, table[r][slot // bs]
                n = min(bs - s0, cu[r + 1] - i)
                src = np.arange(i, i + n) if rows is None else rows[i:i + n]
                for h in range(self.values.shape[1]):
                    run = x[src, h]
                    fin = np.isfinite(run)
                    new = pow2_scale(np.abs(run[fin]).max(initial=0.0))
                    if s0:
                        old = self.scale[page, h]
                        new = max(new, old)
                        self.values[page, h, :s0] = e4m3_round(
                            self.values[page, h, :s0] * (old / new))
                    self.scale[page, h] = new
                    clean = np.where(np.isnan(run), 0.0, run)
                    with np.errstate(over="ignore"):
                        self.values[page, h, s0:s0 + n] = e4m3_round(clean / new)
                i += n

    def rows(self, table_row, slots, h):
        bs = self.values.shape[2]
        page = np.array([table_row[j // bs] for j in slots], dtype=int)
        off = np.array([j % bs for j in slots], dtype=int)
        if len(page) == 0:
            return np.zeros((0, self.values.shape[3]))
        return self.values[page, h, off] * self.scale[page, h][:, None]


def attend(q, kc, vc, table, lens, cu, scale):
    """out [tokens][Hq][d], lse, weights [R][H][max len], and two sums that the
    tolerances use: sum_j p_ij |v_j| and the largest scale * sum_e |q_e k_je|."""
    n, Hq, d = q.shape
    H = kc.values.shape[1]
    G = Hq // H
    R = len(lens)
    out, mass = np.zeros((n, Hq, d)), np.zeros((n, Hq, d))
    lse, reach = np.full((n, Hq), -np.inf), np.zeros((n, Hq))
    weights = np.zeros((R, H, max(list(lens) + [1])))
    for r in range(R):
        new, L = cu[r + 1] - cu[r], lens[r]
        for h in range(H):
            k, v = kc.rows(table[r], range(L), h), vc.rows(table[r], range(L), h)
            for i in range(new):
                see = L - new + i + 1
                if see <= 0:
                    continue
                for g in range(h * G, (h + 1) * G):
                    row = q[cu[r] + i, g]
                    x = scale * (k[:see] @ row)
                    m = x.max()
                    e = np.exp(x - m)
                    p = e / e.sum()
                    out[cu[r] + i, g] = p @ v[:see]
                    mass[cu[r] + i, g] = p @ np.abs(v[:see])
                    lse[cu[r] + i, g] = m + math.log(e.sum())
                    reach[cu[r] + i, g] = abs(scale) * (np.abs(k[:see]) @ np.abs(row)).max()
                    weights[r, h, :see] += p
    return out, lse, weights, mass, reach


def evict(weights, lens, keep, sinks, recent):
    """kept slots per (request, head), ascending."""
    R, H = weights.shape[:2]
    kept = np.full((R, H, keep), -1)
    for r in range(R):
        L = lens[r]
        for h in range(H):
            if L <= keep:
                kept[r, h, :L] = np.arange(L)
                continue
            held = list(range(sinks)) + list(range(L - recent, L))
            rest = range(sinks, L - recent)
            w = [(-math.inf, 1) if math.isnan(weights[r, h, j]) else (weights[r, h, j], 0)
                 for j in range(L)]
            rest = sorted(rest, key=lambda j: (w[j][1], -w[j][0], j))[:keep - len(held)]
            kept[r, h] = sorted(held + rest)
    return kept


def block_table(lens, bs, num_blocks, seed, width=None):
    """Shuffled blocks for each request; unused entries name no block (-1)."""
    rng = np.random.default_rng(seed)
    need = [-(-n // bs) for n in lens]
    order = rng.permutation(num_blocks)
    assert sum(need) <= num_blocks
    table = np.full((len(lens), max(need + [1]) if width is None else width), -1, dtype=np.int32)
    at = 0
    for r, n in enumerate(need):
        table[r, :n] = order[at:at + n]
        at += n
    return table


def random_cache(num_blocks, H, bs, d, seed, scales="pow2"):
    """Codes (uint8, no NaN) and scales, numpy."""
    rng = np.random.default_rng(seed)
    x = rng.standard_normal((num_blocks, H, bs, d)) * np.exp(0.5 * rng.standard_normal((1, H, 1, d)))
    if scales == "pow2":
        scale = np.vectorize(pow2_scale)(np.abs(x).max((2, 3)))
    else:
        scale = np.abs(x).max((2, 3)) / 448.0 * rng.uniform(1.0, 3.0, x.shape[:2])
    scale = scale.astype(np.float32)
    y = torch.tensor(x / scale[:, :, None, None].astype(np.float64)).float().clamp(-448, 448)
    return y.to(torch.float8_e4m3fn).view(torch.uint8).numpy(), scale


def poison(codes, scale, table, lens, bs):
    """Every slot that no request holds gets NaN codes, every block that none
    uses a NaN scale."""
    used = np.zeros(codes.shape[:1] + (bs,), dtype=bool)
    for r, n in enumerate(lens):
        for j in range(n):
            used[table[r][j // bs], j % bs] = True
    codes[~np.broadcast_to(used[:, None, :], codes.shape[:3])] = 0x7F
    scale[~used.any(1)] = np.nan
