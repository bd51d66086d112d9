"""fp32 queries keep what two f16 parts of queries and probabilities give: a tolerance that
one part would not meet, which is shown on the same inputs.

Tolerance.  A query in two f16 parts is off by 2^-22 of itself; a score is a sum of d
products in fp32 (2^-24 each, tensor cores truncate where they align) and three more
roundings: xe = (d + 7) 2^-24 reach (reach: scale * sum |q k|).  A probability's score and its
row's log-sum-exp are each off by that, both over two parts: 4 xe; exponentials take 2^-22 each, the
term's, a raised maximum's, the warps' and the parts' join, numerator and denominator: 8 2^-22.  In
two f16 parts before the product with v: 2^-21.  Additions over n slots, above and below: 2 n
2^-24.  All times sum p |v| (mass); a few roundings of the result, 2^-22 of it."""
import numpy as np
import pytest
import torch

import decode_reference as ref
from test_gpu_attend8_shared import call, make, want_of

pytestmark = pytest.mark.gpu


def one_part(c):
    """The result with probabilities, relative to their row's largest, rounded to 11 bits."""
    n, Hq, d = c["q"].shape
    G = Hq // c["rk"].values.shape[1]
    out = np.zeros((n, Hq, d))
    q = c["q"].double().numpy()
    for p in range(len(c["prefixes"])):
        for r in range(c["groups"][p], c["groups"][p + 1]):
            row = (c["prefix_table"][p], c["prefixes"][p], c["table"][r])
            total, new = c["prefixes"][p] + c["lens"][r], c["cu"][r + 1] - c["cu"][r]
            for h in range(Hq):
                k, v = (x.rows(row, range(total), h // G) for x in (c["rk"], c["rv"]))
                for i in range(new):
                    x = (k[:total - new + i + 1] @ q[c["cu"][r] + i, h]) * d ** -0.5
                    e = np.exp(x - x.max())
                    half = e.astype(np.float16).astype(np.float64)
                    out[c["cu"][r] + i, h] = half @ v[:len(x)] / e.sum()
    return out


@pytest.mark.parametrize("H,G,d,bs,prefixes,members,lens,news", [
    (2, 4, 16, 16, [30], [4], [3, 5, 9, 12], [1] * 4),                 # the prefix in parts
    (1, 8, 32, 8, [17, 40], [2, 2], [2, 12, 5, 7], [1, 3, 2, 1]),
    (1, 2, 16, 16, [24], [2], [40, 41], [35, 40]),                     # more rows than an item's CTA takes
    (1, 5, 48, 5, [12, 0], [1, 2], [9, 20, 16], [1, 2, 1]),
])
def test_two_parts(H, G, d, bs, prefixes, members, lens, news):
    c = make(H, G, d, bs, prefixes, members, lens, news, torch.float32, 51, qscale=0.3)
    o, ls, _, mass, reach = want_of(c)
    n = max(prefixes) + max(lens)
    xe = (d + 7) * 2.0 ** -24 * reach
    rel = 4 * xe + 8 * 2.0 ** -22 + 2.0 ** -21 + 2 * n * 2.0 ** -24
    tol = rel[..., None] * mass + 2.0 ** -22 * np.abs(o) + 1e-30
    out, lse = call(c)
    error = np.abs(out.double().cpu().numpy() - o) / tol
    assert error.max() <= 1, error.max()
    seen = np.isfinite(ls)
    near = 2 * xe + 4 * 2.0 ** -22 + n * 2.0 ** -24 + 2.0 ** -22 * np.abs(np.where(seen, ls, 0))
    assert (np.abs(lse.double().cpu().numpy() - ls)[seen] <= near[seen]).all()
    # one part would be seen
    assert (np.abs(one_part(c) - o) / tol).max() > 1.5
