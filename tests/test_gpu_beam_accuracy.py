"""The log-sum-exps of beam selection, over rows of any length and few or many of them.

Tolerance.  A logit x reaches the sum by steps: x - r with r its thread's reference (its
first chunk's maximum, raised to a chunk's maximum where that is more than 8 above), the
reference's own rises, and its distance to the row's largest reference; all steps together
are at most 2 (max - x) + 16, and max - x where no chunk holds a larger logit of the thread than the
first.  Of a step's argument two roundings and the constant are off by 2^-24 + 2^-24 +
2^-26 < 2^-22.8, so the sum's relative error is at most that times the steps' mean under the softmax.
Then exponentials of 2^-22 each: the term's, the rises' while the old sum counts (its share falls by
e^8 with each: three), a warp's and a CTA's.  And roundings of 2^-24: ten of a chunk's additions,
three of the rises' products, five of a warp's, two of its products.  The running sum over the
chunks carries the rest of each addition along, so that the row's length does not
count."""
import math

import pytest
import torch

from cross_model_kv_transfer_gb300 import kvx

pytestmark = pytest.mark.gpu

FIRST = ("first peak", "falling", "flat")     # no chunk is above the first


def rows_of(V):
    i = torch.arange(V, dtype=torch.float64)
    below = lambda d, at: torch.where(i == at, 0.0, -d)
    return {"first peak": below(14.0, 5), "peak": below(math.log(V) - 1.37, V // 3), "late peak": below(12.3, V - 1),
            "rising": i * (30.0 / V), "slowly": i * (0.6 / V), "steps": torch.floor(i * 7 / V) * 8.5,
            "falling": -i * (30.0 / V), "flat": torch.full((V,), 0.3, dtype=torch.float64),
            "far": 3000.0 + (i * 0.37).remainder(11.0)}


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("V", [5000, 128256, 262143, 1000001, 2000001])
@pytest.mark.parametrize("rows", [9, 306])
def test_log_sum_exps(rows, V, dtype):
    """Few rows are spread over several CTAs each, many take one."""
    kinds = rows_of(V)
    x = torch.stack(list(kinds.values())).to(dtype).cuda()
    exact = x.double()
    lse = torch.logsumexp(exact, -1)
    top = exact.amax(-1)
    steps = ((exact - lse[:, None]).exp() * (top[:, None] - exact)).sum(-1)
    # so that the best score is next to 0 and its rounding to fp32 next to none
    before = (lse - top).float()
    want, order = exact.sort(dim=-1, descending=True, stable=True)
    want = want[:, :4] + before.double()[:, None] - lse[:, None]
    many = rows // len(kinds)
    tokens, parents, new, _ = kvx.beam_select(x.repeat(many, 1), before.repeat(many)[:, None].contiguous(), beams=4)
    assert torch.equal(tokens, order[:, :4].int().repeat(many, 1))
    error = (new.double().view(many, -1, 4) - want).abs() - 2.0 ** -24 * want.abs()
    for k, kind in enumerate(kinds):
        path = steps[k].item() if kind in FIRST else 2 * steps[k].item() + 16
        tol = path * 2.0 ** -22.8 + 6 * 2.0 ** -22 + 20 * 2.0 ** -24
        assert error[:, k].max().item() <= tol, (kind, error[:, k].max().item() / tol)
