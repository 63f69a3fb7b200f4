"""Infinities and NaN in values among the tokens that only some rows of a call see: an infinity
that a row sees is infinite there, whatever later tokens hold that the row does not see.  Bounds as in
test_gpu_prefix_attn.py."""
import math

import pytest
import torch

from cache_ref import attend, attention_inputs, reference
from parity import say
from test_gpu_prefix_attn import bounds, case

import gated_delta_rule_81_amd as kda


def compare_odd(got, x, c):
    out, lse, wgt = reference(x, c)
    bo, bl = bounds(x, c, lse, wgt, out)
    y, z = got[0].double().cpu(), got[1].double().cpu()
    fine = torch.isfinite(out)
    assert torch.equal(torch.isnan(y), torch.isnan(out))
    assert torch.equal(y[out.abs() == math.inf], out[out.abs() == math.inf])
    assert torch.isfinite(y[fine]).all() and ((y - out).abs() <= bo)[fine].all()
    assert ((z - lse).abs() <= bl).all()


@pytest.mark.gpu
@pytest.mark.parametrize("c", [
    case((16,), (40,), 0, 16, 1, 1, 64),
    case((16,), (40,), 0, 16, 2, 2, 128, "f32"),
    case((8, 6), (36, 70), 0, 24, 8, 2, 64, "f32"),
    case((8, 1), (40, 9), 130, 32, 4, 1, 128),
    case((30,), (150,), 0, 16, 1, 1, 64),
    case((40,), (70,), 0, 16, 4, 1, 64),
    case((150, 190), (150, 333), 60, 64, 4, 2, 128),
], ids=lambda c: f"{c['new']}-{c['lens']}-{c['d']}-{c['dtype']}".replace(" ", ""))
def test_infinities_that_some_rows_see(c):
    """An infinity in one of the tokens before the last ones and a NaN or an infinity in later
    ones, in other channels and in the same."""
    page, L, n = c["page"], c["lens"][0], c["new"][0]
    first = L - n  # the first new token's place: every row of the session sees those up to it
    for j, later, value, channel in ((5, L - 1, "nan", 20), (first, L - 5, "nan", 20), (5, L - 2, "inf", 7),
                                     (first - 1, L - 1, "-inf", 20), (first + 2, L - 1, "nan", 7)):
        if j < 0:
            continue
        x = attention_inputs(c, 21)
        x["v"][x["table"][0, j // page], j % page, :, 7] = math.inf
        x["v"][x["table"][0, later // page], later % page, :, channel] = float(value)
        say("prefix_attention: an infinity that some rows see", j, later, value, c)
        got = attend(kda, x, c)
        torch.cuda.synchronize()
        compare_odd(got, x, c)
