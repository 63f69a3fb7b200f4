"""NaN and infinities in the scan's x, B and C: they reach what the definition says
they reach (outputs of their own token and later ones of their sequence, rows and
columns of the state), and nothing else: no earlier token, other row or other
sequence.  What stays finite keeps its bits.
"""
import pytest
import torch

import test_gpu_ssm as ssm
from layer_ref import ssm_ref
from parity import say

import gated_delta_rule_81_amd as kda

NAN, INF = float("nan"), float("inf")
CASES = [
    (2, 150, None, 4, 2, 64, 64, True, True, 0, "bf16", 0.1),
    (1, 150, None, 3, 1, 64, 128, True, False, 0, "bf16", 0.1),
    (1, 0, [70, 0, 65, 40], 1, 1, 128, 128, True, True, 0, "bf16", 0.1),
    (2, 100, None, 2, 1, 64, 64, True, True, 0, "f32", 0.1),
    (1, 0, [70, 0, 33, 40], 2, 2, 128, 64, True, True, 0, "f32", 0.1),
]
PLACES = [  # tensor, value, (sequence's token, channel) of each
    ("x", NAN, [(5, 3)]), ("x", INF, [(31, 63)]), ("x", -INF, [(17, 0), (16, 40)]),
    ("x", NAN, [(0, 9), (63, 10), (64, 11), (33, 3)]),
    ("B", NAN, [(20, 7)]), ("B", INF, [(47, 1)]), ("C", NAN, [(20, 7)]), ("C", -INF, [(63, 63)]),
]


@pytest.mark.gpu
@pytest.mark.parametrize("place", PLACES, ids=str)
@pytest.mark.parametrize("case", CASES, ids=str)
def test_they_reach_nothing_else(case, place):
    what, value, at = place
    dev, f = ssm.make(case, 6)
    say("ssm nan", case, place)
    args = lambda d: (d["x"], d["dt"], d["A"], d["B"], d["C"], d["D"], d["state"])
    clean, clean_fin = kda.ssm_chunk_fwd(*args(dev), dev["cu"])
    b, t0, t1 = f["seqs"][0]
    for t, c in at:
        if t < t1 - t0:
            dev[what][b, t0 + t, -1, c] = value  # of the last head or group
            f[what][b, t0 + t, -1, c] = value
    out, fin = kda.ssm_chunk_fwd(*args(dev), dev["cu"])
    torch.cuda.synchronize()
    ref, ref_fin = ssm_ref(*args(f), f["seqs"])
    for got, was, want in ((out, clean, ref), (fin, clean_fin, ref_fin)):
        got, was = got.cpu(), was.cpu()
        assert torch.equal(torch.isfinite(got), torch.isfinite(want))
        untouched = torch.isfinite(want)
        # finite and behind a poisoned token: only where the poison does not enter
        assert torch.equal(got[untouched], was[untouched])
