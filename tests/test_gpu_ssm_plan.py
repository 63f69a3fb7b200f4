"""The scan at the cuts that large calls have: pieces of three and more blocks (the
state from block to block, both decay buffers again and again), equal rows left
whole, and gradient workgroups of several heads (dB and dC summed over them, the
three decay buffers in turn), whole sets and uneven ones.

How a call is cut follows from its sizes alone and shows in the size of its
workspace: every case states its piece lengths and sets, and the sizes are held
to them, so that another rule fails here instead of leaving these paths untested.
Heads do not depend on each other, nor groups: the 64-bit definition is run for
the first group and the last.
"""
import pytest
import torch

import test_gpu_ssm as ssm
from layer_ref import DTYPES, HALF, ssm_ref, within
from parity import say

import gated_delta_rule_81_amd as kda

# case as in test_gpu_ssm.py; tokens of a piece (None: sequences whole), forward and
# backward; sets of a group's heads in the gradient, heads of the first and last set
PLANS = [
    ((1, 600, None, 256, 64, 64, 64, True, True, 0, "bf16", 1.0), 192, None, 1, (4, 4)),
    ((1, 600, None, 128, 32, 128, 128, True, True, 8, "bf16", 0.1), 192, None, 2, (2, 2)),
    ((1, 1000, None, 140, 20, 64, 128, True, False, 0, "bf16", 0.3), 192, 320, 2, (4, 3)),
    ((1, 1000, None, 84, 12, 64, 64, True, True, 0, "bf16", 1.0), 128, 192, 3, (3, 1)),
    ((1, 600, None, 256, 64, 64, 64, True, True, 0, "f32", 0.3), 192, None, 1, (4, 4)),
    ((1, 300, None, 128, 64, 128, 128, True, False, 4, "f32", 1.0), 128, None, 1, (2, 2)),
    ((4, 200, None, 128, 32, 64, 64, True, True, 0, "bf16", 0.3), None, None, 1, (4, 4)),
    ((4, 100, None, 128, 32, 64, 128, True, True, 0, "f32", 1.0), None, None, 1, (4, 4)),
    ((1, 0, [0, 700, 1, 64, 385, 0, 50], 128, 32, 64, 128, True, True, 0, "bf16", 0.3), 192, 320, 1,
     (4, 4)),
    ((1, 0, [0, 400, 33, 0, 167], 256, 64, 64, 64, True, True, 8, "f32", 1.0), 192, 320, 1, (4, 4)),
]
IDS = [f"{p[0][:7]}-{p[0][10]}" for p in PLANS]


@pytest.mark.parametrize("plan", PLANS, ids=IDS)
def test_plan(plan):
    """The workspaces' sizes are those of the plan."""
    (B, T, lens, H, G, P, N, _, _, _, dtype, _), fwd, bwd, sets, heads = plan
    dt, L = DTYPES[dtype], 64 if dtype == "bf16" else 32
    num = len(lens) if lens else 0
    T = sum(lens) if lens else T
    up = lambda a, b: -(-a // b)

    def pieces(n):  # states of the pieces and their decays
        if n is None:
            return 0
        count = (2 * T // n if lens else B * up(T, n)) * H
        return 8 * (up(count, 2) * 2) + 4 * count * P * N

    assert kda.ssm_workspace_size(B, T, H, P, N, num_seqs=num) == pieces(fwd)
    blocks = T // L + num + 1 if lens else B * up(T, L)
    parts = 2 * sets * B * T * G * N if sets > 1 else 0
    want = 2 * pieces(bwd) + 4 * (2 * blocks * H * P * N + up(2 * blocks * H, 4) * 4 + parts)
    assert kda.ssm_bwd_workspace_size(B, T, H, G, P, N, dt, num_seqs=num) == want
    # what the plan is here for
    whole = max(lens) if lens else T
    assert (bwd or whole) > 2 * L and (fwd or whole) > 2 * L or sets > 2
    per_set = up(H // G, sets)
    assert heads == (per_set, H // G - per_set * (sets - 1)) and per_set > 1


def of_groups(t, name, j, per):
    """The part of a tensor that belongs to group j's heads."""
    if t is None:
        return None
    at = slice(j, j + 1) if name in ("B", "C", "dB", "dC") else slice(j * per, (j + 1) * per)
    return t[at] if name in ("A", "D", "dA", "dD") else (
        t[:, at] if name in ("state", "d_initial_state") else t[:, :, at])


def reference_of(f, j, per):
    out = {k: of_groups(v, k, j, per) for k, v in f.items() if k != "seqs"}
    return {**out, "seqs": f["seqs"]}


@pytest.mark.gpu
@pytest.mark.parametrize("plan", PLANS, ids=IDS)
def test_forward(plan):
    case = plan[0]
    H, G, dt = case[3], case[4], DTYPES[case[10]]
    dev, f = ssm.make(case, 11)
    say("ssm plan forward", case)
    args = (dev["x"], dev["dt"], dev["A"], dev["B"], dev["C"], dev["D"])
    out, fin = kda.ssm_chunk_fwd(*args, dev["state"], dev["cu"])
    st = dev["state"].clone()
    again, same = kda.ssm_chunk_fwd(*args, st, dev["cu"], final_state=st)  # in place
    torch.cuda.synchronize()
    assert torch.equal(out, again) and torch.equal(fin, st)
    h = HALF[dt]
    for j in (0, G - 1):
        r = reference_of(f, j, H // G)
        ref, ref_fin = ssm_ref(*(r[k] for k in ("x", "dt", "A", "B", "C", "D", "state", "seqs")))
        m, m_fin = ssm.magnitudes(r)
        fy, fs = ssm.factors(torch.float32, f["x"].shape[1] // 32 + 1)
        within(of_groups(fin, "state", j, H // G), ref_fin, fs * m_fin + 1e-37, f"final state {j}")
        within(of_groups(out, "out", j, H // G), ref, h * ref.abs() + fy * (1 + h) * m + 1e-37,
               f"out {j}")


@pytest.mark.gpu
@pytest.mark.parametrize("plan", PLANS, ids=IDS)
def test_backward(plan):
    """As in test_gpu_ssm.py; dB and dC of a group add up its heads."""
    case = plan[0]
    H, G, dt = case[3], case[4], DTYPES[case[10]]
    dev, f = ssm.make(case, 12)
    g = torch.Generator().manual_seed(78)
    d_out = torch.randn(f["x"].shape, generator=g).to(dt)
    d_fin = torch.randn(f["state"].shape, generator=g)
    say("ssm plan backward", case)
    got = kda.ssm_chunk_bwd(dev["x"], dev["dt"], dev["A"], dev["B"], dev["C"], d_out.to(ssm.DEV),
                            dev["D"], d_fin.to(ssm.DEV), dev["state"], dev["cu"])
    torch.cuda.synchronize()
    h = HALF[dt]
    fy, _ = ssm.factors(torch.float32, f["x"].shape[1] // 32 + 1)
    for j in (0, G - 1):
        r = reference_of(f, j, H // G)
        do = of_groups(d_out, "x", j, H // G).double()
        df = of_groups(d_fin, "state", j, H // G).double()
        names = ["x", "dt", "A", "B", "C", "state"] + ([] if r["D"] is None else ["D"])
        v = {k: None if r[k] is None else r[k].clone().requires_grad_()
             for k in ("x", "dt", "A", "B", "C", "D", "state")}
        y, fin = ssm_ref(*v.values(), r["seqs"])
        ref = dict(zip(names, torch.autograd.grad([y, fin], [v[k] for k in names], [do, df])))
        mag = ssm.grad_magnitudes(r, do, df)
        for name, key in (("dx", "x"), ("ddt", "dt"), ("dA", "A"), ("dB", "B"), ("dC", "C"),
                          ("dD", "D"), ("d_initial_state", "state")):
            if ref.get(key) is None:
                assert got[name] is None
                continue
            bound = 2 * fy * mag[name] * (1 + h) + 1e-37
            if name in ("dx", "dB", "dC"):
                bound = bound + h * ref[key].abs()
            within(of_groups(got[name], name, j, H // G), ref[key], bound, f"{name} {j}")


@pytest.mark.gpu
@pytest.mark.parametrize("plan", [PLANS[0], PLANS[2], PLANS[4], PLANS[6], PLANS[9]], ids=str)
def test_nan_from_block_to_block(plan):
    """A NaN of x in the second block of a piece, and one in the first head: the
    row's outputs and state from there on, nothing else."""
    case = plan[0]
    H, G = case[3], case[4]
    dev, f = ssm.make(case, 13)
    say("ssm plan nan", case)
    args = (dev["x"], dev["dt"], dev["A"], dev["B"], dev["C"], dev["D"], dev["state"], dev["cu"])
    clean, clean_fin = kda.ssm_chunk_fwd(*args)
    n = 1 if case[2] else 0
    b, t0, t1 = f["seqs"][n]
    spots = [(H - 1, 77, 13), (0, 2, 5)]
    for h, t, p in spots:
        dev["x"][b, t0 + t, h, p] = float("nan")
    out, fin = kda.ssm_chunk_fwd(*args)
    torch.cuda.synchronize()
    odd_out, odd_fin = torch.zeros_like(out, dtype=torch.bool), torch.zeros_like(fin, dtype=torch.bool)
    for h, t, p in spots:
        odd_out[b, t0 + t: t1, h, p] = True
        odd_fin[n, h, p] = True
    for got, was, odd in ((out, clean, odd_out), (fin, clean_fin, odd_fin)):
        assert torch.isnan(got[odd]).all() and torch.equal(got[~odd], was[~odd])
