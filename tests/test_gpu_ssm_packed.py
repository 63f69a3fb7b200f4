"""The scan over packed sequences of which some are cut into pieces and many are
not, forward and backward: the bounds of test_gpu_ssm.py against the 64-bit
definition, a workspace of exactly the size that is asked for between two
guards, and the state updated in place.
"""
import pytest
import torch

import test_gpu_ssm as ssm
from layer_ref import DTYPES
from parity import say

import gated_delta_rule_81_amd as kda

DEV = "cuda:0"
LENS = [
    # around one, two and three pieces of 64, empty ones between and at both ends
    [0, 65, 64, 0, 66, 1, 129, 63, 0, 0, 192, 193, 64, 65, 0],
    [1] * 70 + [128] + [1] * 70,
    [64] * 9,
    [65] * 9,
]
DIMS = [("bf16", 2, 1, 64, 64), ("f32", 1, 1, 64, 128), ("bf16", 1, 1, 128, 64)]


def case_of(lens, dims):
    dtype, H, G, P, N = dims
    return (1, 0, lens, H, G, P, N, True, True, 0, dtype, 1.0)


def guarded(size):
    """A workspace of `size` bytes between two guards, and a check of these."""
    room = torch.full((size + 512,), 0x5A, dtype=torch.uint8, device=DEV)
    check = lambda: bool((room[:256] == 0x5A).all()) and bool((room[256 + size:] == 0x5A).all())
    return room[256: 256 + size], check


@pytest.mark.gpu
@pytest.mark.parametrize("dims", DIMS, ids=str)
@pytest.mark.parametrize("lens", LENS, ids=range(len(LENS)))
def test_forward(lens, dims):
    dtype, H, G, P, N = dims
    ssm.test_forward(case_of(lens, dims))
    dev, _ = ssm.make(case_of(lens, dims))
    args = (dev["x"], dev["dt"], dev["A"], dev["B"], dev["C"], dev["D"])
    want, want_fin = kda.ssm_chunk_fwd(*args, dev["state"], dev["cu"])
    ws, whole = guarded(kda.ssm_workspace_size(1, sum(lens), H, P, N, num_seqs=len(lens)))
    st = dev["state"].clone()
    out, _ = kda.ssm_chunk_fwd(*args, st, dev["cu"], workspace=ws, final_state=st)
    torch.cuda.synchronize()
    assert whole() and torch.equal(out, want) and torch.equal(st, want_fin)


@pytest.mark.gpu
@pytest.mark.parametrize("dims", DIMS, ids=str)
@pytest.mark.parametrize("lens", LENS, ids=range(len(LENS)))
def test_backward(lens, dims):
    dtype, H, G, P, N = dims
    ssm.test_backward(case_of(lens, dims))
    dev, f = ssm.make(case_of(lens, dims))
    g = torch.Generator().manual_seed(5)
    d_out = torch.randn(f["x"].shape, generator=g).to(DTYPES[dtype]).to(DEV)
    d_fin = torch.randn(f["state"].shape, generator=g).to(DEV)
    args = (dev["x"], dev["dt"], dev["A"], dev["B"], dev["C"], d_out, dev["D"], d_fin, dev["state"],
            dev["cu"])
    want = kda.ssm_chunk_bwd(*args)
    ws, whole = guarded(kda.ssm_bwd_workspace_size(1, sum(lens), H, G, P, N, DTYPES[dtype],
                                                   num_seqs=len(lens)))
    got = kda.ssm_chunk_bwd(*args, workspace=ws)
    torch.cuda.synchronize()
    assert whole()
    for k, v in want.items():
        assert torch.equal(got[k], v), k


@pytest.mark.gpu
def test_a_workspace_for_many_prompts():
    """Prompts shorter than a piece: 1,000 of them, in 96 heads, need a fraction of
    the states they would fill (each 16 KiB a head), and one long prompt among them
    is still cut (its outputs are those of its own call)."""
    H, P, N = 96, 64, 64
    lens = [3] * 500 + [700] + [3] * 500
    say("ssm packed: 1,001 prompts")
    dev, f = ssm.make((1, 0, lens, H, 8, P, N, False, True, 0, "bf16", 1.0))
    size = kda.ssm_workspace_size(1, sum(lens), H, P, N, num_seqs=len(lens))
    assert 0 < size < (len(lens) * H * P * N * 4) // 8
    ws, whole = guarded(size)
    out, fin = kda.ssm_chunk_fwd(dev["x"], dev["dt"], dev["A"], dev["B"], dev["C"], dev["D"], None,
                                 dev["cu"], workspace=ws)
    torch.cuda.synchronize()
    assert whole()
    for n in (0, 499, 500, 501, 1000):
        _, t0, t1 = f["seqs"][n]
        c = lambda t: t[:, t0:t1].double().cpu()
        g = {k: c(dev[k]) for k in ("x", "dt", "B", "C")}
        one = (g["x"], g["dt"], f["A"], g["B"], g["C"], f["D"], f["state"][n: n + 1], [(0, 0, t1 - t0)])
        ref, ref_fin = ssm.ssm_ref(*one)
        ab = tuple(v.abs() if torch.is_tensor(v) and i != 2 else v for i, v in enumerate(one))
        m, m_fin = ssm.ssm_ref(*ab)
        fy, fs = ssm.factors(torch.bfloat16, 700 // 32 + 1)
        h = ssm.HALF[torch.bfloat16]
        ssm.within(fin[n: n + 1], ref_fin, fs * m_fin + 1e-37, "final state")
        ssm.within(out[:, t0:t1], ref, h * ref.abs() + fy * (1 + h) * m + 1e-37, "out")
