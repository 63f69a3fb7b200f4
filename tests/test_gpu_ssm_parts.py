"""The scan's fp32 operands on the matrix unit: the state and the block's weights
where they enter y, and Q where it enters dB and dC, hold 24 bits whatever the
inputs' type.  Sums of two terms that cancel to about 2^-14 of their size show
operands of fewer bits; their results are then rounded once.

Bounds, u = 2^-24, h = half a step of the output's type, mag the two terms'
absolute sum.  Every factor but one is a power of two and every decay is e^0, so a
term enters as three parts whose products are exact: six additions, each off by at
most 2 u mag (one rounding, or one cut-off, of a partial sum no larger than mag).
Q = dP dt: dP is a sum of three exact products (6 u).
"""
import pytest
import torch

from layer_ref import DTYPES, HALF, U, spans, ssm_ref, within
from parity import say

import gated_delta_rule_81_amd as kda

DEV = "cuda:0"
DIMS = [(2, 1, 64, 64), (2, 1, 64, 128), (3, 1, 64, 128), (1, 1, 128, 64), (1, 1, 128, 128)]


def zeros(n, T, H, G, P, N):
    z = torch.zeros
    return dict(x=z(n, T, H, P), dt=z(n, T, H), A=z(H), B=z(n, T, G, N), C=z(n, T, G, N), D=z(H),
                state=z(n, H, P, N))


def on_device(d, dt):
    return {k: (v.to(dt) if k in ("x", "B", "C") else v).to(DEV) for k, v in d.items()}


def reference(d, T, f=lambda v: v):
    v = {k: f(t.double()) for k, t in d.items()}
    return ssm_ref(v["x"], v["dt"], v["A"], v["B"], v["C"], v["D"], v["state"],
                   spans(d["x"].shape[0], T, None))


def positions(n, T, seed):
    """Two different tokens each, the earlier first: in one tile of 16, in two, in
    two halves of a block."""
    g = torch.Generator().manual_seed(seed)
    p = [(0, 1), (14, 15), (15, 16), (31, 32), (3, 60), (47, 48)]
    while len(p) < n:
        a, b = sorted(torch.randperm(T, generator=g)[:2].tolist())
        p.append((a, b))
    return p[:n]


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("H,G,P,N", DIMS)
def test_state_in_the_output(H, G, P, N, dtype):
    """y_t = S C_t of two channels that nearly cancel, no new input, no decay."""
    n, T = 2, 130
    g = torch.Generator().manual_seed(P + N)
    d = zeros(n, T, H, G, P, N)
    v = torch.randn(n, H, P, N // 2, generator=g)
    d["state"] = torch.cat([v, v + 2.0 ** -14 * torch.randn(v.shape, generator=g)], -1)
    for t in range(T):
        j = int(torch.randint(N // 2, (), generator=g))
        d["C"][:, t, :, j], d["C"][:, t, :, j + N // 2] = 1.0, -1.0
    say("ssm parts: state", H, P, N, dtype)
    dev = on_device(d, DTYPES[dtype])
    out, fin = kda.ssm_chunk_fwd(*(dev[k] for k in ("x", "dt", "A", "B", "C", "D", "state")))
    torch.cuda.synchronize()
    ref, _ = reference(d, T)
    mag, _ = reference(d, T, torch.abs)
    h = HALF[DTYPES[dtype]]
    assert torch.equal(fin.cpu(), d["state"])
    within(out, ref, h * ref.abs() + 12 * U * mag * (1 + h), "out")


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("skip", [False, True])
@pytest.mark.parametrize("H,G,P,N", DIMS)
def test_weights_of_the_block(H, G, P, N, skip, dtype):
    """y_t = dt_a x_a + dt_b x_b (+ D x_t) with x_b = -x_a and dt_b close to dt_a; B
    and C are one channel.  With D, which comes close to -dt_b, b's own output
    cancels in its weight, one more rounding."""
    n, T = 12, 64
    g = torch.Generator().manual_seed(P + N)
    d = zeros(n, T, H, G, P, N)
    d["B"][..., 5] = d["C"][..., 5] = 1.0
    near = lambda v: v * (1 + 2.0 ** -14 * torch.randn(v.shape, generator=g))
    base = torch.rand(H, generator=g) + 0.5
    if skip:
        d["D"] = -near(base)
    for i, (a, b) in enumerate(positions(n, T, 1)):
        d["dt"][i, a], d["dt"][i, b] = near(base), near(base)
        d["x"][i, a] = torch.randint(2, (H, P), generator=g) * 2.0 - 1
        d["x"][i, b] = -d["x"][i, a]
    say("ssm parts: weights", H, P, N, skip, dtype)
    dev = on_device(d, DTYPES[dtype])
    out, _ = kda.ssm_chunk_fwd(*(dev[k] for k in ("x", "dt", "A", "B", "C", "D", "state")))
    torch.cuda.synchronize()
    ref, _ = reference(d, T)
    mag, _ = reference(d, T, torch.abs)
    h = HALF[DTYPES[dtype]]
    within(out, ref, h * ref.abs() + 14 * U * mag * (1 + h), "out")


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("side", ["dB", "dC"])
@pytest.mark.parametrize("H,G,P,N", DIMS)
def test_q_in_the_gradients(H, G, P, N, side, dtype):
    """dB_s = Q_as C_a + Q_bs C_b with C_b = -C_a, and dC_t = Q_ta B_a + Q_tb B_b
    with B_b = -B_a: Q = 1 + 2^-8 r + 2^-16 q, r the same, q another."""
    n, T = 12, 64
    g = torch.Generator().manual_seed(P + N)
    d = zeros(n, T, H, G, P, N)
    d_out = torch.zeros_like(d["x"])
    at = torch.randperm(P, generator=g)[:3]
    many, one = (d_out, d["x"]) if side == "dB" else (d["x"], d_out)
    row = "C" if side == "dB" else "B"
    for i, (a, b) in enumerate(positions(n, T, 2)):
        near = lambda: (torch.randn(H, generator=g) * 2).bfloat16().float()
        r = (1 + torch.rand(H, generator=g)).bfloat16().float()
        for t, s in ((a, 1.0), (b, -1.0)):
            many[i, t][:, at] = torch.stack([torch.ones(H), r, near()], -1)
            d[row][i, t, :, 9] = s
        # the token on the other side: at or before both (dB), at or behind both (dC)
        t = int(torch.randint(0, a + 1, (), generator=g)) if side == "dB" else int(
            torch.randint(b, T, (), generator=g))
        if t in (a, b):
            many[i, t] = 0  # its own row holds `one` then; its pair is left alone
            d[row][i, t] = 0
        one[i, t][:, at] = torch.tensor([1.0, 2.0 ** -8, 2.0 ** -16])
        d["dt"][i] = 1.0
    say("ssm parts: Q", side, H, P, N, dtype)
    dt = DTYPES[dtype]
    dev = on_device(d, dt)
    got = kda.ssm_chunk_bwd(dev["x"], dev["dt"], dev["A"], dev["B"], dev["C"], d_out.to(dt).to(DEV),
                            dev["D"], None, dev["state"])
    torch.cuda.synchronize()

    def grads(f):
        v = {k: f(t.double()).requires_grad_() for k, t in d.items()}
        y, _ = ssm_ref(v["x"], v["dt"], v["A"], v["B"], v["C"], v["D"], v["state"],
                       spans(n, T, None))
        return torch.autograd.grad(y, [v["B"], v["C"]], f(d_out.double()))

    k = 0 if side == "dB" else 1
    ref, mag = grads(lambda v: v)[k], grads(torch.abs)[k]
    h = HALF[dt]
    # H heads of a group add up: 6 more additions each
    within(got[side], ref, h * ref.abs() + (20 + 12 * (H // G - 1)) * U * mag * (1 + h), side)
