"""The operators around the recurrence run together with it, as a layer does:
projection rows -> short convolution -> norm (and rotation) of queries and keys
-> KDA, for a packed prompt with states, for single tokens after it, and for the
gradient; and projection rows -> short convolution -> state space scan.

Each stage's own bounds are in its own test module; here the chain is held to
its inputs' type: every stage passes on values rounded to the type (half a step
h = 2^-8 for bf16, 2^-24 for fp32), so after three stages the 2-norm of the
difference is under 3 h of the result's plus the recurrence's own parity bound
(2e-2 for bf16, 1e-4 for fp32, tests/parity.py), which is the larger part.
"""
import numpy as np
import pytest
import torch

import oracle
from layer_ref import DTYPES, HALF, conv_ref, offsets, qk_ref, rel, spans, ssm_ref
from parity import TOL, say

import gated_delta_rule_81_amd as kda

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
H, D, W = 3, 64, 4
C = H * D


def weights(seed, dt):
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(s, generator=g)
    p = dict(wq=r(C, W) * 0.5, wk=r(C, W) * 0.5, wv=r(C, W) * 0.5, b=r(C) * 0.1)
    a = torch.arange(400, dtype=torch.float64)[:, None] * 100.0 ** -(torch.arange(16) / 16)
    p["table"] = torch.cat([a.cos(), a.sin()], -1).float()
    return p, r


def prompt(lens, dt, seed):
    p, r = weights(seed, dt)
    T, n = sum(lens), len(lens)
    d = dict(rows=r(1, T, 3 * C + 8).to(dt), log_alpha=-torch.nn.functional.softplus(r(1, T, H, D) - 2),
             beta=torch.sigmoid(r(1, T, H)), state=r(n, H, D, D) * 0.1,
             conv=[r(n, W - 1, C).to(dt) for _ in range(3)],
             pos=torch.cat([torch.arange(5, 5 + x) for x in lens]).int()[None])
    return p, d


def front(p, d, dt, cu):
    """conv and norm on the GPU: (q, k, v, the convolutions' states)."""
    rows = d["rows"].to(DEV)
    outs, states = [], []
    for i, name in enumerate(("wq", "wk", "wv")):
        y, s = kda.short_conv(rows[..., i * C:(i + 1) * C], p[name].to(DEV), p["b"].to(DEV),
                              d["conv"][i].to(DEV), cu)
        outs.append(y.unflatten(-1, (H, D)))
        states.append(s)
    q, k = kda.qk_norm(outs[0], outs[1], table=p["table"].to(DEV), positions=d["pos"].to(DEV))
    return q, k, outs[2], states, outs


def front_ref(p, d, seqs):
    x = d["rows"].double()
    f = lambda i, n: conv_ref(x[..., i * C:(i + 1) * C], p[n].double(), p["b"].double(),
                              d["conv"][i].double(), "silu", seqs)[0].unflatten(-1, (H, D))
    norm = lambda y: qk_ref(y, None, p["table"].double(), d["pos"], "l2", 1e-6, False)
    return norm(f(0, "wq")), norm(f(1, "wk")), f(2, "wv")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_packed_prompt_then_tokens(dtype):
    dt = DTYPES[dtype]
    lens = [70, 1, 0, 33]
    steps = 4
    full = [x + steps for x in lens]
    p, d = prompt(full, dt, 5)
    say("layer: packed prompt then tokens", dtype)
    seqs = spans(1, None, full)
    cut = torch.cat([torch.arange(t0, t1 - steps) for _, t0, t1 in seqs])
    part = {k: (v[:, cut] if k in ("rows", "log_alpha", "beta", "pos") else v) for k, v in d.items()}
    cu = offsets(lens).to(DEV)
    q, k, v, conv, _ = front(p, part, dt, cu)
    out, state = kda.chunk_fwd(q, k, v.contiguous(), part["log_alpha"].to(DEV),
                               part["beta"].to(DEV), d["state"].to(DEV), cu)
    outs = []
    for i in range(steps):
        at = torch.tensor([t1 - steps + i for _, _, t1 in seqs])
        row = d["rows"][0, at].to(DEV)
        y = [kda.short_conv_step(row[:, j * C:(j + 1) * C], p[n].to(DEV), conv[j], p["b"].to(DEV))
             .unflatten(-1, (H, D)) for j, n in enumerate(("wq", "wk", "wv"))]
        qi, ki = kda.qk_norm(y[0], y[1], table=p["table"].to(DEV), positions=d["pos"][0, at].to(DEV))
        outs.append(kda.decode_step(qi, ki, y[2], d["log_alpha"][0, at].to(DEV).contiguous(),
                                    d["beta"][0, at].to(DEV).contiguous(), state))
    torch.cuda.synchronize()
    q, k, v = (t[0].numpy() for t in front_ref(p, d, seqs))
    st = np.cumsum([0] + full)
    ref, ref_state = oracle.kda_forward(q, k, v, d["log_alpha"][0].double().numpy(),
                                        d["beta"][0].double().numpy(),
                                        state0=d["state"].double().numpy(), seq_start=st)
    ref = torch.from_numpy(ref)
    tol = TOL[dt] + 3 * HALF[dt]
    assert rel(out[0], ref[cut]) < tol
    for i in range(steps):
        at = torch.tensor([t1 - steps + i for _, _, t1 in seqs])
        assert rel(outs[i], ref[at]) < tol, i
    assert rel(state, torch.from_numpy(ref_state)) < tol


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_gradient_through_the_layer(dtype):
    """chunk_bwd, then qk_norm_bwd, then three short_conv_bwd, against autograd of
    the front's definition fed with the oracle's gradients."""
    dt = DTYPES[dtype]
    lens = [50, 3, 41]
    p, d = prompt(lens, dt, 6)
    d["conv"] = [torch.zeros_like(c) for c in d["conv"]]
    say("layer: gradient", dtype)
    cu, seqs = offsets(lens).to(DEV), spans(1, None, lens)
    g = torch.Generator().manual_seed(1)
    d_out = torch.randn(1, sum(lens), H, D, generator=g).to(dt)
    q, k, v, _, raw = front(p, d, dt, cu)
    la, be, s0 = (d[n].to(DEV) for n in ("log_alpha", "beta", "state"))
    gr = kda.chunk_bwd(q, k, v.contiguous(), la, be, d_out.to(DEV), None, s0, cu)
    gn = kda.qk_norm_bwd(raw[0], raw[1], gr["dq"], gr["dk"], table=p["table"].to(DEV),
                         positions=d["pos"].to(DEV))
    rows = d["rows"].to(DEV)
    got = [kda.short_conv_bwd(rows[..., i * C:(i + 1) * C], p[n].to(DEV), dy.flatten(-2), p["b"].to(DEV),
                              None, d["conv"][i].to(DEV), cu)
           for i, (n, dy) in enumerate((("wq", gn["dq"]), ("wk", gn["dk"]), ("wv", gr["dv"])))]
    torch.cuda.synchronize()
    x = d["rows"].double().requires_grad_()
    w = {n: p[n].double().requires_grad_() for n in ("wq", "wk", "wv", "b")}
    qr, kr, vr = front_ref({**p, **w}, {**d, "rows": x}, seqs)
    n64 = lambda t: t[0].detach().numpy()
    og = oracle.kda_backward(n64(qr), n64(kr), n64(vr), n64(d["log_alpha"].double()),
                             n64(d["beta"].double()), n64(d_out.double()),
                             state0=d["state"].double().numpy(), seq_start=np.cumsum([0] + lens))
    up = [torch.from_numpy(og[n])[None] for n in ("dq", "dk", "dv")]
    ref = torch.autograd.grad([qr, kr, vr], [x, w["wq"], w["wk"], w["wv"], w["b"]], up)
    tol = TOL[dt] + 4 * HALF[dt]
    assert rel(torch.cat([t["dx"] for t in got], -1), ref[0][..., : 3 * C]) < tol
    for i in range(3):
        assert rel(got[i]["dweight"], ref[1 + i]) < tol, i
    assert rel(sum(t["dbias"] for t in got), ref[4]) < tol


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_convolution_into_the_scan(dtype):
    """One convolution over x | B | C, its output's slices into the scan, then one
    token more through both, and the gradient back to the projection's rows."""
    dt = DTYPES[dtype]
    G, P, N = 1, 64, 128
    ch = H * P + 2 * G * N
    lens = [90, 0, 70]
    say("layer: convolution into the scan", dtype)
    g = torch.Generator().manual_seed(8)
    r = lambda *s: torch.randn(s, generator=g)
    T, n = sum(lens), len(lens)
    rows, tok = r(1, T, ch).to(dt), r(n, ch).to(dt)
    w, b = r(ch, W) * 0.5, r(ch) * 0.1
    step, A, Dp = torch.nn.functional.softplus(r(1, T, H) - 2), -torch.rand(H, generator=g) * 4, r(H)
    step1 = torch.nn.functional.softplus(r(n, H) - 2)
    d_out = r(1, T, H, P).to(dt)
    cu, seqs = offsets(lens).to(DEV), spans(1, None, lens)
    split = lambda t: (t[..., : H * P].unflatten(-1, (H, P)),
                       t[..., H * P: H * P + G * N].unflatten(-1, (G, N)),
                       t[..., H * P + G * N:].unflatten(-1, (G, N)))
    dw, db, dA, dD, dstep = (t.to(DEV) for t in (w, b, A, Dp, step))
    y, conv = kda.short_conv(rows.to(DEV), dw, db, cu_seqlens=cu)
    x, B, Cc = split(y)  # slices of the convolution's rows
    out, state = kda.ssm_chunk_fwd(x, dstep, dA, B, Cc, dD, cu_seqlens=cu)
    kept = state.clone()
    y1 = kda.short_conv_step(tok.to(DEV), dw, conv, db)
    x1, B1, C1 = split(y1)
    out1 = kda.ssm_decode_step(x1, step1.to(DEV), dA, B1, C1, state, dD)
    back = torch.empty_like(y)
    dx, dB, dC = split(back)
    gs = kda.ssm_chunk_bwd(x, dstep, dA, B, Cc, d_out.to(DEV), dD, cu_seqlens=cu,
                           grads={"dx": dx, "dB": dB, "dC": dC})  # into one row again
    gc = kda.short_conv_bwd(rows.to(DEV), dw, back, db, cu_seqlens=cu)
    torch.cuda.synchronize()
    leaf = lambda t: t.double().requires_grad_()
    xr, wr, Ar = leaf(rows), leaf(w), leaf(A)
    yr, _ = conv_ref(xr, wr, b.double(), torch.zeros(n, W - 1, ch, dtype=torch.float64), "silu", seqs)
    a, Bm, Cm = split(yr)
    ref, ref_state = ssm_ref(a, step.double(), Ar, Bm, Cm, Dp.double(),
                             torch.zeros(n, H, P, N, dtype=torch.float64), seqs)
    gr = torch.autograd.grad(ref, [xr, wr, Ar], d_out.double())
    # two roundings to the type on the way forward, three on the way back
    assert rel(out, ref) < 2 * HALF[dt] + 1e-5
    assert rel(kept, ref_state) < HALF[dt] + 1e-5
    assert rel(gc["dx"], gr[0]) < 4 * HALF[dt] + 2e-5
    assert rel(gc["dweight"], gr[1]) < 4 * HALF[dt] + 2e-5
    assert rel(gs["dA"], gr[2]) < 4 * HALF[dt] + 1e-4
    # the token behind: its convolution sees the prompt's last rows
    long = torch.cat([torch.cat([rows[0, t0:t1], tok[i: i + 1]]) for i, (_, t0, t1) in enumerate(seqs)])
    seq1 = spans(1, None, [x + 1 for x in lens])
    yl, _ = conv_ref(long[None].double(), w.double(), b.double(),
                     torch.zeros(n, W - 1, ch, dtype=torch.float64), "silu", seq1)
    xs, Bs, Cs = split(yl)
    steps = torch.cat([torch.cat([step[0, t0:t1], step1[i: i + 1]]) for i, (_, t0, t1) in enumerate(seqs)])
    full, fin = ssm_ref(xs, steps[None].double(), A.double(), Bs, Cs, Dp.double(),
                        torch.zeros(n, H, P, N, dtype=torch.float64), seq1)
    last = torch.tensor([t1 - 1 for _, _, t1 in seq1])
    assert rel(out1, full[0, last]) < 2 * HALF[dt] + 1e-5
    assert rel(state, fin) < HALF[dt] + 1e-5
