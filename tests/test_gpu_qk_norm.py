"""GPU parity of the query/key norm with rotation (forward, backward) with its
64-bit definition, through the public calls.

Bounds, element by element, u = 2^-24, h = half a step of the output's type:
the sum of d squares is 8 terms in a chain and 4 levels of a tree after a
rounding each (13 u), its mean and eps 2 u, which the root halves; the root
itself 2 u, two products 2 u: under 13 u of |y|.  A rotated value is two
products and a sum of such: under 16 u (|y_a| + |y_b|).  Backward: g likewise
3 u (|dy_a| + |dy_b|); its product with w, the sum of d products (16 u of
sum |h x|), four more products, a difference: under 48 u inv (|h| + |x| inv^2
sum |h x| / m).
"""
import pytest
import torch

from layer_ref import DTYPES, HALF, U, qk_ref, within
from parity import say

import gated_delta_rule_81_amd as kda

DEV = "cuda:0"

CASES = [  # lead, hq, hk, d, kind, weight, rot, inter, pad, dtype
    ((1, 1), 1, 1, 64, "l2", False, 0, False, 0, "bf16"),
    ((3,), 4, 2, 128, "l2", True, 128, False, 0, "f32"),
    ((2, 37), 6, 2, 128, "rms", True, 64, False, 0, "bf16"),
    ((1, 50), 3, 1, 64, "rms", True, 16, True, 8, "bf16"),
    ((1, 19), 9, 0, 64, "rms", False, 48, False, 64, "f32"),
    ((1, 70), 33, 7, 128, "rms", True, 112, False, 8, "bf16"),
    ((2, 5), 2, 17, 128, "l2", False, 96, True, 0, "f32"),
    ((1, 600), 5, 5, 64, "rms", True, 64, True, 0, "f32"),
]


def make(case, seed=0):
    lead, hq, hk, d, kind, weight, rot, inter, pad, dtype = case
    dt, g = DTYPES[dtype], torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(s, generator=g)
    wide = r(*lead, (hq + hk) * d + pad).to(dt)
    if pad:
        wide[..., (hq + hk) * d:] = float("nan")
    cut = lambda t: (t[..., : hq * d].unflatten(-1, (hq, d)),
                     t[..., hq * d: (hq + hk) * d].unflatten(-1, (hk, d)))
    if hk == 0:
        cut = lambda t: (t[..., : hq * d].unflatten(-1, (hq, d)), t.new_empty(*lead, 0, d))
    q, k = cut(wide)
    dq, dk = r(*lead, hq, d).to(dt), r(*lead, hk, d).to(dt)
    wq, wk = (r(d) + 1.0, r(d) + 1.0) if weight else (None, None)
    table = pos = None
    if rot:
        a = torch.arange(99, dtype=torch.float64)[:, None] * 2.0 ** -torch.arange(rot // 2)
        table = torch.cat([a.cos(), a.sin()], -1).float()
        pos = torch.randint(0, 99, lead, generator=g, dtype=torch.int32)
    qd, kd = cut(wide.to(DEV))
    to = lambda v: None if v is None else v.to(DEV)
    dev = dict(q=qd, k=kd, dq=to(dq), dk=to(dk), wq=to(wq), wk=to(wk), table=to(table), pos=to(pos))
    f = lambda v: None if v is None else v.double()
    ref = dict(q=f(q), k=f(k), dq=f(dq), dk=f(dk), wq=f(wq), wk=f(wk), table=f(table), pos=pos)
    return dev, ref


def turned_abs(y, table, rot, inter):
    """|y_a| + |y_b| for rotated channels, |y| for the others."""
    y = y.abs()
    if table is None:
        return y
    half = rot // 2
    i = torch.arange(half)
    a, b = (2 * i, 2 * i + 1) if inter else (i, i + half)
    out = y.clone()
    out[..., a] = out[..., b] = y[..., a] + y[..., b]
    return out


@pytest.mark.gpu
@pytest.mark.parametrize("case", CASES, ids=str)
def test_forward(case):
    kind, rot, inter, dt = case[4], case[6], case[7], DTYPES[case[9]]
    dev, ref = make(case)
    say("qk_norm", case)
    got = kda.qk_norm(dev["q"], dev["k"], dev["wq"], dev["wk"], dev["table"], dev["pos"],
                      kind=kind, interleaved=inter)
    torch.cuda.synchronize()
    for name, y in zip("qk", got):
        x, w = ref[name], ref["w" + name]
        want = qk_ref(x, w, ref["table"], ref["pos"], kind, 1e-6, inter)
        flat = qk_ref(x, w, None, None, kind, 1e-6, inter)
        m = turned_abs(flat, ref["table"], rot, inter)
        within(y, want, HALF[dt] * want.abs() + 16 * U * m * (1 + HALF[dt]), name)


@pytest.mark.gpu
@pytest.mark.parametrize("case", CASES, ids=str)
def test_backward(case):
    lead, hq, hk, d, kind, weight, rot, inter, pad, dtype = case
    dt = DTYPES[dtype]
    dev, ref = make(case, 1)
    say("qk_norm_bwd", case)
    g = kda.qk_norm_bwd(dev["q"], dev["k"], dev["dq"], dev["dk"], dev["wq"], dev["wk"],
                        dev["table"], dev["pos"], kind=kind, interleaved=inter)
    torch.cuda.synchronize()
    for name in "qk":
        x = ref[name].clone().requires_grad_()
        w = None if ref["w" + name] is None else ref["w" + name].clone().requires_grad_()
        dy = ref["d" + name]
        y = qk_ref(x, w, ref["table"], ref["pos"], kind, 1e-6, inter)
        if not x.numel():
            assert g["d" + name].numel() == 0
            continue
        want = torch.autograd.grad(y, [x] + ([] if w is None else [w]), dy)
        m = 1 if kind == "l2" else d
        x = x.detach()
        inv = 1 / torch.sqrt((x * x).sum(-1, keepdim=True) / m + 1e-6)
        ga = turned_abs(dy, ref["table"], rot, inter)
        ha = ga if w is None else ga * w.detach().abs()
        mag = inv * (ha + x.abs() * inv ** 2 * (ha * x.abs()).sum(-1, keepdim=True) / m)
        h = HALF[dt]
        within(g["d" + name], want[0], h * want[0].abs() + 48 * U * mag * (1 + h), "d" + name)
        if w is None:
            assert g["d" + name + "_weight"] is None
        else:
            n = x.numel() // d  # additions on one value's way: at most one per head
            tot = (ga * x.abs() * inv).reshape(-1, d).sum(0)
            within(g["d" + name + "_weight"], want[1], (n + 20) * U * tot, "dw")


def test_reference_gradient_by_differences():
    g = torch.Generator().manual_seed(3)
    r = lambda *s: torch.randn(s, generator=g, dtype=torch.float64).requires_grad_()
    a = torch.arange(5, dtype=torch.float64)[:, None] * torch.tensor([1.0, 0.3])
    table, pos = torch.cat([a.cos(), a.sin()], -1), torch.tensor([[3, 0, 4]])
    for kind, inter in (("l2", False), ("rms", True)):
        f = lambda x, w: qk_ref(x, w, table, pos, kind, 1e-6, inter)
        assert torch.autograd.gradcheck(f, (r(1, 3, 2, 8), r(8)))


@pytest.mark.gpu
def test_positions_outside_the_table_are_moved_into_it():
    say("qk_norm: positions outside the table")
    q = torch.randn(1, 4, 2, 64, device=DEV)
    t = torch.randn(10, 32, device=DEV)
    pos = torch.tensor([[-5, 0, 9, 2 ** 31 - 1]], dtype=torch.int32, device=DEV)
    got = kda.qk_norm(q, q.clone(), table=t, positions=pos)
    want = kda.qk_norm(q, q.clone(), table=t, positions=pos.clamp(0, 9))
    torch.cuda.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


@pytest.mark.gpu
def test_zero_rows_and_no_eps():
    """A head of zeros gives zeros (and its gradient dy / sqrt(eps)); with
    eps = 0 only that head's own values are lost, not the weights' gradient of a
    batch whose last pass is not full."""
    say("qk_norm: rows of zeros")
    q = torch.randn(1, 3, 3, 64, device=DEV)
    q[0, 1, 1] = 0
    y, _ = kda.qk_norm(q, q.clone(), kind="rms")
    d = torch.randn_like(q)
    w = torch.ones(64, device=DEV)
    g = kda.qk_norm_bwd(q, q.clone(), d, d.clone(), w, w.clone(), kind="l2")
    clean = torch.randn(1, 1, 3, 64, device=DEV)
    g0 = kda.qk_norm_bwd(clean, clean.clone(), clean * 2, clean * 2, w, w.clone(), eps=0.0)
    torch.cuda.synchronize()
    assert (y[0, 1, 1] == 0).all() and torch.isfinite(y).all()
    # 1 / sqrt(1e-6), one product: 3 u
    assert torch.allclose(g["dq"][0, 1, 1].double(), d[0, 1, 1].double() / 1e-6 ** 0.5, rtol=6 * U)
    assert torch.isfinite(g0["dq_weight"]).all() and torch.isfinite(g0["dq"]).all()


@pytest.mark.gpu
def test_captured_and_replayed():
    say("qk_norm: graph")
    q, k = torch.randn(1, 70, 8, 128, device=DEV).bfloat16(), torch.randn(1, 70, 2, 128, device=DEV).bfloat16()
    w = torch.randn(128, device=DEV)
    t = torch.randn(100, 64, device=DEV)
    pos = torch.arange(70, dtype=torch.int32, device=DEV)[None]

    def both():
        y = kda.qk_norm(q, k, w, w.clone(), t, pos, kind="rms")
        g = kda.qk_norm_bwd(q, k, y[0], y[1], w, w.clone(), t, pos, kind="rms")
        return [*y, g["dq"], g["dk"], g["dq_weight"], g["dk_weight"]]

    both()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = both()
    for i in range(3):
        q.copy_(torch.randn_like(q))
        graph.replay()
        torch.cuda.synchronize()
        want = both()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want)), i
