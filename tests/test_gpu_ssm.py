"""GPU parity of the state space scan (prompts, single tokens) with its 64-bit
definition, through the public calls.

Bounds, element by element, u = 2^-24, h = half a step of the output's type.
Every output is a sum of products; mag is the same sum over absolute values
(the definition run on |x|, |B|, |C|, |D|, |state|).  Relative to mag:
  sums of at most 64 tokens and 128 channels in fp32: 200 u;
  a decay e^z, z <= 0: its exponent is a difference of fp64 sums rounded once
    (|z| u relative) and exp2 is good to 2 u; decays under e^-104 are nothing in
    fp32, so 106 u each;
  the state from block to block: 3 u a block (decay 2, sum 1), and one more
    decay where pieces are joined;
  bf16 inputs: the state and the block's weights enter y's products as two bf16
    parts, off by 2^-7 2^-8 each; the rest (fp32 inputs, states) as three, which
    leave under 4 u.
"""
import pytest
import torch

from layer_ref import DTYPES, HALF, U, offsets, spans, ssm_ref, within
from parity import say

import gated_delta_rule_81_amd as kda

DEV = "cuda:0"

CASES = [  # batch, seq_len, lens, H, G, P, N, state, skip, pad, dtype, decay
    (1, 1, None, 1, 1, 64, 64, True, True, 0, "bf16", 1.0),
    (2, 64, None, 2, 1, 64, 128, True, False, 0, "bf16", 1.0),
    (1, 65, None, 3, 3, 128, 64, False, True, 8, "bf16", 1.0),
    (1, 130, None, 4, 2, 128, 128, True, True, 0, "bf16", 8.0),
    (1, 33, None, 2, 2, 64, 64, True, True, 0, "f32", 1.0),
    (2, 97, None, 2, 1, 128, 128, True, True, 4, "f32", 8.0),
    (1, 31, None, 2, 1, 128, 64, False, False, 0, "f32", 1.0),
    (1, 0, [0, 1, 63, 64, 65, 0, 17, 0], 2, 1, 64, 128, True, True, 0, "bf16", 1.0),
    (1, 0, [0, 1, 63, 64, 65, 0, 17, 0], 2, 1, 64, 128, True, True, 0, "f32", 1.0),
    # cut into pieces of 256 tokens
    (1, 700, None, 2, 1, 64, 64, True, True, 0, "bf16", 1.0),
    (2, 513, None, 1, 1, 128, 128, False, True, 0, "f32", 1.0),
    (1, 0, [300, 0, 257, 2, 511, 256, 0], 2, 2, 64, 128, True, True, 0, "bf16", 1.0),
    (1, 0, [700, 1, 300], 1, 1, 64, 64, True, False, 0, "f32", 0.1),
    # heads of 64 rows, two a workgroup: three pairs a group, and no pairs in a group of three
    (1, 0, [130, 0, 1, 260, 15], 12, 2, 64, 128, True, True, 8, "bf16", 1.0),
    (1, 300, None, 6, 2, 64, 64, True, True, 0, "bf16", 8.0),
    (1, 449, None, 3, 1, 128, 128, True, False, 0, "bf16", 0.1),
]


def make(case, seed=0):
    batch, T, lens, H, G, P, N, state, skip, pad, dtype, decay = case
    dt_, g = DTYPES[dtype], torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(s, generator=g)
    T = sum(lens) if lens is not None else T
    n = len(lens) if lens is not None else batch
    wide = r(batch, T, H * P + 2 * G * N + pad).to(dt_)
    if pad:
        wide[..., H * P + 2 * G * N:] = float("nan")
    cut = lambda w: dict(x=w[..., : H * P].unflatten(-1, (H, P)),
                         B=w[..., H * P: H * P + G * N].unflatten(-1, (G, N)),
                         C=w[..., H * P + G * N: H * P + 2 * G * N].unflatten(-1, (G, N)))
    if not pad:
        cut0 = cut
        cut = lambda w: {k: v.contiguous() for k, v in cut0(w).items()}
    rest = dict(dt=torch.nn.functional.softplus(r(batch, T, H) - 3),
                A=-(torch.rand(H, generator=g) * 4 + 0.5) * decay, D=r(H) if skip else None,
                state=r(n, H, P, N) if state else None)
    rest["dt"][:, ::7] = 0  # tokens that leave the state as it is
    f = {k: None if v is None else v.double() for k, v in {**cut(wide), **rest}.items()}
    dev = {**cut(wide.to(DEV)), **{k: None if v is None else v.to(DEV) for k, v in rest.items()}}
    dev["cu"] = offsets(lens).to(DEV) if lens is not None else None
    f["seqs"] = spans(batch, T, lens)
    if f["state"] is None:
        f["state"] = torch.zeros(n, H, P, N, dtype=torch.float64)
    return dev, f


def magnitudes(f):
    return ssm_ref(f["x"].abs(), f["dt"], f["A"], f["B"].abs(), f["C"].abs(),
                   None if f["D"] is None else f["D"].abs(), f["state"].abs(), f["seqs"])


def factors(dt, blocks):
    """Relative to mag: (of y, of the state)."""
    state = (64 + 2 * 106 + 4 + 3 * blocks) * U
    y = (200 + 4 * 106 + 8 + 3 * blocks) * U
    return (y + (2 * 2.0 ** -15 if dt == torch.bfloat16 else 0)), state


@pytest.mark.gpu
@pytest.mark.parametrize("case", CASES, ids=str)
def test_forward(case):
    dt = DTYPES[case[10]]
    dev, f = make(case)
    say("ssm_chunk_fwd", case)
    out, fin = kda.ssm_chunk_fwd(dev["x"], dev["dt"], dev["A"], dev["B"], dev["C"], dev["D"],
                                 dev["state"], dev["cu"])
    torch.cuda.synchronize()
    ref, ref_fin = ssm_ref(f["x"], f["dt"], f["A"], f["B"], f["C"], f["D"], f["state"], f["seqs"])
    m, m_fin = magnitudes(f)
    fy, fs = factors(dt, f["x"].shape[1] // 32 + 1)
    h = HALF[dt]
    within(fin, ref_fin, fs * m_fin + 1e-37, "final state")
    within(out, ref, h * ref.abs() + fy * (1 + h) * m + 1e-37, "out")


BWD_CASES = CASES + [
    # several sets of a group's heads, their parts of dB and dC summed
    (1, 200, None, 7, 1, 64, 64, True, True, 0, "bf16", 1.0),
    (1, 0, [40, 0, 70], 6, 2, 128, 128, True, True, 8, "f32", 1.0),
]


def grad_magnitudes(f, d_out, d_final):
    """The gradients' sums over absolute values: autograd of the definition on
    |x|, |B|, |C|, |D|, |state|, |d_out|, |d_final| with the decays' own signs
    turned so that every path adds (dA, ddt: |x . du| + |A| dl)."""
    ab = lambda v: None if v is None else v.abs().requires_grad_()
    x, B, C, D, st = ab(f["x"]), ab(f["B"]), ab(f["C"]), ab(f["D"]), ab(f["state"])
    # decay and input weight apart: exp(-(dt |A|)) enters with a slope of its own
    dt_in, dt_l = f["dt"].clone().requires_grad_(), f["dt"].clone().requires_grad_()
    A = f["A"].clone().requires_grad_()
    l = dt_l * A
    ones = torch.ones_like(f["A"])
    y, fin = ssm_ref(x * dt_in[..., None], l, ones, B / 1.0, C, None, st, f["seqs"], raw=True)
    if D is not None:
        y = y + D[:, None] * x
    leaves = [x, dt_in, dt_l, A, B, C, st] + ([] if D is None else [D])
    g = torch.autograd.grad([y, fin], leaves, [d_out.abs(), d_final.abs()])
    out = dict(dx=g[0], ddt=g[1] + g[2].abs(), dA=g[3].abs(), dB=g[4], dC=g[5], d_initial_state=g[6])
    out["dD"] = None if D is None else g[7]
    return out


@pytest.mark.gpu
@pytest.mark.parametrize("case", BWD_CASES, ids=str)
def test_backward(case):
    """Each gradient against autograd of the definition.  Its products chain two
    block sums (G with dP, M with dy, the states with dy or x), each as the
    forward's: twice the forward's factors; bf16 dB and dC take Q as two bf16
    parts (2^-15)."""
    dt = DTYPES[case[10]]
    dev, f = make(case, 2)
    g = torch.Generator().manual_seed(77)
    d_out = torch.randn(f["x"].shape, generator=g).to(dt)
    d_fin = torch.randn(f["state"].shape, generator=g) if case[7] else None
    say("ssm_chunk_bwd", case)
    got = kda.ssm_chunk_bwd(dev["x"], dev["dt"], dev["A"], dev["B"], dev["C"], d_out.to(DEV),
                            dev["D"], None if d_fin is None else d_fin.to(DEV), dev["state"], dev["cu"])
    torch.cuda.synchronize()
    leaf = lambda k: None if f[k] is None else f[k].clone().requires_grad_()
    names = ["x", "dt", "A", "B", "C", "state"] + ([] if f["D"] is None else ["D"])
    v = {k: leaf(k) for k in ("x", "dt", "A", "B", "C", "D", "state")}
    y, fin = ssm_ref(v["x"], v["dt"], v["A"], v["B"], v["C"], v["D"], v["state"], f["seqs"])
    df = torch.zeros_like(fin) if d_fin is None else d_fin.double()
    ref = dict(zip(names, torch.autograd.grad([y, fin], [v[k] for k in names], [d_out.double(), df])))
    mag = grad_magnitudes(f, d_out.double(), df)
    blocks = f["x"].shape[1] // 32 + 1
    _, fs = factors(torch.float32, blocks)
    fy, _ = factors(torch.float32, blocks)
    h = HALF[dt]
    for name, key in (("dx", "x"), ("ddt", "dt"), ("dA", "A"), ("dB", "B"), ("dC", "C"),
                      ("dD", "D"), ("d_initial_state", "state")):
        if ref.get(key) is None:
            assert got[name] is None
            continue
        rounded = name in ("dx", "dB", "dC")
        two = 2 * 2.0 ** -15 if name in ("dB", "dC") and dt == torch.bfloat16 else 0
        bound = (2 * fy + two) * mag[name] * (1 + h) + (h * ref[key].abs() if rounded else 0) + 1e-37
        within(got[name], ref[key], bound, name)


def test_reference_gradient_by_differences():
    """The 64-bit reference's gradient against central differences."""
    g = torch.Generator().manual_seed(3)
    r = lambda *s: torch.randn(s, generator=g, dtype=torch.float64).requires_grad_()
    seqs = spans(1, 6, [3, 0, 1, 2])
    dt = (torch.rand(1, 6, 2, generator=g, dtype=torch.float64) + 0.1).requires_grad_()
    f = lambda x, t, A, B, C, D, s: ssm_ref(x, t, -A.abs(), B, C, D, s, seqs)
    assert torch.autograd.gradcheck(f, (r(1, 6, 2, 3), dt, r(2), r(1, 6, 1, 2), r(1, 6, 1, 2), r(2),
                                        r(4, 2, 3, 2)))


@pytest.mark.gpu
def test_far_decays():
    """Steps of e^-1000 and e^-1e30 between ordinary ones: what lies before them
    is forgotten, and what comes after is as exact as without them."""
    dev, f = make((1, 150, None, 2, 1, 64, 64, True, True, 0, "f32", 1.0), 5)
    for t, v in ((5, 1e3), (40, 1e30), (41, 0.0), (70, 3e5), (140, 1e3)):
        dev["dt"][0, t] = v
        f["dt"][0, t] = float(torch.tensor(v, dtype=torch.float32))
    f["x"][0, :, :] = dev["x"][0].double().cpu()
    for t in (5, 40, 70, 140):  # their own input at an ordinary size
        dev["x"][0, t] /= dev["dt"][0, t, 0]
        f["x"][0, t] = dev["x"][0, t].double().cpu()
    say("ssm_chunk_fwd: far decays")
    out, fin = kda.ssm_chunk_fwd(dev["x"], dev["dt"], dev["A"], dev["B"], dev["C"], dev["D"],
                                 dev["state"])
    torch.cuda.synchronize()
    ref, ref_fin = ssm_ref(f["x"], f["dt"], f["A"], f["B"], f["C"], f["D"], f["state"], f["seqs"])
    m, m_fin = magnitudes(f)
    fy, fs = factors(torch.float32, 5)
    # inputs of 1e-30 lose their last bf16 part to fp32's own small end: one part in 2^-16
    within(fin, ref_fin, fs * m_fin + 1e-30, "final state")
    within(out, ref, fy * 2 * m + 1e-30, "out")


@pytest.mark.gpu
@pytest.mark.parametrize("B,H,G,P,N,skip,dtype", [(1, 1, 1, 64, 64, True, "bf16"),
                                                  (3, 6, 2, 64, 128, False, "f32"),
                                                  (2, 3, 1, 128, 64, True, "f32"),
                                                  (150, 4, 4, 128, 128, True, "bf16")])
def test_step(B, H, G, P, N, skip, dtype):
    """One token against the definition: a product, a sum, the decay, then a sum
    of N products: under 200 u of the sum of absolute values."""
    dt, g = DTYPES[dtype], torch.Generator().manual_seed(B)
    r = lambda *s: torch.randn(s, generator=g)
    x, Bt, Ct = r(B, H, P).to(dt), r(B, G, N).to(dt), r(B, G, N).to(dt)
    step, A, D = torch.nn.functional.softplus(r(B, H)), -torch.rand(H, generator=g) * 4, r(H)
    st = r(B, H, P, N)
    say("ssm_decode_step", B, H, G, P, N, dtype)
    dst = st.to(DEV)
    y = kda.ssm_decode_step(x.to(DEV), step.to(DEV), A.to(DEV), Bt.to(DEV), Ct.to(DEV), dst,
                            D.to(DEV) if skip else None)
    torch.cuda.synchronize()
    d = lambda v: v.double()
    args = lambda f: (f(d(x))[:, None], d(step)[:, None], d(A), f(d(Bt))[:, None],
                      f(d(Ct))[:, None], f(d(D)) if skip else None, f(d(st)), spans(B, 1, None))
    ref, ref_st = ssm_ref(*args(lambda v: v))
    m, m_st = ssm_ref(*args(torch.abs))
    h = HALF[dt]
    within(dst, ref_st, 40 * U * m_st, "state")
    within(y, ref[:, 0], h * ref[:, 0].abs() + 240 * U * m[:, 0] * (1 + h), "out")


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_prompt_then_tokens(dtype):
    """A prompt cut in two calls and single tokens after it give the whole
    prompt's outputs and state, within the two sides' bounds."""
    case = (2, 140, None, 4, 2, 64, 128, True, True, 0, dtype, 1.0)
    dev, f = make(case, 9)
    say("ssm: prompt, prompt, tokens", dtype)
    cut = lambda a, b: [dev[k][:, a:b].contiguous() for k in ("x", "dt", "B", "C")]
    o1, s1 = kda.ssm_chunk_fwd(*(lambda x, t, B, C: (x, t, dev["A"], B, C))(*cut(0, 70)),
                               dev["D"], dev["state"])
    x, t, B, C = cut(70, 130)
    o2, s2 = kda.ssm_chunk_fwd(x, t, dev["A"], B, C, dev["D"], s1, final_state=s1)  # in place
    assert s2.data_ptr() == s1.data_ptr()
    toks = []
    for i in range(130, 140):
        toks.append(kda.ssm_decode_step(dev["x"][:, i], dev["dt"][:, i].contiguous(), dev["A"],
                                        dev["B"][:, i], dev["C"][:, i], s1, dev["D"]))
    torch.cuda.synchronize()
    ref, ref_fin = ssm_ref(f["x"], f["dt"], f["A"], f["B"], f["C"], f["D"], f["state"], f["seqs"])
    m, m_fin = magnitudes(f)
    fy, fs = factors(DTYPES[dtype], 20)
    h = HALF[DTYPES[dtype]]
    got = torch.cat([o1, o2, torch.stack(toks, 1)], 1)
    within(got, ref, h * ref.abs() + fy * (1 + h) * m, "out")
    within(s1, ref_fin, 2 * fs * m_fin, "state")


@pytest.mark.gpu
@pytest.mark.parametrize("case", [CASES[9], CASES[11], CASES[3], CASES[13], CASES[14]], ids=str)
def test_state_updated_in_place(case):
    """final_state = initial_state, in one piece and in several (whose first and
    last workgroups both use the state): the bits of the call with two buffers."""
    say("ssm_chunk_fwd in place", case)
    dev, _ = make(case, 4)
    args = (dev["x"], dev["dt"], dev["A"], dev["B"], dev["C"], dev["D"])
    want, fin = kda.ssm_chunk_fwd(*args, dev["state"], dev["cu"])
    st = dev["state"].clone()
    out, got = kda.ssm_chunk_fwd(*args, st, dev["cu"], final_state=st)
    torch.cuda.synchronize()
    assert got.data_ptr() == st.data_ptr()
    assert torch.equal(out, want) and torch.equal(st, fin)


@pytest.mark.gpu
def test_tokens_behind_the_last_sequence_stay():
    say("ssm_chunk_fwd: tokens behind the last offset")
    dev, _ = make((1, 0, [100, 30], 2, 1, 64, 64, True, True, 0, "bf16", 1.0))
    cu = torch.tensor([0, 60, 101], dtype=torch.int32, device=DEV)
    out = torch.full_like(dev["x"], 7.0)
    args = (dev["dt"], dev["A"], dev["B"], dev["C"], dev["D"], dev["state"], cu)
    kda.ssm_chunk_fwd(dev["x"], *args, out=out)
    cutx = [dev[k][:, :101].contiguous() for k in ("x", "dt", "B", "C")]
    ref, _ = kda.ssm_chunk_fwd(cutx[0], cutx[1], dev["A"], cutx[2], cutx[3], dev["D"], dev["state"], cu)
    torch.cuda.synchronize()
    assert (out[:, 101:] == 7).all() and torch.equal(out[:, :101], ref)


@pytest.mark.gpu
def test_two_streams_and_a_graph():
    """Two calls at once on two streams (a workspace each), and a captured call
    replayed with eager work between, all with the eager result."""
    say("ssm_chunk_fwd: streams and graph")
    sets = [make((1, 700, None, 2, 1, 64, 128, True, True, 0, "bf16", 1.0), s)[0] for s in (1, 2)]
    run = lambda d: kda.ssm_chunk_fwd(d["x"], d["dt"], d["A"], d["B"], d["C"], d["D"], d["state"])
    want = [run(d) for d in sets]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = []
    for d, s in zip(sets, streams):
        with torch.cuda.stream(s):
            got.append(run(d))
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    d = sets[0]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = run(d)
        st = d["state"].clone()
        y = kda.ssm_decode_step(d["x"][:, 5], d["dt"][:, 5].contiguous(), d["A"], d["B"][:, 5],
                                d["C"][:, 5], st, d["D"])
    for i in range(3):
        d["x"].copy_(torch.randn_like(d["x"]))
        graph.replay()
        torch.cuda.synchronize()
        eager = run(d)
        st2 = d["state"].clone()
        y2 = kda.ssm_decode_step(d["x"][:, 5], d["dt"][:, 5].contiguous(), d["A"], d["B"][:, 5],
                                 d["C"][:, 5], st2, d["D"])
        torch.cuda.synchronize()
        for a, b in zip((*out, st, y), (*eager, st2, y2)):
            assert torch.equal(a, b), i
