"""The operators around the recurrence where sizes change what runs: long runs of
tokens in the convolution, several rounds of the norm's gradient, several launches
of the norm, and tensors of more than 2^31 elements.

A value's own arithmetic does not depend on how a call is cut, so outputs that are
no sums over tokens have the bits of a call on a part of the tensor (small calls
are held to the 64-bit definition in the operators' own modules); gradients of
weights are sums in another order, and the scan joins its pieces elsewhere.
"""
import pytest
import torch

import test_gpu_qk_norm
from layer_ref import DTYPES, HALF, U, offsets, rel
from parity import say

import gated_delta_rule_81_amd as kda

DEV = "cuda:0"


def randn(gen, *shape, dtype=torch.float32):
    return torch.empty(shape, dtype=dtype, device=DEV).normal_(generator=gen)


@pytest.mark.gpu
@pytest.mark.parametrize("C,W,lens,dtype", [
    (65536, 4, [700, 0, 1, 37, 1262], "bf16"),   # forward runs of 32 tokens, backward of 64
    (16384, 3, [2000], "bf16"),                  # 8 and 64
    (131072, 2, [1, 2, 3, 600, 0], "f32"),       # 40 and 64
    (5001, 4, [1024, 3, 900], "f32"),            # one channel a lane: 24 and 64
])
def test_convolution_in_long_runs(C, W, lens, dtype):
    dt, g = DTYPES[dtype], torch.Generator(device=DEV).manual_seed(1)
    T, n = sum(lens), len(lens)
    x, d_out = randn(g, 1, T, C, dtype=dt), randn(g, 1, T, C, dtype=dt)
    w, b = randn(g, C, W), randn(g, C)
    st, d_fin = randn(g, n, W - 1, C, dtype=dt), randn(g, n, W - 1, C, dtype=dt)
    cu = offsets(lens).to(DEV)
    say("short_conv: long runs", C, W, lens, dtype)
    out, fin = kda.short_conv(x, w, b, st, cu)
    gr = kda.short_conv_bwd(x, w, d_out, b, d_fin, st, cu)
    for c0 in (0, C // 2, C - 8):
        c = lambda t: t[..., c0: c0 + 8].contiguous()
        wp, bp = w[c0: c0 + 8].contiguous(), b[c0: c0 + 8].contiguous()
        o, f = kda.short_conv(c(x), wp, bp, c(st), cu)
        p = kda.short_conv_bwd(c(x), wp, c(d_out), bp, c(d_fin), c(st), cu)
        torch.cuda.synchronize()
        assert torch.equal(c(out), o) and torch.equal(c(fin), f), c0
        assert torch.equal(c(gr["dx"]), p["dx"]), c0
        assert torch.equal(c(gr["d_initial_state"]), p["d_initial_state"]), c0
        # additions on one value's way on either side; silu's slope is under 1.1
        chain = 64 + 4 + 16 + T // 64
        total = 1.1 * c(d_out).double().abs().sum((0, 1))
        top = torch.cat([c(x).flatten(0, 1), c(st).flatten(0, 1)]).double().abs().amax(0)
        off = (gr["dweight"][c0: c0 + 8] - p["dweight"]).abs().double()
        assert (off <= (2 * chain * U * total * top)[:, None]).all(), c0
        assert ((gr["dbias"][c0: c0 + 8] - p["dbias"]).abs() <= 2 * chain * U * total).all(), c0


@pytest.mark.gpu
@pytest.mark.parametrize("case", [((1, 5000), 3, 1, 64, "rms", True, 64, False, 0, "f32"),
                                  ((2, 3000), 9, 4, 128, "l2", True, 128, True, 8, "bf16")], ids=str)
def test_norm_gradient_in_several_rounds(case):
    """More units of work than the workgroups of the gradient take at once."""
    test_gpu_qk_norm.test_backward(case)


@pytest.mark.gpu
def test_norm_in_several_launches():
    """2^25 + 9 tokens of one head: two launches, and offsets past 2^31 elements."""
    say("qk_norm: two launches")
    g = torch.Generator(device=DEV).manual_seed(2)
    q = randn(g, (1 << 25) + 9, 1, 64, dtype=torch.bfloat16)
    k = q.new_empty(q.shape[0], 0, 64)
    y, _ = kda.qk_norm(q, k)
    for part in (slice(0, 5), slice((1 << 25) - 3, (1 << 25) + 9)):
        want, _ = kda.qk_norm(q[part].contiguous(), k[part].contiguous())
        torch.cuda.synchronize()
        assert torch.equal(y[part], want)


@pytest.mark.gpu
def test_convolution_past_32_bit_offsets():
    """70,000 rows of 65,536 channels, 4.6e9 values."""
    say("short_conv: offsets past 32 bits")
    g = torch.Generator(device=DEV).manual_seed(3)
    T, C, tail = 70000, 65536, 90
    x = randn(g, 1, T, C, dtype=torch.bfloat16)
    w = randn(g, C, 4)
    out, fin = kda.short_conv(x, w)
    before = x[:, T - tail - 3: T - tail].contiguous()
    last = x[:, T - tail:].contiguous()
    o, f = kda.short_conv(last, w, None, before)
    torch.cuda.synchronize()
    assert torch.equal(out[:, T - tail:], o) and torch.equal(fin, f)
    gr = kda.short_conv_bwd(x, w, out, output_initial_state_grad=False)  # out as its own gradient
    p = kda.short_conv_bwd(last, w, o, None, None, before)
    torch.cuda.synchronize()
    assert torch.equal(gr["dx"][:, T - tail:], p["dx"])


@pytest.mark.gpu
def test_scan_past_32_bit_offsets():
    """270,000 tokens of 128 heads of 64, 2.2e9 values: the last tokens against a
    call of their own that goes on from the state before them.  Both round the
    same numbers, off by a few fp32 roundings, once."""
    say("ssm: offsets past 32 bits")
    g = torch.Generator(device=DEV).manual_seed(4)
    T, H, G, P, N, tail = 270000, 128, 2, 64, 64, 150
    x = randn(g, 1, T, H, P, dtype=torch.bfloat16)
    B, C = randn(g, 1, T, G, N, dtype=torch.bfloat16), randn(g, 1, T, G, N, dtype=torch.bfloat16)
    dt = torch.nn.functional.softplus(randn(g, 1, T, H) - 3)
    A = -torch.rand(H, device=DEV, generator=g) - 0.5
    out, fin = kda.ssm_chunk_fwd(x, dt, A, B, C)
    cut = lambda t: t[:, : T - tail].contiguous()
    end = lambda t: t[:, T - tail:].contiguous()
    _, state = kda.ssm_chunk_fwd(cut(x), cut(dt), A, cut(B), cut(C))
    o, f = kda.ssm_chunk_fwd(end(x), end(dt), A, end(B), end(C), None, state)
    torch.cuda.synchronize()
    h = HALF[torch.bfloat16]
    assert rel(end(out), o.double().cpu()) < 2 * h and rel(fin, f.double().cpu()) < 1e-5
    gr = kda.ssm_chunk_bwd(x, dt, A, B, C, x, output_initial_state_grad=False)
    p = kda.ssm_chunk_bwd(end(x), end(dt), A, end(B), end(C), end(x), None, None, state)
    torch.cuda.synchronize()
    for k in ("dx", "dB", "dC"):
        assert rel(end(gr[k]), p[k].double().cpu()) < 2 * h, k
    assert rel(end(gr["ddt"]), p["ddt"].double().cpu()) < 1e-4


@pytest.mark.gpu
def test_steps_past_32_bit_offsets():
    """1,400 sessions of 96 heads of 128 x 128: 2.2e9 values of state."""
    say("ssm_decode_step: offsets past 32 bits")
    g = torch.Generator(device=DEV).manual_seed(5)
    n, H, G, P, N = 1400, 96, 8, 128, 128
    st = randn(g, n, H, P, N)
    x, B, C = (randn(g, n, *s, dtype=torch.bfloat16) for s in ((H, P), (G, N), (G, N)))
    dt, A = torch.rand(n, H, device=DEV, generator=g), -torch.rand(H, device=DEV, generator=g)
    s = lambda t: t[n - 2:].clone()
    own = s(st)
    y = kda.ssm_decode_step(x, dt, A, B, C, st)
    want = kda.ssm_decode_step(s(x), s(dt), A, s(B), s(C), own)
    torch.cuda.synchronize()
    assert torch.equal(y[n - 2:], want) and torch.equal(st[n - 2:], own)


@pytest.mark.gpu
def test_scan_gradient_captured_and_on_two_streams():
    """ssm_chunk_bwd in a graph, replayed with eager work between, and two calls at
    once on two streams with a workspace each: the bits of the eager call."""
    say("ssm_chunk_bwd: graph and streams")

    def inputs(seed):
        g = torch.Generator(device=DEV).manual_seed(seed)
        T, H, G, P, N = 500, 6, 2, 64, 128
        r = lambda *s: randn(g, 1, T, *s, dtype=torch.bfloat16)
        return dict(x=r(H, P), dt=torch.rand(1, T, H, device=DEV, generator=g) * 0.1,
                    A=-torch.rand(H, device=DEV, generator=g), B=r(G, N), C=r(G, N), d_out=r(H, P),
                    D=randn(g, H), d_final_state=randn(g, 2, H, P, N),
                    initial_state=randn(g, 2, H, P, N), cu_seqlens=offsets([420, 80]).to(DEV))

    sets = [inputs(s) for s in (1, 2)]
    want = [kda.ssm_chunk_bwd(**d) for d in sets]
    torch.cuda.synchronize()
    got = []
    for d, s in zip(sets, [torch.cuda.Stream(), torch.cuda.Stream()]):
        with torch.cuda.stream(s):
            got.append(kda.ssm_chunk_bwd(**d))
    torch.cuda.synchronize()
    same = lambda a, b: all(torch.equal(a[k], b[k]) for k in a)
    assert same(got[0], want[0]) and same(got[1], want[1])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = kda.ssm_chunk_bwd(**sets[0])
    for i in range(3):
        sets[0]["x"].copy_(torch.randn_like(sets[0]["x"]))
        graph.replay()
        torch.cuda.synchronize()
        eager = kda.ssm_chunk_bwd(**sets[0])
        torch.cuda.synchronize()
        assert same(held, eager), i
