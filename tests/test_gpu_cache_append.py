"""GPU parity of the append to a paged cache with its 64-bit definition, through the
public call.

Bound, element by element, u = 2^-24, h = half a step of the type: a rotated value
is two products and their sum, 3 u (|a| + |b|), then rounded once; everything
else is copied, bit for bit, and no other place of the cache changes.
"""
import pytest
import torch

from cache_ref import DEV, new_places, on_gpu, pool, rotate_ref, second, tables
from layer_ref import DTYPES, HALF, U, offsets, within
from parity import say

import gated_delta_rule_81_amd as kda

CASES = [  # new, held, page, hq, h, d, rot, off, inter, dtype, order, packed, pad
    ((1,), (0,), 16, 1, 1, 64, 0, 0, False, "bf16", "token", False, 0),
    ((1, 1, 1), (5, 0, 47), 16, 4, 2, 128, 128, 0, False, "f32", "head", False, 0),
    ((3, 0, 17, 1), (0, 9, 30, 2), 24, 6, 2, 64, 32, 16, False, "bf16", "pair", True, 8),
    ((2, 2), (1, 64), 1, 0, 3, 128, 64, 0, True, "bf16", "token", False, 0),
    ((70, 1, 5), (3, 0, 100), 64, 0, 1, 576, 64, 512, True, "bf16", "token", True, 0),
    ((9,), (0,), 7, 5, 5, 576, 16, 0, False, "f32", "token", True, 24),
    ((1,) * 70, tuple(range(70)), 8, 17, 1, 64, 64, 0, True, "f32", "pair", True, 0),
    ((40, 300), (0, 11), 32, 33, 7, 128, 96, 32, False, "bf16", "head", True, 8),
]


def make(case, seed=0):
    new, had, page, hq, h, d, rot, off, inter, dtype, order, packed, pad = case
    g, dt = torch.Generator().manual_seed(seed), DTYPES[dtype]
    lens = [a + b for a, b in zip(new, had)]
    table, _, pages = tables([-(-n // page) for n in lens], 0, page, g)
    k_cache = pool(pages, page, h, d, dt, order, g)
    latent = d == 576 and dtype == "bf16"
    v_cache = None if latent else second(k_cache, order, g)
    T = sum(new)
    wide = torch.randn(T, (hq + 2 * h) * d + pad, generator=g).to(dt)
    if pad:
        wide[:, (hq + 2 * h) * d:] = float("nan")
    rope = pos = None
    if rot:
        a = torch.arange(99, dtype=torch.float64)[:, None] * 2.0 ** -torch.arange(rot // 2)
        rope = torch.cat([a.cos(), a.sin()], -1).float()
        pos = torch.randint(-3, 103, (T,), generator=g, dtype=torch.int32)
    return dict(wide=wide, k_cache=k_cache, v_cache=v_cache, table=table, rope=rope, pos=pos,
                lens=torch.tensor(lens, dtype=torch.int32), cu=offsets(new) if packed else None)


def cut(wide, case):
    hq, h, d = case[3:6]
    part = lambda a, n: wide[:, a * d: (a + n) * d].unflatten(1, (n, d))
    return (part(0, hq) if hq else None), part(hq, h), part(hq + h, h)


def append(x, case, **kw):
    to = lambda t: None if t is None else t.to(DEV)
    q, k, v = cut(to(x["wide"]), case)
    kc, vc = on_gpu(x["k_cache"], x["v_cache"], case[10])
    out = kda.cache_append(k, None if vc is None else v, kc, vc, to(x["table"]), to(x["lens"]),
                           to(x["cu"]), q=q, table=to(x["rope"]), positions=to(x["pos"]),
                           rotary_offset=case[7], interleaved=case[8], **kw)
    torch.cuda.synchronize()
    return out, kc, vc


def expect(got, x, case, what):
    """Compare with the definition."""
    new, page, hq, rot, off, inter, dt = case[0], case[2], case[3], case[6], case[7], case[8], DTYPES[case[9]]
    out, kc, vc = got
    q, k, v = cut(x["wide"], case)
    i = torch.arange(rot // 2)
    a, b = (off + 2 * i, off + 2 * i + 1) if inter else (off + i, off + i + rot // 2)

    def turned(t):
        y, m = t.double(), torch.zeros_like(t.double())
        if rot:
            m[..., a] = m[..., b] = y[..., a].abs() + y[..., b].abs()
            y = rotate_ref(y, x["rope"].double(), x["pos"], off, inter)
        return y, HALF[dt] * y.abs() * (m > 0) + 3 * U * m * (1 + HALF[dt])

    if hq:
        y, m = turned(q)
        within(out, y, m, what + " q")
    y, m = turned(k)
    want, bound = x["k_cache"].double(), torch.zeros(x["k_cache"].shape, dtype=torch.float64)
    values = None if vc is None else x["v_cache"].double()
    for t, _, p, slot in new_places(x["table"], x["lens"], new, page):
        if 0 <= p < want.shape[0]:
            want[p, slot], bound[p, slot] = y[t], m[t]
            if vc is not None:
                values[p, slot] = v[t].double()
    within(kc, want, bound, what + " k")
    if vc is not None:
        assert torch.equal(vc.double().cpu(), values), what + " v"


@pytest.mark.gpu
@pytest.mark.parametrize("case", CASES, ids=str)
def test_append(case):
    say("cache_append", case)
    x = make(case)
    expect(append(x, case), x, case, "append")


@pytest.mark.gpu
def test_tokens_without_a_place():
    """Lengths under the new tokens', over the table's width, under zero, pages that are none:
    those tokens are left out, their q rotated all the same; tokens behind the last offset
    are left as they were."""
    case = ((3, 4, 2, 5), (0, 0, 0, 0), 4, 2, 2, 64, 32, 0, False, "bf16", "token", True, 0)
    x = make(case)
    x["lens"] = torch.tensor([1, 400, -7, 5], dtype=torch.int32)
    x["table"][3, 0] = x["k_cache"].shape[0]
    x["table"][3, 1] = -2 ** 31
    say("cache_append: tokens without a place")
    expect(append(x, case), x, case, "without a place")
    x = make(case)
    x["cu"] = offsets((3, 4))  # two sessions, seven tokens of the fourteen
    x["lens"], x["table"] = x["lens"][:2].clone(), x["table"][:2].clone()
    out = torch.full((14, 2, 64), 7.0, dtype=torch.bfloat16, device=DEV)
    got, kc, vc = append(x, case, out_q=out)
    assert got is out and (out[7:] == 7).all()
    short = ((3, 4),) + case[1:]
    y = dict(x, wide=x["wide"][:7], pos=x["pos"][:7])
    expect((out[:7], kc, vc), y, short, "before the last offset")


@pytest.mark.gpu
def test_copies_are_bitwise():
    """NaN, infinities and signed zeros outside the rotated channels are copied as they are."""
    case = ((6,), (1,), 4, 2, 2, 64, 16, 32, False, "bf16", "token", False, 0)
    x = make(case)
    x["wide"].view(torch.int16)[:, ::5] = torch.tensor(-1, dtype=torch.int16)  # a NaN's bits
    x["wide"][:, 1::7] = float("-inf")
    say("cache_append: odd values")
    _, kc, vc = append(x, case)
    _, k, v = cut(x["wide"], case)
    for t, _, p, slot in new_places(x["table"], x["lens"], case[0], 4):
        keep = [c for c in range(64) if not 32 <= c < 48]
        bits = lambda z: z.contiguous().cpu().view(torch.int16)
        assert torch.equal(bits(kc[p, slot])[:, keep], bits(k[t])[:, keep])
        assert torch.equal(bits(vc[p, slot]), bits(v[t]))


@pytest.mark.gpu
def test_rotated_in_place():
    case = CASES[7]
    x = make(case)
    say("cache_append: q in place")
    want, k0, v0 = append(x, case)
    wide = x["wide"].to(DEV)
    q, k, v = cut(wide, case)
    kc, vc = on_gpu(x["k_cache"], x["v_cache"], case[10])
    to = lambda t: t.to(DEV)
    got = kda.cache_append(k, v, kc, vc, to(x["table"]), to(x["lens"]), to(x["cu"]), q=q,
                           table=to(x["rope"]), positions=to(x["pos"]), rotary_offset=case[7],
                           out_q=q)
    torch.cuda.synchronize()
    assert got is q and torch.equal(q, want) and torch.equal(kc, k0) and torch.equal(vc, v0)
    assert torch.equal(k.cpu(), cut(x["wide"], case)[1])


@pytest.mark.gpu
def test_captured_follows_lengths():
    """A captured call appends where lens, tables and positions say at each replay."""
    say("cache_append: graph")
    N, H, d, page = 5, 2, 64, 8
    k, v = (torch.randn(N, H, d, device=DEV).bfloat16() for _ in range(2))
    kc, vc = (torch.zeros(40, page, H, d, device=DEV, dtype=torch.bfloat16) for _ in range(2))
    table = torch.randperm(40, device=DEV).int()[: N * 6].reshape(N, 6).contiguous()
    lens = torch.ones(N, dtype=torch.int32, device=DEV)
    a = torch.arange(64, device=DEV)[:, None] * torch.rand(32, device=DEV)
    rope, pos = torch.cat([a.cos(), a.sin()], -1), torch.zeros(N, dtype=torch.int32, device=DEV)
    call = lambda c, w: kda.cache_append(k, v, c, w, table, lens, q=k, table=rope, positions=pos)
    call(kc.clone(), vc.clone())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        q = call(kc, vc)
    k1, v1 = kc.clone(), vc.clone()
    for step in range(4):
        k.copy_(torch.randn_like(k)), v.copy_(torch.randn_like(v))
        lens.copy_(torch.randint(1, 49, (N,), device=DEV)), pos.copy_(lens)
        graph.replay()
        torch.cuda.synchronize()
        want = call(k1, v1)
        torch.cuda.synchronize()
        assert torch.equal(q, want) and torch.equal(kc, k1) and torch.equal(vc, v1), step
