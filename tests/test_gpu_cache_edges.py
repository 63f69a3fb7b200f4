"""Calls on a paged cache that the documentation allows and that stand at its edges: values
that are no number where they are seen, groups that divide no tile, pages that divide none, thousands of
sessions of which most are empty, offsets outside the tokens, the Python paths against each other.  Bounds as
in test_gpu_prefix_attn.py."""
import math

import pytest
import torch

from cache_ref import DEV, attend, attention_inputs, reference
from parity import say
from test_gpu_prefix_attn import bounds, case, compare

import gated_delta_rule_81_amd as kda


@pytest.mark.gpu
@pytest.mark.parametrize("c", [
    case((1,) * 7, (3, 150, 64, 1, 90, 129, 500), 300, 1, 10, 2, 64),
    case((50, 1, 9), (50, 77, 200), 333, 3, 10, 2, 128),
    case((1,) * 30, tuple(range(5, 35)), 131, 7, 12, 1, 128, "f32"),
    case((1, 1), (300, 2), 70, 5, 40, 1, 64),
    case((1, 1, 1), (700, 0, 31), 0, 11, 66, 2, 128, "f32"),
    case((130, 131), (131, 260), 65, 9, 5, 1, 128),
    case((1,) * 3, (65, 1, 200), 130, 1, 5, 1, 576),
    case((3, 40), (70, 41), 67, 3, 7, 1, 576),
    case((20, 33), (20, 140), 0, 13, 14, 2, 576),
], ids=str)
def test_groups_and_pages_that_divide_no_tile(c):
    say("prefix_attention", c)
    x = attention_inputs(c, 11)
    got = attend(kda, x, c)
    torch.cuda.synchronize()
    compare(got, x, c, "odd groups and pages")


@pytest.mark.gpu
@pytest.mark.parametrize("where", ["query", "prefix key", "own key", "prefix value", "own value"])
@pytest.mark.parametrize("c", [
    case((1, 1, 1), (40, 130, 257), 300, 24, 8, 2, 64),
    case((1,) * 40, tuple(range(30, 70)), 200, 16, 4, 2, 128),
    case((1,) * 34, (70,) * 34, 130, 24, 4, 2, 128, "f32"),
    case((150, 190), (150, 333), 260, 64, 4, 2, 128),
    case((3, 40, 2), (31, 90, 32), 150, 16, 8, 2, 64, "f32"),
    case((1,) * 5, (50, 33, 64, 65, 200), 140, 64, 16, 1, 576),
    case((60, 3), (60, 70), 50, 32, 8, 2, 576),
], ids=lambda c: f"{c['new'][:3]}-{c['d']}-{c['dtype']}")
def test_a_nan_that_is_seen(c, where):
    """The rows that see it are NaN as the formula says, and no others."""
    page, H = c["page"], c["h"]
    which, name = (where + " ").split(" ", 1)
    size = c["prefix"] if which == "prefix" else c["lens"][0]
    places = [sum(c["new"]) // 2] if which == "query" else sorted({0, 29, size // 2, size - 1})
    for j in places:
        x = attention_inputs(c, 7)
        if which == "query":
            x["q"][j, c["d"] * (c["hq"] - 1) + 5] = float("nan")
        else:
            t = x["k"] if name.strip() == "key" or x["v"] is None else x["v"]
            entry = x["prefix_pages"][j // page] if which == "prefix" else x["table"][0, j // page]
            t[entry, j % page, H - 1, 9] = float("nan")
        say("prefix_attention: a NaN that is seen", where, j, c)
        got = attend(kda, x, c)
        torch.cuda.synchronize()
        out, lse, wgt = reference(x, c)
        y, z = got[0].double().cpu(), got[1].double().cpu()
        assert torch.isnan(out).any()
        wrong = (torch.isnan(y) != torch.isnan(out)).nonzero().tolist()
        assert not wrong, (j, len(wrong), wrong[:20])
        assert torch.equal(torch.isnan(z), torch.isnan(lse))
        bo, bl = bounds(x, c, lse, wgt, out)
        fine, same = ~torch.isnan(out), ~torch.isnan(lse) & (lse > -math.inf)
        bo, off = bo.nan_to_num(0, 0, 0), (y - out).abs()
        assert (off[fine] <= bo[fine]).all()
        assert ((z - lse).abs()[same] <= bl[same]).all()


@pytest.mark.gpu
@pytest.mark.parametrize("c", [
    case((1,) * 5, (50, 33, 64, 65, 200), 300, 8, 96, 1, 576),
    case((60, 3, 20), (60, 170, 90), 150, 8, 8, 2, 576),
    case((150, 190), (150, 333), 260, 8, 4, 2, 128),
    case((1, 1, 1), (140, 130, 257), 300, 8, 8, 2, 64, "f32"),
], ids=lambda c: f"{c['new'][:3]}-{c['d']}-{c['dtype']}")
def test_pages_that_are_none_among_others(c):
    """Every third page of the prefix and of each session is none; the first page, which is looked at
    in their place, holds NaN and is nobody's."""
    x = attention_inputs(c, 8)
    for t in [x["k"]] + ([] if x["v"] is None else [x["v"]]):
        t[0] = float("nan")
    for pages in (x["table"], x["prefix_pages"]):
        pages[pages == 0] = -1
        flat = pages.view(-1)
        flat[1::3] = torch.tensor([-1, x["k"].shape[0], 2 ** 31 - 1])[torch.arange(len(flat[1::3])) % 3].int()
    say("prefix_attention: pages that are none among others", c)
    got = attend(kda, x, c)
    torch.cuda.synchronize()
    compare(got, x, c, "pages that are none")


@pytest.mark.gpu
def test_thousands_of_sessions():
    """Packed, most of them empty, the first and the last among them; and the same of one token each."""
    g = torch.Generator().manual_seed(1)
    new = torch.randint(-7, 3, (5000,), generator=g).clamp_min(0)
    new[:70] = 0
    new[-131:] = 0
    lens = torch.where(new > 0, new + torch.randint(0, 20, (5000,), generator=g), 0)
    for c in (case(tuple(new.tolist()), tuple(lens.tolist()), 70, 8, 4, 2, 64),
              case((1,) * 2111, tuple(i % 23 for i in range(2111)), 33, 4, 2, 1, 64, "f32"),
              case((1,) * 300, tuple(i % 13 for i in range(300)), 33, 4, 6, 1, 576)):
        x = attention_inputs(c, 2)
        say("prefix_attention: sessions", len(c["new"]))
        got = attend(kda, x, c)
        torch.cuda.synchronize()
        compare(got, x, c, "many sessions")


@pytest.mark.gpu
@pytest.mark.parametrize("d", [64, 128, 576])
def test_offsets_outside_the_tokens(d):
    """Offsets under 0 and over the tokens count as those ends, in both calls."""
    c = case((10, 40, 30), (10, 45, 90), 50, 16, 4, 1, d)
    x = attention_inputs(c, 3)
    say("offsets outside the tokens", d)
    want = attend(kda, x, c)
    q = x["q"][:, :d].unsqueeze(1).contiguous().to(DEV)
    caches = []
    for cu in (x["cu"], torch.tensor([-9, 10, 50, 10 ** 9], dtype=torch.int32)):
        k = x["k"].clone().to(DEV)
        v = None if x["v"] is None else x["v"].clone().to(DEV)
        kda.cache_append(q, None if v is None else q, k, v, x["table"].to(DEV), x["lens"].to(DEV), cu.to(DEV))
        caches.append((k, v))
        got = attend(kda, dict(x, cu=cu), c)
        torch.cuda.synchronize()
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    assert torch.equal(caches[0][0], caches[1][0])
    assert d == 576 or torch.equal(caches[0][1], caches[1][1])
    assert not torch.equal(caches[0][0].cpu(), x["k"])


@pytest.mark.gpu
@pytest.mark.parametrize("d,dtype", [(64, "f32"), (128, "bf16"), (576, "bf16")])
def test_both_ways_through_python(d, dtype):
    """The common case and the checks in words behind it: the same bits."""
    c = case((2, 0, 33, 1), (9, 4, 60, 1), 100, 16, 6, 2, d, dtype, packed=True)
    x = attention_inputs(c, 4)
    say("both ways through Python", d, dtype)
    want = attend(kda, x, c)
    got = attend(kda, x, c, out=torch.empty_like(want[0]))
    torch.cuda.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    T = 36
    k = x["k"].to(DEV)
    q, kv = (torch.randn(T, h, d, device=DEV).to(k.dtype) for h in (6, 2))
    table = torch.randn(50, 32, device=DEV)
    pos = torch.arange(T, dtype=torch.int32, device=DEV)
    both = []
    for given in (None, torch.empty_like(q)):
        kc, vc = k.clone(), None if d == 576 else k.clone()
        y = kda.cache_append(kv, None if vc is None else kv, kc, vc, x["table"].to(DEV), x["lens"].to(DEV),
                             x["cu"].to(DEV), q=q, table=table, positions=pos, out_q=given)
        torch.cuda.synchronize()
        assert given is None or y is given
        both.append((y, kc) if vc is None else (y, kc, vc))
    assert all(torch.equal(a, b) for a, b in zip(*both))


@pytest.mark.gpu
def test_shapes_that_the_common_case_leaves():
    """Tensors on the device whose shapes are no call's: said in words, nothing launched."""
    c = case((2, 1), (2, 1), 20, 16, 4, 2, 64)
    x = attention_inputs(c)
    to = lambda t: t.to(DEV)
    k, v, table, lens = to(x["k"]), to(x["v"]), to(x["table"]), to(x["lens"])
    q = torch.randn(2, 4, 64, device=DEV).bfloat16()
    for bad in (q[0, 0, 0], q[0], q[None]):
        with pytest.raises(ValueError):
            kda.prefix_attention(bad, k, v, table, lens)
        with pytest.raises(ValueError):
            kda.cache_append(bad, bad, k, v, table, lens)
    with pytest.raises(ValueError):
        kda.prefix_attention(q, k[0], v[0], table, lens)
    with pytest.raises(ValueError):
        kda.prefix_attention(q, k, v, table[0], lens)
    with pytest.raises((TypeError, ValueError)):
        kda.prefix_attention(q.half(), k, v, table, lens)
    out, lse = kda.prefix_attention(q[:0], k, v, table[:0], lens[:0], output_lse=True)
    assert out.shape == (0, 4, 64) and lse.shape == (0, 4)
