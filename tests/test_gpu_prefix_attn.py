"""GPU parity of the attention over a shared prefix and each session's own tokens with
its 64-bit definition, through the public call.

Bounds, element by element, u = 2^-24, h = half a step of the type (of fp32 inputs'
probabilities: none): a score is a sum of d products, d u of scale sum |q k| <= A
(by the norms of q's and k's rows), its exponent 8 u more of its size; the values'
and the probabilities' sums of N terms N u each.  Relative to sum p |v| that is
(2 (d + 8) A + 2 N + 100) u, and h for the probabilities of bf16 inputs; then the
output's own rounding.  lse: ((d + 8) A + N + 32 + 8 |lse|) u.
"""
import math

import pytest
import torch

from cache_ref import DEV, attend, attention_inputs, d_v, heads_of, reference
from layer_ref import DTYPES, HALF, U
from parity import say

import gated_delta_rule_81_amd as kda


def case(new, lens, prefix, page, hq, h, d, dtype="bf16", order="token", packed=None, **kw):
    packed = len(set(new)) > 1 if packed is None else packed
    return dict(new=new, lens=lens, prefix=prefix, page=page, hq=hq, h=h, d=d, dtype=dtype,
                order=order, packed=packed, **kw)


CASES = [
    # one token each: few rows, prefix and own tokens
    case((1,), (1,), 0, 16, 1, 1, 64),
    case((1,), (33,), 100, 16, 4, 2, 128, "f32", "head"),
    case((1, 1, 1), (0, 130, 257), 300, 24, 8, 2, 64, order="pair"),
    case((1, 1), (5, 700), 129, 1, 6, 3, 128),
    case((1,) * 4, (64, 63, 65, 1), 64, 64, 16, 4, 64, "f32", pad=8),
    case((1,) * 3, (300, 1, 40), 1100, 7, 9, 9, 128, "f32", "pair"),
    # over 32 rows for the prefix
    case((1,) * 40, tuple(range(40)), 200, 16, 4, 2, 128, order="head"),
    case((1,) * 37, tuple(3 * i for i in range(37)), 333, 32, 5, 1, 64, pad=16),
    case((1,) * 34, (70,) * 34, 130, 24, 4, 2, 128, "f32"),
    case((1,) * 50, tuple(7 * i for i in range(50)), 65, 24, 6, 2, 64, "f32", "head"),
    # several tokens each, ragged and empty ones, rows in both kernels
    case((3, 1, 0, 40, 2), (3, 20, 15, 90, 2), 150, 16, 8, 2, 128),
    case((4, 4), (4, 100), 0, 32, 12, 1, 64),
    case((70, 200), (80, 200), 0, 64, 4, 4, 64, "f32"),
    case((5, 33), (5, 300), 40, 24, 8, 1, 128, "f32", "pair"),
    # prompts: one walk over prefix and own tokens
    case((150, 190), (150, 333), 260, 64, 4, 2, 128),
    case((300,), (300,), 77, 16, 2, 2, 64, order="head"),
    case((129, 140), (200, 140), 100, 24, 3, 1, 64, "f32"),
    # latent rows
    case((1, 1), (40, 0), 100, 16, 12, 1, 576),
    case((1,) * 5, (1, 33, 64, 65, 200), 140, 64, 96, 1, 576, order="head", pad=8),
    case((2, 0, 9), (30, 5, 9), 70, 24, 16, 2, 576),
    case((60, 3), (60, 70), 50, 32, 16, 1, 576),
]


def bounds(x, c, lse, wgt, out, scale=None):
    q, d, dt = heads_of(x["q"], c["hq"], c["d"]).double(), c["d"], DTYPES[c["dtype"]]
    norm = lambda t: t.double().nan_to_num(0, 0, 0).norm(dim=-1).max() if t.numel() else torch.tensor(0.0)
    A = float(norm(q) * norm(x["k"])) * (d ** -0.5 if scale is None else scale)
    N = c["prefix"] + max([0, *c["lens"]])
    h = HALF[dt]
    rounded = h if c["dtype"] == "bf16" else 0.0
    b = h * out.abs() + (rounded + (2 * (d + 8) * A + 2 * N + 100) * U) * wgt * (1 + h)
    return b, ((d + 8) * A + N + 32 + 8 * lse.abs().nan_to_num(0, 0, 0)) * U


def compare(got, x, c, what, scale=None):
    out, lse, wgt = reference(x, c, scale)
    bo, bl = bounds(x, c, lse, wgt, out, scale)
    y, z = got[0].double().cpu(), got[1].double().cpu()
    assert y.shape == out.shape and z.shape == lse.shape
    empty = lse == -math.inf
    assert torch.equal(z == -math.inf, empty), what
    assert (y[empty] == 0).all(), what + ": rows that see nothing"
    off, lo = (y - out).abs(), (z - lse).abs()[~empty]
    assert torch.isfinite(y).all() and torch.isfinite(z[~empty]).all(), what
    assert (off <= bo).all(), f"{what}: {float((off / bo.clamp_min(1e-300)).max()):.2f} times the bound"
    assert (lo <= bl[~empty]).all(), f"{what} lse: {float((lo / bl[~empty]).max()):.2f} times the bound"


@pytest.mark.gpu
@pytest.mark.parametrize("c", CASES, ids=lambda c: "-".join(str(v) for v in c.values()).replace(" ", "")[:80])
def test_attention(c):
    say("prefix_attention", c)
    x = attention_inputs(c)
    got = attend(kda, x, c)
    torch.cuda.synchronize()
    compare(got, x, c, "attention")


MASKS = [c for c in CASES if c["new"] in ((1, 1, 1), (3, 1, 0, 40, 2), (5, 33), (150, 190), (60, 3), (1,) * 34)]


@pytest.mark.gpu
@pytest.mark.parametrize("c", MASKS, ids=lambda c: str(c["new"])[:24])
def test_what_is_not_seen_does_not_reach(c):
    """NaN and infinities behind the lengths, in other pages, behind the prefix and in later
    tokens' rows; the later tokens' own outputs are what the formula says."""
    x = attention_inputs(c, 3)
    say("prefix_attention: hidden values", c)
    page = c["page"]
    used = torch.zeros(x["k"].shape[:2], dtype=torch.bool)
    if c["prefix"]:
        for j in range(c["prefix"]):
            used[x["prefix_pages"][j // page], j % page] = True
    last = []
    for s, n in enumerate(c["lens"]):
        for j in range(n):
            used[x["table"][s, j // page], j % page] = True
        if c["new"][s] > 1 and n:
            last.append((s, int(x["table"][s, (n - 1) // page]), (n - 1) % page))
    clean = {k: v if v is None else v.clone() for k, v in x.items()}
    for t in (x["k"], x["v"]):
        if t is not None:
            t[~used] = float("nan")
    got = attend(kda, x, c)
    torch.cuda.synchronize()
    compare(got, clean, c, "behind the lengths")
    # the last token of each session of several: seen by that token alone
    ends, t = [], 0
    for n in c["new"]:
        ends.append(t + n - 1)
        t += n
    vals = x["k"] if x["v"] is None else x["v"]
    for s, p, slot in last:
        vals[p, slot, :, 0] = float("inf")
        vals[p, slot, :, 33] = float("nan")
    if not last:
        return
    got = attend(kda, x, c)
    torch.cuda.synchronize()
    mine = torch.zeros(sum(c["new"]), dtype=torch.bool)
    for s, _, _ in last:
        mine[ends[s]] = True
    want = attend(kda, clean, c)
    torch.cuda.synchronize()
    # the other tokens: as without them (their products go in one by one then)
    ref, lse, wgt = reference(clean, c)
    bo, _ = bounds(clean, c, lse, wgt, ref)
    y = got[0].double().cpu()
    assert torch.isfinite(y[~mine]).all()
    assert ((y - ref).abs() <= bo)[~mine].all()
    if x["v"] is not None:  # latent keys hold the same values, so their scores are odd too
        assert (y[mine][:, :, 0] == math.inf).all() and torch.isnan(y[mine][:, :, 33]).all()
        assert ((y - ref).abs() <= bo)[mine][:, :, 1:33].all()
        assert torch.equal(got[1], want[1])


@pytest.mark.gpu
def test_bad_pages_and_lengths():
    """Entries that are no page hide their tokens; lengths under zero, under the new tokens' and
    over the table count as the documentation says."""
    for c in (case((1, 1, 1, 1), (100, 40, 90, 64), 130, 16, 4, 2, 64),
              case((40, 3, 37, 20), (100, 40, 90, 64), 130, 16, 8, 2, 128, packed=True),
              case((1,) * 40, tuple(range(40, 80)), 130, 16, 2, 1, 64, "f32")):
        x = attention_inputs(c, 5)
        x["table"][0, 1] = x["k"].shape[0]
        x["table"][2, 0] = -1
        x["table"][2, 2] = 2 ** 31 - 1
        x["prefix_pages"][3] = -2 ** 31
        x["prefix_pages"][8] = x["k"].shape[0] + 5
        say("prefix_attention: pages that are none", c)
        got = attend(kda, x, c)
        torch.cuda.synchronize()
        compare(got, x, c, "bad pages")
        lens = list(c["lens"])
        lens[0], lens[1], lens[3] = -5, c["new"][1] - 1, 10 ** 9
        x["lens"] = torch.tensor(lens, dtype=torch.int32)
        x["table"][x["table"] < 0] = 0  # the room behind the pages is read now
        x["prefix_len"][0] = 10 ** 9
        c2 = dict(c, lens=tuple(min(n, x["table"].shape[1] * 16) for n in lens), prefix=144)
        say("prefix_attention: lengths", c2)
        got = attend(kda, x, c2)
        torch.cuda.synchronize()
        compare(got, x, c2, "lengths")
        x["prefix_len"][0] = -1
        got = attend(kda, x, c2)
        torch.cuda.synchronize()
        compare(got, x, c2, "no prefix")


@pytest.mark.gpu
def test_nothing_to_see_at_all():
    say("prefix_attention: nothing to see")
    for d, dv, dt in ((64, 64, torch.float32), (128, 128, torch.bfloat16), (576, 512, torch.bfloat16)):
        q = torch.randn(40, 4, d, device=DEV).to(dt)
        cache = torch.full((2, 16, 2, d), float("nan"), device=DEV, dtype=dt)
        v = None if d == 576 else cache.clone()
        lens = torch.zeros(40, dtype=torch.int32, device=DEV)
        for width in (0, 3):
            for prefix in (False, True):
                table = torch.zeros(40, width, dtype=torch.int32, device=DEV)
                pp = torch.zeros(2, dtype=torch.int32, device=DEV) if prefix else None
                pl = torch.zeros(1, dtype=torch.int32, device=DEV) if prefix else None
                for n in (1, 40):
                    out, lse = kda.prefix_attention(q[:n], cache, v, table[:n].contiguous(), lens[:n],
                                                    pp, pl, output_lse=True)
                    torch.cuda.synchronize()
                    assert out.shape == (n, 4, dv) and (out == 0).all() and (lse == -math.inf).all()


@pytest.mark.gpu
def test_scores_of_minus_infinity():
    """Keys of minus infinity that are seen: weight zero beside others; alone, the formula's NaN."""
    say("prefix_attention: scores of -inf")
    q = torch.ones(2, 1, 64, device=DEV)
    k = torch.zeros(2, 16, 1, 64, device=DEV)
    v = torch.randn_like(k)
    k[0, 3, 0, 0] = -math.inf
    k[1, :, 0, 0] = -math.inf
    table = torch.tensor([[0], [1]], dtype=torch.int32, device=DEV)
    lens = torch.tensor([16, 16], dtype=torch.int32, device=DEV)
    out, lse = kda.prefix_attention(q, k, v, table, lens, output_lse=True)
    torch.cuda.synchronize()
    keep = [i for i in range(16) if i != 3]
    assert torch.allclose(out[0, 0], v[0, keep, 0].mean(0), atol=1e-6)
    assert abs(float(lse[0, 0]) - math.log(15)) < 1e-6
    assert torch.isnan(out[1]).all() and float(lse[1, 0]) == -math.inf


@pytest.mark.gpu
def test_large_scores():
    """Scores of some thousands, rising and falling along the tokens."""
    c = case((1, 1, 40), (200, 300, 90), 400, 16, 8, 2, 128)
    x = attention_inputs(c, 9)
    j = torch.linspace(-3, 3, x["k"].shape[0])[:, None, None, None]
    x["k"] = (x["k"].float() * (1 + 20 * j.abs()) + 8 * j).bfloat16()
    say("prefix_attention: large scores")
    got = attend(kda, x, c, scale=0.5)
    torch.cuda.synchronize()
    compare(got, x, c, "large scores", 0.5)


@pytest.mark.gpu
def test_outputs_in_place_of_new_ones():
    """out as a slice of a wider row, lse, and a workspace of the size that is asked for."""
    c = case((3, 1, 0, 40, 2), (3, 20, 15, 90, 2), 150, 16, 8, 2, 128)
    x = attention_inputs(c)
    want = attend(kda, x, c)
    wide = torch.full((46, 8 * 128 + 16), 5.0, dtype=torch.bfloat16, device=DEV)
    out = wide[:, : 8 * 128].unflatten(1, (8, 128))
    lse = torch.empty(46, 8, device=DEV)
    n = kda.prefix_attention_workspace_size(46, 5, 8, 2, 128, 128, 16, x["table"].shape[1],
                                            x["prefix_pages"].shape[0], torch.bfloat16)
    ws = torch.full((n + 64,), 0xFF, dtype=torch.uint8, device=DEV)
    say("prefix_attention: given outputs")
    got = attend(kda, x, c, out=out, lse=lse, workspace=ws[:n])
    torch.cuda.synchronize()
    assert got[0] is out and got[1] is lse
    assert torch.equal(out, want[0]) and torch.equal(lse, want[1])
    assert (wide[:, 8 * 128:] == 5).all() and (ws[n:] == 0xFF).all()


@pytest.mark.gpu
def test_tokens_behind_the_last_offset():
    for c in (case((1, 5, 0), (3, 20, 15), 150, 16, 8, 2, 64), case((1, 5, 0), (3, 20, 15), 0, 16, 8, 2, 64),
              case((30, 50), (30, 50), 64, 16, 8, 2, 64), case((1, 5, 0), (3, 20, 15), 150, 16, 8, 2, 576)):
        x = attention_inputs(c)
        T = sum(c["new"])
        x["q"] = torch.cat([x["q"], torch.randn(9, x["q"].shape[1]).to(x["q"].dtype)])
        out = torch.full((T + 9, 8, d_v(c)), 5.0, dtype=torch.bfloat16, device=DEV)
        lse = torch.full((T + 9, 8), 5.0, device=DEV)
        x["cu"] = torch.tensor([0] + [sum(c["new"][: i + 1]) for i in range(len(c["new"]))], dtype=torch.int32)
        say("prefix_attention: behind the last offset", c)
        attend(kda, x, c, out=out, lse=lse)
        torch.cuda.synchronize()
        assert (out[T:] == 5).all() and (lse[T:] == 5).all()
        compare((out[:T], lse[:T]), dict(x, q=x["q"][:T]), c, "before it")


@pytest.mark.gpu
def test_captured_follows_lengths():
    """A captured call follows lens, prefix_len, tables and offsets; two captured calls with a
    workspace each, replayed in turn, and the eager results in between."""
    N, H, G, d, page = 6, 2, 4, 128, 16
    g = torch.Generator(device=DEV).manual_seed(4)
    r = lambda *s: torch.randn(*s, device=DEV, generator=g).bfloat16()
    kc, vc = r(200, page, H, d), r(200, page, H, d)
    order = torch.randperm(200, device=DEV, generator=g).int()
    table, pp = order[: N * 20].reshape(N, 20).contiguous(), order[N * 20: N * 20 + 40].contiguous()
    lens = torch.full((N,), 7, dtype=torch.int32, device=DEV)
    pl = torch.tensor([100], dtype=torch.int32, device=DEV)
    say("prefix_attention: graphs")
    for T, cu in ((N, None), (3 * N, None), (80, torch.tensor([0, 1, 5, 5, 50, 60, 80], dtype=torch.int32, device=DEV))):
        q = r(T, H * G, d)
        call = lambda: kda.prefix_attention(q, kc, vc, table, lens, pp, pl, cu, output_lse=True)
        call()
        graphs, outs = [torch.cuda.CUDAGraph() for _ in range(2)], []
        for graph in graphs:
            with torch.cuda.graph(graph):
                outs.append(call())
        for step in range(4):
            q.copy_(r(T, H * G, d))
            lens.copy_(torch.randint(0, 321, (N,), device=DEV, generator=g))
            pl.fill_((0, 640, 333, 5)[step])
            for graph in graphs:
                graph.replay()
            torch.cuda.synchronize()
            want = call()
            torch.cuda.synchronize()
            for got in outs:
                assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1]), (T, step)


@pytest.mark.gpu
def test_two_streams_and_repeats():
    """The same call on two streams at once and again: the same bits."""
    c = case((3, 1, 0, 40, 2), (3, 20, 15, 90, 2), 350, 16, 8, 2, 128)
    x = attention_inputs(c)
    want = attend(kda, x, c)
    torch.cuda.synchronize()
    say("prefix_attention: two streams")
    streams, got = [torch.cuda.Stream() for _ in range(2)], []
    for i in range(6):
        with torch.cuda.stream(streams[i % 2]):
            got.append(attend(kda, x, c))
    torch.cuda.synchronize()
    for out, lse in got:
        assert torch.equal(out, want[0]) and torch.equal(lse, want[1])


@pytest.mark.gpu
@pytest.mark.parametrize("d", [128, 576])
def test_split_prefix_is_the_same_attention(d):
    """A prefix as every session's own first pages gives the same result."""
    N, H, G, page, P = 5, 1, 8, 16, 192
    g = torch.Generator(device=DEV).manual_seed(6)
    r = lambda *s: torch.randn(*s, device=DEV, generator=g).bfloat16()
    kc = r(120, page, H, d)
    vc = None if d == 576 else r(120, page, H, d)
    order = torch.randperm(120, device=DEV, generator=g).int()
    pp, own = order[:12].contiguous(), order[12: 12 + N * 4].reshape(N, 4)
    lens = torch.tensor([1, 17, 64, 5, 33], dtype=torch.int32, device=DEV)
    q = r(N, H * G, d)
    say("prefix_attention: prefix as own pages", d)
    a = kda.prefix_attention(q, kc, vc, own.contiguous(), lens, pp,
                             torch.tensor([P], dtype=torch.int32, device=DEV), output_lse=True)
    both = torch.cat([pp.expand(N, 12), own], 1).contiguous()
    b = kda.prefix_attention(q, kc, vc, both, lens + P, output_lse=True)
    torch.cuda.synchronize()
    dv = 512 if d == 576 else d
    # each of the two is within the bound of CASES of the same value: probabilities and
    # outputs of |v| <= 5 rounded once each
    assert (a[0].double() - b[0].double()).abs().max() <= 2 * 2 * 2.0 ** -8 * 5
    assert torch.allclose(a[1], b[1], atol=1e-4) and a[0].shape == (N, H * G, dv)
