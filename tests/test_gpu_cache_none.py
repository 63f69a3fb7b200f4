"""Tokens of which nothing is there: every page that they could see is none, or the cache has
no pages at all.  Their output is 0 and their lse -inf as for lengths of zero; beside them stand
sessions and later tokens that see something.  Each walk, with and without parts; bounds as in
test_gpu_prefix_attn.py."""
import math

import pytest
import torch

from cache_ref import DEV, attend, attention_inputs, d_v, reference
from parity import say
from test_gpu_prefix_attn import case, compare

import gated_delta_rule_81_amd as kda

CASES = [
    # few rows: of the prefix and of own tokens; own ones in one part, which is the output, and packed
    case((1, 1, 1), (40, 130, 257), 300, 24, 8, 2, 64),
    case((1, 1), (33, 70), 0, 16, 1, 1, 128, "f32", room=0),
    case((1, 1, 1), (0, 1, 64), 0, 32, 8, 2, 64, room=0),
    case((2, 0, 8), (2, 0, 40), 0, 16, 4, 1, 64, room=0),
    case((20,), (52,), 0, 16, 1, 1, 64, room=0),
    # the prefix by tiles
    case((1,) * 40, tuple(range(30, 70)), 200, 16, 4, 2, 128),
    case((1,) * 34, (70,) * 34, 130, 24, 4, 2, 128, "f32"),
    # own tokens by tiles, in parts and in one
    case((3, 1, 0, 40, 2), (3, 20, 15, 90, 2), 150, 16, 8, 2, 128),
    case((4, 4), (4, 100), 0, 32, 12, 1, 64),
    case((60,), (90,), 0, 32, 4, 1, 128, room=0),
    case((70, 40), (80, 96), 0, 16, 2, 2, 64, "f32", room=0),
    # one walk over both
    case((150, 190), (150, 333), 260, 64, 4, 2, 128),
    case((129, 140), (200, 140), 100, 24, 3, 1, 64, "f32"),
    # latent rows, in parts and in one
    case((1,) * 5, (1, 33, 64, 65, 200), 140, 64, 96, 1, 576),
    case((60, 3, 20), (60, 170, 90), 150, 8, 8, 2, 576),
    case((60,), (90,), 0, 32, 4, 1, 576, room=0),
]
ID = lambda c: f"{c['new'][:3]}-{c['lens'][:3]}-{c['prefix']}-{c['d']}-{c['dtype']}".replace(" ", "")


def check(x, c, what):
    say("prefix_attention:", what, c)
    got = attend(kda, x, c)
    torch.cuda.synchronize()
    compare(got, x, c, what)


@pytest.mark.gpu
@pytest.mark.parametrize("c", CASES, ids=ID)
def test_every_page_is_none(c):
    x = attention_inputs(c, 12)
    for t in [x["k"]] + ([] if x["v"] is None else [x["v"]]):
        t[0] = float("nan")  # looked at in their place, and nobody's
    for pages in (x["table"], x["prefix_pages"]):
        if pages is not None:
            pages[pages == 0] = -1
    none = torch.tensor([-1, x["k"].shape[0], 2 ** 31 - 1, -2 ** 31]).int()
    keep = {k: None if x[k] is None else x[k].clone() for k in ("table", "prefix_pages")}
    x["table"][0] = none[torch.arange(x["table"].shape[1]) % 4]
    check(x, c, "the first session's pages are none")
    if c["prefix"]:
        x["prefix_pages"][:] = none[torch.arange(len(x["prefix_pages"])) % 4]
        check(x, c, "and the prefix's")
        x["table"][:] = keep["table"]
        x["table"][:, 0] = -1  # later tokens of a session see its other pages
        check(x, c, "the prefix's and each session's first")
    x["table"][:] = -1
    check(x, c, "all of them")
    if c["prefix"]:
        x["prefix_pages"][:] = keep["prefix_pages"]
        check(x, c, "all but the prefix's")


@pytest.mark.gpu
@pytest.mark.parametrize("c", CASES, ids=ID)
def test_first_own_pages_are_none(c):
    x = attention_inputs(c, 13)
    x["table"][:, 0] = -1
    if c["prefix"]:
        x["prefix_len"][0] = 0
    check(x, dict(c, prefix=0), "the first own page of each session")


@pytest.mark.gpu
@pytest.mark.parametrize("c", [c for c in CASES if c["order"] == "token"], ids=ID)
def test_a_cache_without_pages(c):
    x = attention_inputs(c, 14)
    x["k"] = x["k"][:0]
    x["v"] = None if x["v"] is None else x["v"][:0]
    say("prefix_attention: no pages", c)
    out, lse = attend(kda, x, c)
    torch.cuda.synchronize()
    assert out.shape == (sum(c["new"]), c["hq"], d_v(c))
    assert (out == 0).all() and (lse == -math.inf).all()


@pytest.mark.gpu
@pytest.mark.parametrize("d,dtype", [(64, "f32"), (128, "bf16"), (576, "bf16")])
def test_a_padded_row_of_a_captured_batch(d, dtype):
    """A row whose table is none, of any length, among others that change at each replay."""
    c = case((1,) * 6, (40, 1, 90, 33, 64, 7), 0, 16, 8, 2, d, dtype)
    x = attention_inputs(c, 15)
    x["table"][x["table"] < 0] = 0
    to = lambda t: None if t is None else t.to(DEV)
    q = to(x["q"]).unflatten(1, (8, d))
    k, v, table, lens = to(x["k"]), to(x["v"]), to(x["table"]), to(x["lens"])
    call = lambda: kda.prefix_attention(q, k, v, table, lens, output_lse=True)
    say("prefix_attention: padded rows, captured", d, dtype)
    call()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = call()
    held = table.clone()
    for step, rows in enumerate(([], [1], [0, 4], [0, 1, 2, 3, 4, 5], [5])):
        table.copy_(held)
        table[rows] = -1
        new = tuple(1 + (n * (step + 3)) % 90 for n in c["lens"])
        lens.copy_(torch.tensor(new, dtype=torch.int32))
        graph.replay()
        torch.cuda.synchronize()
        y = dict(x, table=table.cpu(), lens=lens.cpu())
        compare(got, y, dict(c, lens=new), f"replay {step}")
        assert (reference(y, c)[1][rows] == -math.inf).all()
        want = call()
        torch.cuda.synchronize()
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
