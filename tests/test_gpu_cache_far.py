"""Caches whose places lie further apart than 2^32 bytes, in every kernel that reads or
writes them: pages of a view with a page stride of 2^31 elements give what the
same pages side by side give, bit for bit."""
import pytest
import torch

from parity import say

import gated_delta_rule_81_amd as kda

DEV = "cuda:0"
APART = (1 << 31) + 4096  # elements between pages
PAGES = 5


@pytest.fixture(scope="module")
def room():
    """Memory for the pages of both caches, apart; only the pages themselves are touched."""
    t = torch.empty(PAGES * APART * 4, dtype=torch.uint8, device=DEV)
    yield t
    del t
    torch.cuda.empty_cache()


def far(room, near, shift):
    """near's values in pages APART elements apart (for fp32 half as far), `shift` elements in."""
    flat = room.view(near.dtype)
    n, page, h, d = near.shape
    apart = APART if near.dtype == torch.bfloat16 else APART // 2
    view = flat[shift:].as_strided((n, page, h, d), (apart, h * d, d, 1))
    view.copy_(near)
    return view


CASES = [  # d, dtype, tokens a session, sessions, heads
    (128, torch.bfloat16, 1, 3, 2), (64, torch.bfloat16, 1, 40, 1), (128, torch.float32, 2, 3, 2),
    (64, torch.float32, 40, 2, 2), (128, torch.bfloat16, 150, 2, 1), (576, torch.bfloat16, 1, 2, 1),
    (576, torch.bfloat16, 70, 1, 1),
]


@pytest.mark.gpu
@pytest.mark.parametrize("d,dtype,each,sessions,heads", CASES, ids=str)
def test_far_pages(room, d, dtype, each, sessions, heads):
    g = torch.Generator(device=DEV).manual_seed(d + each)
    r = lambda *s: torch.randn(*s, device=DEV, generator=g).to(dtype)
    page, T = 128, each * sessions
    k0 = r(PAGES, page, heads, d)
    v0 = None if d == 576 else r(PAGES, page, heads, d)
    k1 = far(room, k0, 0)
    v1 = None if v0 is None else far(room, v0, page * heads * d)
    # the sessions' pages may be shared here: append writes the same rows to all of them
    table = torch.tensor([[4, 1]] * sessions, dtype=torch.int32, device=DEV)
    lens = torch.full((sessions,), 200, dtype=torch.int32, device=DEV)
    pp = torch.tensor([3, 0], dtype=torch.int32, device=DEV)
    pl = torch.tensor([190], dtype=torch.int32, device=DEV)
    k = r(each, heads, d).repeat(sessions, 1, 1)
    v = None if v0 is None else r(each, heads, d).repeat(sessions, 1, 1)
    q = r(T, 4 * heads, d)
    say("far pages", d, dtype, each, sessions, heads)
    got = []
    for kc, vc in ((k0, v0), (k1, v1)):
        kda.cache_append(k, v, kc, vc, table, lens)
        got.append(kda.prefix_attention(q, kc, vc, table, lens, pp, pl, output_lse=True))
    torch.cuda.synchronize()
    assert torch.equal(k0, k1) and (v0 is None or torch.equal(v0, v1))
    for a, b in zip(*got):
        assert torch.isfinite(a).all() and torch.equal(a, b)
