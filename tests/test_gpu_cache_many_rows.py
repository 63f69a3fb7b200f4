"""A call of 2^24 rows in parts: the same bits as its sessions in calls of an eighth, which are cut alike."""
import pytest
import torch

from cache_ref import DEV
from parity import say

import gated_delta_rule_81_amd as kda


@pytest.mark.gpu
def test_rows_past_2_24():
    N, hq, H, d, page = 1 << 17, 128, 8, 64, 16
    g = torch.Generator(device=DEV).manual_seed(3)
    r = lambda *s: torch.randn(*s, device=DEV, generator=g, dtype=torch.bfloat16)
    k, v = r(4096, page, H, d), r(4096, page, H, d)
    table = torch.randint(0, 4096, (N, 1), device=DEV, generator=g).int()
    lens = torch.randint(0, page + 1, (N,), device=DEV, generator=g).int()
    pp = torch.tensor([7, 4095, 0], dtype=torch.int32, device=DEV)
    pl = torch.tensor([41], dtype=torch.int32, device=DEV)
    q = r(N, hq, d)
    say("prefix_attention: 2^24 rows in parts")
    out, lse = kda.prefix_attention(q, k, v, table, lens, pp, pl, output_lse=True)
    torch.cuda.synchronize()
    for s in torch.arange(N, device=DEV).chunk(8):
        a, b = int(s[0]), int(s[-1]) + 1
        say("prefix_attention: sessions", a, b)
        want, wl = kda.prefix_attention(q[a:b], k, v, table[a:b], lens[a:b], pp, pl, output_lse=True)
        torch.cuda.synchronize()
        assert torch.equal(out[a:b], want) and torch.equal(lse[a:b], wl)
        assert torch.isfinite(want).all() and torch.isfinite(wl).all()
