"""Prompts without a shared prefix: one session of some thousand tokens, chunks behind a long text of
their own, one prompt among single tokens.  Bounds as in test_gpu_prefix_attn.py."""
import pytest
import torch

from cache_ref import attend, attention_inputs
from parity import say
from test_gpu_prefix_attn import case, compare

import gated_delta_rule_81_amd as kda


@pytest.mark.gpu
@pytest.mark.parametrize("c", [
    case((1500,), (1500,), 0, 64, 4, 2, 64),
    case((700,), (700,), 0, 24, 8, 1, 128, "f32"),
    case((130,), (2000,), 0, 16, 4, 1, 128),
    case((300, 1, 1, 2), (700, 1200, 31, 2), 0, 32, 8, 2, 64),
    case((400, 1, 0, 1), (400, 90, 0, 1), 0, 16, 8, 1, 128, "f32"),
    case((256, 256), (256, 900), 0, 16, 2, 2, 64, order="head"),
    case((260,), (260,), 0, 64, 16, 1, 576),
    case((64, 1), (300, 200), 0, 32, 16, 1, 576),
], ids=lambda c: f"{c['new']}-{c['lens']}-{c['d']}-{c['dtype']}".replace(" ", ""))
def test_prompts_without_a_prefix(c):
    say("prefix_attention: prompts of their own", c)
    x = attention_inputs(c, 31)
    got = attend(kda, x, c)
    torch.cuda.synchronize()
    compare(got, x, c, "prompts of their own")
    again = attend(kda, x, c)
    torch.cuda.synchronize()
    assert torch.equal(got[0], again[0]) and torch.equal(got[1], again[1])
