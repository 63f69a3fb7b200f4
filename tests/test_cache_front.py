"""The Python side of the operators on a paged cache: refusals of shapes that no call has."""
import pytest
import torch

import gated_delta_rule_81_amd as kda


@pytest.mark.parametrize("device", ["cpu", pytest.param("cuda:0", marks=pytest.mark.gpu)])
@pytest.mark.parametrize("given", [{}, {"scale": 0.5}, {"output_lse": True}])
def test_heads_without_channels_are_refused_in_words(given, device):
    z = lambda *s: torch.zeros(*s, device=device)
    i = lambda *s: torch.zeros(*s, dtype=torch.int32, device=device)
    with pytest.raises(ValueError, match="channels"):
        kda.prefix_attention(z(4, 8, 0), z(9, 16, 2, 0), z(9, 16, 2, 0), i(4, 3), i(4), **given)
