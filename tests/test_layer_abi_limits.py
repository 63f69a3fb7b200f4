"""Refusals of the C ABI of include/kda_layer.h and of its Python front end at the
edges: calls without tokens, and sizes past a launch or past 32 bits.  As in
test_layer_abi.py: fake addresses, a host without a GPU.
"""
import pytest
import torch

from gated_delta_rule_81_amd._lib import lib
from test_layer_abi import DEVICE, NULL, OK, call

pytestmark = pytest.mark.skipif(torch.cuda.device_count() > 0, reason="runs on a host without a GPU")


@pytest.mark.parametrize("packed", [False, True])
def test_scan_without_tokens_needs_its_decays(packed):
    """Sequences without tokens still have states to pass on, and the kernel that
    does so reads A; dt, x, B, C and out have no element then."""
    kw = dict(seq_len=0, x=None, dt=None, B=None, C=None, out=None)
    if packed:
        kw.update(batch=1, cu_seqlens=1 << 50, num_seqs=3)
    assert call("kda_ssm_chunk_fwd", **kw) == DEVICE
    assert call("kda_ssm_chunk_fwd", **kw, A=None) == NULL
    # nothing to pass on: nothing is read
    none = dict(kw, num_seqs=0) if packed else dict(kw, batch=0)
    assert call("kda_ssm_chunk_fwd", **none, A=None) == OK


def scan_space(batch, seq_len, num_seqs, heads, groups, p, n, dtype=1):
    """Workspace bytes of the scan and of its gradient."""
    return (lib().kda_ssm_chunk_fwd_workspace_size(batch, seq_len, num_seqs, heads, p, n),
            lib().kda_ssm_chunk_bwd_workspace_size(batch, seq_len, num_seqs, heads, groups, p, n,
                                                   dtype))


def test_workspace_of_many_short_sequences():
    """Sequences that are not cut need no room for pieces: however many prompts the
    tokens are shared by, the scan asks for the same."""
    H, P, N = 96, 128, 128
    one = scan_space(1, 32768, 1, H, 1, P, N)[0]
    assert 0 < one < 128 << 20
    for num in (2, 16, 256, 4096, 32768):
        fwd, bwd = scan_space(1, 32768, num, H, 1, P, N)
        assert fwd == one
        # the gradient keeps the state at every block twice, at most one more a sequence
        blocks = 32768 // 64 + num + 1
        assert bwd < 2 * blocks * H * (P * N * 4 + 8) + 4 * one + 64
    # many more sequences than tokens
    assert scan_space(1, 100, 1 << 20, H, 1, P, N)[0] < 128 << 20
