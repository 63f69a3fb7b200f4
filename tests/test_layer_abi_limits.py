"""Refusals of the C ABI of include/kda_layer.h and of its Python front end at the
edges: calls without tokens, and sizes past a launch or past 32 bits.  As in
test_layer_abi.py: fake addresses, a host without a GPU.
"""
import pytest
import torch

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
