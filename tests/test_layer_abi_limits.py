"""Refusals of the C ABI of include/kda_layer.h and of its Python front end at the
edges: calls without tokens, and sizes past a launch or past 32 bits.  As in
test_layer_abi.py: fake addresses, a host without a GPU.
"""
import pytest
import torch

import gated_delta_rule_81_amd as kda
from gated_delta_rule_81_amd._lib import lib
from test_layer_abi import DECLARED, DEVICE, NULL, OK, UNSUP, call

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


def packed(num):
    return dict(batch=1, cu_seqlens=1 << 59, num_seqs=num)


WIDE = {s: 1 << 28 for s in ("x_stride", "d_out_stride", "dx_stride")}
PAST_A_LAUNCH = [  # entry point, the most that fits (or close to it), the least that does not
    # a workgroup of 256 threads copies four rows of states
    ("kda_short_conv_fwd", packed((1 << 24) // 3 * 4 - 64), packed((1 << 24) // 3 * 4 + 64)),
    # ... forms the gradient of four states
    ("kda_short_conv_bwd", packed((1 << 26) - 64), packed(1 << 26)),
    # the sum of five gradients a channel, 64 of them in 1024 threads
    ("kda_short_conv_bwd", dict(batch=1, seq_len=1, channels=(1 << 28) // 5 - 64, **WIDE),
     dict(batch=1, seq_len=1, channels=(1 << 28) // 5 + 64, **WIDE)),
    ("kda_short_conv_step", dict(batch=(1 << 26) - 4), dict(batch=1 << 26)),
    # a pair of heads in 256 threads, and one head where a group has one
    ("kda_ssm_chunk_fwd", dict(batch=(1 << 23) - 8, seq_len=1), dict(batch=1 << 23, seq_len=1)),
    ("kda_ssm_chunk_fwd", dict(batch=(1 << 22) - 8, seq_len=1, num_groups=4),
     dict(batch=1 << 22, seq_len=1, num_groups=4)),
    ("kda_ssm_chunk_fwd", packed((1 << 23) - 16), packed(1 << 23)),
    ("kda_ssm_chunk_fwd", packed(1), packed(1 << 30)),  # 2^32 workgroups
    # both directions of the walk at once; 512 threads a block and group
    ("kda_ssm_chunk_bwd", dict(batch=(1 << 22) - 8, seq_len=1), dict(batch=1 << 22, seq_len=1)),
    ("kda_ssm_decode_step", dict(batch=(1 << 22) - 1), dict(batch=1 << 22)),
]


@pytest.mark.parametrize("name,fits,past", PAST_A_LAUNCH)
def test_calls_past_a_launch(name, fits, past):
    """A launch holds less than 2^32 threads: more work is refused before any of it
    is done."""
    kw = dict(workspace=1 << 60, workspace_bytes=1 << 62, state=1 << 60)
    if name.startswith("kda_ssm"):
        kw.update(initial_state=None, final_state=None, d_initial_state=None, d_final_state=None)
    kw = {k: v for k, v in kw.items() if k in DECLARED[name]}
    assert call(name, **kw, **fits) == DEVICE
    assert call(name, **kw, **past) == UNSUP


def test_sizes_past_32_bits():
    """The C calls count in 32 bits; a size past them is refused and not cut off
    (a T of 2^32 + 8 would run as 8 tokens)."""
    n = (1 << 32) + 8
    m = lambda *s, dtype=torch.bfloat16: torch.empty(s, dtype=dtype, device="meta")
    f = lambda *s: m(*s, dtype=torch.float32)
    for run in [
        lambda: kda.short_conv(m(1, n, 1), f(1, 4)),
        lambda: kda.short_conv(m(n, 0, 1), f(1, 4), output_final_state=False),
        lambda: kda.short_conv(m(1, 2, n), f(n, 4)),
        lambda: kda.short_conv(m(1, 8, 1), f(1, n)),
        lambda: kda.short_conv(m(1, 8, 1), f(1, 4), cu_seqlens=m(n + 1, dtype=torch.int32)),
        lambda: kda.short_conv_bwd(m(1, n, 1), f(1, 4), m(1, n, 1)),
        lambda: kda.short_conv_step(m(n, 1), f(1, 4), m(n, 3, 1)),
        lambda: kda.qk_norm(m(1 << 20, 1 << 13, 1, 64), m(1 << 20, 1 << 13, 0, 64)),
        lambda: kda.qk_norm(m(2, 1, 64), m(2, 1, 64), table=f(n, 16),
                            positions=m(2, dtype=torch.int32)),
        lambda: kda.qk_norm(m(1, n, 64), m(1, 1, 64)),
        lambda: kda.ssm_chunk_fwd(m(1, n, 1, 64), f(1, n, 1), f(1), m(1, n, 1, 64), m(1, n, 1, 64)),
        lambda: kda.ssm_chunk_bwd(m(1, n, 1, 64), f(1, n, 1), f(1), m(1, n, 1, 64), m(1, n, 1, 64),
                                  m(1, n, 1, 64)),
        lambda: kda.ssm_decode_step(m(n, 1, 64), f(n, 1), f(1), m(n, 1, 64), m(n, 1, 64),
                                    f(n, 1, 64, 64)),
        lambda: kda.short_conv_bwd_workspace_size(1, n, 1, 4),
        lambda: kda.qk_norm_bwd_workspace_size(n, 1, 1, 64),
        lambda: kda.ssm_workspace_size(1, n, 1, 64, 64),
        lambda: kda.ssm_bwd_workspace_size(1, n, 1, 1, 64, 64, torch.bfloat16),
    ]:
        with pytest.raises(ValueError, match="32 bits"):
            run()
