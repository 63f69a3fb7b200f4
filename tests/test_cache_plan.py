"""What a call of kda_prefix_attn_fwd asks for by its sizes alone (no GPU needed): a workspace
that stays beside the places of the card, and no refusal of work that its launches hold."""
import pytest
import torch

from gated_delta_rule_81_amd import _lib
from test_cache_abi import ATTN, BF16, DECLARED, DEVICE, F32, LATENT, SIZE, UNSUP, VALUES, call, pytestmark  # noqa: F401


def size(**kw):
    return getattr(_lib.lib(), SIZE)(*[{**VALUES, **kw}[a] for a in DECLARED[SIZE]])


def heads(hq, hk, d):
    return dict(q_heads=hq, kv_heads=hk, head_dim=d, v_dim=d, q_stride=hq * d, out_stride=hq * d,
                head_stride=d, token_stride=hk * d, page_stride=64 * hk * d, page_size=64)


@pytest.mark.parametrize("hq,hk", [(32, 8), (96, 8), (16, 16), (8, 1), (4, 2)])
@pytest.mark.parametrize("tokens,seqs", [(1, 1), (33, 1), (256, 1), (4096, 1), (8192, 1), (32768, 1),
                                         (131072, 1), (8192, 16), (32768, 7), (4196, 101)])
@pytest.mark.parametrize("prefix", [0, 16, 1024])
def test_parts_of_prompts_fit_the_places(tokens, seqs, hq, hk, prefix):
    """Sessions of 128 rows or more on average are cut only where workgroups of 128 rows leave
    some of the 512 places empty: the parts are at most what fills them."""
    rows = tokens * (hq // hk)
    if rows < seqs * 128:
        pytest.skip("few rows a session")
    for dtype in (BF16, F32):
        for width in (8, 512, 4096):
            kw = dict(tokens=tokens, num_seqs=seqs, table_width=width, prefix_width=prefix, dtype=dtype,
                      **heads(hq, hk, 128))
            assert 0 <= size(**kw) <= 512 * 128 * (4 * 128 + 8), kw
    # more workgroups than places: the one part is the output
    if rows // 128 * hk >= 512:
        assert size(**kw) == 0


def test_long_prompts_without_a_prefix_are_not_refused():
    big = dict(tokens=131072, num_seqs=1, table_width=2048, prefix_width=0, prefix_pages=None, prefix_len=None,
               num_pages=4096, **heads(96, 8, 128))
    assert call(ATTN, **big) == DEVICE
    assert call(ATTN, **big, workspace=None, workspace_bytes=0) == DEVICE


def test_rows_that_one_join_holds():
    """Parts of 2^24 rows and more: a wave a row (two with 512 channels), 2^32 threads at most."""
    step = lambda n, **kw: call(ATTN, tokens=n, num_seqs=n, num_pages=1 << 20, table_width=1, **kw)
    one = heads(128, 8, 128)
    assert step(1 << 17, **one) == DEVICE and step(1 << 18, **one) == DEVICE
    assert step((1 << 19) - 1, **one) == DEVICE  # 2^26 rows less one token's
    assert step(1 << 19, **one) == UNSUP
    latent = {**LATENT, "q_heads": 64, "q_stride": 64 * 576, "out_stride": 64 * 512}
    assert step(1 << 18, **latent) == DEVICE and step((1 << 19) - 1, **latent) == DEVICE
    assert step(1 << 19, **latent) == UNSUP
