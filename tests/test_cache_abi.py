"""The C ABI of include/kda_cache.h: exports, and the refusal of bad arguments on
the host before any device work; the Python front end's own refusals; and the
CPython module's, which says nothing (no GPU needed).  Pointers are fake addresses
far apart: validation never reads them.
"""
import ctypes
import os
import re

import pytest
import torch

import gated_delta_rule_81_amd as kda
from gated_delta_rule_81_amd import _lib

# the addresses are fake: only a host on which every call stops at the device check
pytestmark = pytest.mark.skipif(torch.cuda.device_count() > 0, reason="runs on a host without a GPU")

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
OK, NULL, SHAPE, UNSUP, ALIGN, ALIAS, DEVICE = 0, -1, -2, -3, -4, -5, -6
F32, BF16 = 0, 1
TB = 1 << 40


def declared():
    text = open(os.path.join(ROOT, "include", "kda_cache.h")).read()
    text = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
    out = {}
    for name, args in re.findall(r"\b(kda_\w+)\s*\(([^)]*)\)\s*;", text):
        out[name] = [a.split()[-1].lstrip("*") for a in args.split(",")]
    return out


DECLARED = declared()
APPEND, ATTN, SIZE = "kda_cache_append", "kda_prefix_attn_fwd", "kda_prefix_attn_workspace_size"


def test_library_exports_what_the_header_declares():
    handle = ctypes.CDLL(_lib.LIB_PATH)
    assert set(DECLARED) == set(_lib.CACHE_SIGNATURES) == {APPEND, ATTN, SIZE}
    assert not set(_lib.CACHE_SIGNATURES) & (set(_lib.SIGNATURES) | set(_lib.LAYER_SIGNATURES))
    for name, args in DECLARED.items():
        assert hasattr(handle, name), name
        assert len(_lib.CACHE_SIGNATURES[name][0]) == len(args), name


POINTERS = {"q", "k", "v", "table", "positions", "page_table", "lens", "cu_seqlens", "out_q",
            "k_cache", "v_cache", "prefix_pages", "prefix_len", "out", "lse", "workspace"}
VALUES = dict(tokens=12, num_seqs=4, q_heads=8, kv_heads=2, head_dim=64, v_dim=64, rotary_dim=32,
              rotary_offset=16, table_rows=100, num_pages=50, page_size=16, table_width=7,
              prefix_width=30, interleaved=0, dtype=BF16, stream=None, scale=0.125,
              workspace_bytes=1 << 40, q_stride=512, k_stride=128, v_stride=128, out_q_stride=512,
              out_stride=512, page_stride=16 * 128, token_stride=128, head_stride=64)
LATENT = dict(head_dim=576, v_dim=512, kv_heads=1, v_cache=None, q_stride=8 * 576, out_stride=8 * 512,
              page_stride=16 * 576, token_stride=576, head_stride=576)


def call(name, **kw):
    """Call `name` with valid arguments, those in kw in their places."""
    args, nxt = [], 1 << 44
    for a in DECLARED[name]:
        args.append(kw[a] if a in kw else None if a == "cu_seqlens" else nxt if a in POINTERS else VALUES[a])
        nxt += 4 * TB
    return getattr(_lib.lib(), name)(*args)


CALLS = [APPEND, ATTN]


@pytest.mark.parametrize("name", CALLS)
def test_valid_arguments_reach_the_device_check(name):
    assert call(name) == DEVICE
    assert call(name, cu_seqlens=1 << 60, tokens=11) == DEVICE  # ragged
    assert call(name, dtype=F32) == DEVICE
    assert call(name, num_pages=0, k_cache=None, v_cache=None,
                **({"v": None} if name == APPEND else {})) == DEVICE
    assert call(name, table_width=0, page_table=None) == DEVICE
    lat = {**LATENT, "v": None, "k_stride": 576, "out_q_stride": 8 * 576} if name == APPEND else LATENT
    assert call(name, **lat) == DEVICE


REQUIRED = {APPEND: ["q", "k", "table", "positions", "page_table", "lens", "out_q", "k_cache"],
            ATTN: ["q", "k_cache", "v_cache", "page_table", "lens", "prefix_pages", "prefix_len", "out",
                   "workspace"]}
OPTIONAL = {APPEND: ["cu_seqlens"], ATTN: ["lse", "cu_seqlens"]}


@pytest.mark.parametrize("name,arg", [(n, a) for n in CALLS for a in REQUIRED[n]])
def test_required_pointers(name, arg):
    assert call(name, **{arg: None}) == NULL


@pytest.mark.parametrize("name,arg", [(n, a) for n in CALLS for a in OPTIONAL[n]])
def test_optional_pointers(name, arg):
    assert call(name, **{arg: None}) == DEVICE


def test_values_and_their_cache_go_together():
    assert call(APPEND, v=None) == NULL and call(APPEND, v_cache=None) == NULL
    assert call(APPEND, v=None, v_cache=None) == DEVICE
    assert call(ATTN, **{**LATENT, "v_cache": 1 << 60}) == UNSUP
    # without a rotation or queries what they need is not looked at
    assert call(APPEND, rotary_dim=0, table=None, positions=None, table_rows=0) == DEVICE
    assert call(APPEND, q_heads=0, q=None, out_q=None) == DEVICE
    assert call(ATTN, prefix_width=0, prefix_pages=None, prefix_len=None) == DEVICE


@pytest.mark.parametrize("name", CALLS)
@pytest.mark.parametrize("size", ["tokens", "num_seqs", "q_heads", "kv_heads", "num_pages", "page_size",
                                  "table_width", "prefix_width", "rotary_dim", "rotary_offset",
                                  "page_stride", "token_stride", "head_stride"])
def test_negative_sizes(name, size):
    if size in DECLARED[name]:
        assert call(name, **{size: -1}) == SHAPE


@pytest.mark.parametrize("name", CALLS)
def test_shapes(name):
    assert call(name, tokens=13) == SHAPE           # not the same number for each session
    assert call(name, num_seqs=0) == SHAPE and call(name, num_seqs=0, cu_seqlens=1 << 60) == OK
    assert call(name, page_size=0) == SHAPE
    assert call(name, page_size=1 << 20, table_width=1 << 12) == SHAPE  # own tokens pass 32 bits
    assert call(name, dtype=2) == UNSUP
    assert call(name, head_dim=96, v_dim=96) == SHAPE  # longer than the strides
    short = dict(rotary_dim=16, rotary_offset=0) if name == APPEND else dict(v_dim=32)
    assert call(name, head_dim=32, **short) == UNSUP
    assert call(name, q_stride=511) == SHAPE and call(name, q_stride=516) == ALIGN
    # places of two tokens, heads or pages that share bytes
    assert call(name, token_stride=64) == SHAPE and call(name, head_stride=56) == SHAPE
    assert call(name, page_stride=16 * 128 - 8) == SHAPE
    assert call(name, token_stride=64, head_stride=64 * 16) == DEVICE  # a head's tokens together
    assert call(name, token_stride=0, page_size=1, page_stride=128) == DEVICE
    assert call(name, num_pages=1, page_stride=0) == DEVICE
    # places of a head past 2^32 units of their strides' largest power of two
    assert call(name, num_pages=2 ** 31 - 1, page_stride=16 * 128 + 8) == UNSUP
    assert call(name, num_pages=1 << 20, page_stride=1 << 19) == DEVICE
    assert call(name, num_pages=1 << 20, page_stride=(1 << 19) + 64) == UNSUP
    assert call(name, page_stride=(1 << 45) + 8) == SHAPE
    for a in ("page_stride", "token_stride", "head_stride"):
        assert call(name, **{a: VALUES[a] + 4}) in (ALIGN, SHAPE), a
    assert call(name, page_stride=16 * 128 + 4) == ALIGN


def test_append_shapes():
    assert call(APPEND, rotary_dim=24) == UNSUP and call(APPEND, rotary_offset=8) == UNSUP
    assert call(APPEND, rotary_dim=64) == SHAPE and call(APPEND, table_rows=0) == SHAPE
    assert call(APPEND, k_stride=127) == SHAPE and call(APPEND, v_stride=127) == SHAPE
    assert call(APPEND, out_q_stride=511) == SHAPE and call(APPEND, k_stride=132) == ALIGN
    assert call(APPEND, q_heads=2 ** 23, q_stride=1 << 40, out_q_stride=1 << 40) == UNSUP


def test_attention_shapes():
    assert call(ATTN, q_heads=7) == SHAPE and call(ATTN, kv_heads=0) == SHAPE
    assert call(ATTN, scale=0.0) == SHAPE and call(ATTN, scale=-1.0) == SHAPE
    assert call(ATTN, scale=float("nan")) == SHAPE and call(ATTN, scale=float("inf")) == SHAPE
    assert call(ATTN, v_dim=128, out_stride=1024) == UNSUP and call(ATTN, v_dim=0) == SHAPE
    assert call(ATTN, **{**LATENT, "dtype": F32}) == UNSUP
    assert call(ATTN, out_stride=511) == SHAPE and call(ATTN, out_stride=516) == ALIGN
    assert call(ATTN, prefix_width=1 << 28) == SHAPE


@pytest.mark.parametrize("name", CALLS)
def test_alignment(name):
    wide = {"q", "k", "v", "out_q", "k_cache", "v_cache", "table", "out", "workspace"}
    for a in DECLARED[name]:
        if a in POINTERS:
            assert call(name, **{a: (1 << 60) + 1}) == ALIGN, a
            assert call(name, **{a: (1 << 60) + 4}) == (ALIGN if a in wide else DEVICE), a


OUTPUTS = {APPEND: ["out_q", "k_cache", "v_cache"], ATTN: ["out", "lse", "workspace"]}


@pytest.mark.parametrize("name", CALLS)
def test_outputs_overlap_nothing(name):
    at = 1 << 60
    for o in OUTPUTS[name]:
        for a in DECLARED[name]:
            if a != o and a in POINTERS:
                in_place = name == APPEND and {o, a} == {"q", "out_q"}
                assert call(name, **{o: at, a: at}) == (DEVICE if in_place else ALIAS), (o, a)
    if name == APPEND:
        assert call(name, q=at, out_q=at + 16) == ALIAS  # shifted
        assert call(name, q=at, out_q=at, out_q_stride=520) == ALIAS
        # rotated in place in rows that hold q, k and v: 512 + 128 + 128 values
        rows = dict(q=at, out_q=at, k=at + 1024, v=at + 1280, q_stride=768, out_q_stride=768,
                    k_stride=768, v_stride=768)
        assert call(name, **rows) == DEVICE
        assert call(name, **{**rows, "k": at + 1008}) == ALIAS
        assert call(name, **{**rows, "k_stride": 776}) == ALIAS


def test_halves_of_a_page():
    """Keys and values as halves of each page, of each token, of each head; and shifted into
    each other."""
    at, page, row = 1 << 60, 16 * 128 * 2, 128 * 2
    half = dict(k_cache=at, page_stride=2 * 16 * 128)
    assert call(APPEND, **half, v_cache=at + page) == DEVICE
    assert call(APPEND, **half, v_cache=at - page) == DEVICE
    assert call(APPEND, **half, v_cache=at + page - 16) == ALIAS
    assert call(APPEND, **half, v_cache=at + page + 16) == ALIAS  # the last one meets the next page
    tok = dict(k_cache=at, page_stride=2 * 16 * 128, token_stride=256)
    assert call(APPEND, **tok, v_cache=at + row) == DEVICE
    assert call(APPEND, **tok, v_cache=at + row - 16) == ALIAS
    head = dict(k_cache=at, page_stride=2 * 16 * 128, token_stride=256, head_stride=128)
    assert call(APPEND, **head, v_cache=at + 128) == DEVICE
    assert call(APPEND, **head, v_cache=at + 112) == ALIAS
    assert call(APPEND, k_cache=at, v_cache=at + 50 * page) == DEVICE
    assert call(APPEND, k_cache=at, v_cache=at + 49 * page) == ALIAS
    assert call(ATTN, k_cache=at, v_cache=at) == DEVICE  # read only


def test_workspace_size():
    lib = _lib.lib()
    size = lambda **kw: getattr(lib, SIZE)(*[{**VALUES, **kw}[a] for a in DECLARED[SIZE]])
    need = size()
    # what a call of equal sessions or packed ones asks for at most
    assert need > 0 and call(ATTN, workspace_bytes=need) == DEVICE
    assert call(ATTN, cu_seqlens=1 << 60, workspace_bytes=need) == DEVICE
    assert call(ATTN, workspace_bytes=15) == SHAPE
    assert size(tokens=0) == 0 and size(num_seqs=0) == 0 and size(table_width=0, prefix_width=0) == 0
    for kw in (dict(tokens=-1), dict(page_size=0), dict(head_dim=96), dict(dtype=3), dict(q_heads=7),
               dict(v_dim=128), dict(table_width=1 << 30), dict(head_dim=576, v_dim=512, dtype=F32)):
        assert size(**kw) == -1, kw
    # one part alone is the output itself
    assert size(tokens=1, num_seqs=1, table_width=8, prefix_width=0) == 0
    assert call(ATTN, tokens=1, num_seqs=1, table_width=8, prefix_width=0, workspace=None,
                workspace_bytes=0) == DEVICE


@pytest.mark.parametrize("name", CALLS)
def test_empty_work_needs_no_device(name):
    assert call(name, tokens=0) == OK
    assert call(name, tokens=0, num_seqs=0, q=None, lens=None, page_table=None) == OK
    assert call(name, q_heads=0, kv_heads=0) == OK


@pytest.mark.parametrize("name", CALLS)
def test_more_work_than_a_launch_holds(name):
    if name == ATTN:  # 2^24 sessions of eight heads, a workgroup each and more
        assert call(name, tokens=1 << 24, num_seqs=1 << 24, table_width=1, num_pages=4, kv_heads=8,
                    head_stride=64, token_stride=512, page_stride=8192) == UNSUP
    else:             # in several launches
        assert call(name, tokens=1 << 27, num_seqs=1 << 27, table_width=1) == DEVICE


# ---------------------------------------------------------------- Python front end
def tensors(**kw):
    z = torch.zeros
    t = dict(k=z(4, 2, 64), v=z(4, 2, 64), k_cache=z(9, 16, 2, 64), v_cache=z(9, 16, 2, 64),
             page_table=z(4, 3, dtype=torch.int32), lens=z(4, dtype=torch.int32), cu_seqlens=None)
    return {**t, **kw}


def append(**kw):
    return kda.cache_append(**tensors(**kw))


def attend(**kw):
    t = tensors(**kw)
    for n in ("k", "v"):
        t.pop(n)
    t.setdefault("q", torch.zeros(4, 8, 64))
    return kda.prefix_attention(**t)


def test_python_refusals():
    z, i = torch.zeros, lambda *s: torch.zeros(*s, dtype=torch.int32)
    both = [
        (TypeError, dict(k_cache=None)), (ValueError, dict(k_cache=z(9, 16, 64))),
        (ValueError, dict(k_cache=z(9, 16, 2, 32))), (TypeError, dict(k_cache=z(9, 16, 2, 64).bfloat16())),
        (ValueError, dict(v_cache=z(8, 16, 2, 64))), (TypeError, dict(v_cache=z(9, 16, 2, 64).bfloat16())),
        (ValueError, dict(v_cache=z(9, 2, 16, 64).transpose(1, 2))),  # another order in memory
        (ValueError, dict(k_cache=z(9, 16, 64, 2).transpose(2, 3))),  # channels apart
        (ValueError, dict(k_cache=z(9, 0, 2, 64), v_cache=z(9, 0, 2, 64))),
        (ValueError, dict(page_table=i(4))), (ValueError, dict(page_table=i(5, 3))),
        (TypeError, dict(page_table=z(4, 3))), (ValueError, dict(page_table=i(3, 4).t())),
        (ValueError, dict(lens=i(5))), (TypeError, dict(lens=z(4))), (TypeError, dict(lens=None)),
        (ValueError, dict(cu_seqlens=i(4))), (TypeError, dict(cu_seqlens=z(5))),
        (ValueError, dict(page_table=i(3, 3), lens=i(3))),  # four tokens of three sessions
    ]
    for err, kw in both:
        for f in (append, attend):
            if f is attend and kw.get("k_cache", 0) is None:
                err = ValueError
            with pytest.raises(err):
                f(**kw)
    for err, kw in [
        (TypeError, dict(k=None)), (TypeError, dict(k=z(4, 2, 64).half())), (ValueError, dict(k=z(4, 64))),
        (ValueError, dict(v=None)), (ValueError, dict(v_cache=None)), (ValueError, dict(v=z(4, 3, 64))),
        (TypeError, dict(v=z(4, 2, 64).bfloat16())), (ValueError, dict(k=z(4, 64, 2).transpose(1, 2))),
        (ValueError, dict(k=z(1, 2, 64).expand(4, 2, 64))),
        (ValueError, dict(q=z(4, 64))), (ValueError, dict(q=z(3, 8, 64))), (ValueError, dict(q=z(4, 8, 32))),
        (ValueError, dict(out_q=z(4, 8, 64))), (ValueError, dict(table=z(9, 32))),
        (ValueError, dict(positions=i(4))), (ValueError, dict(table=z(32), positions=i(4))),
        (TypeError, dict(table=z(9, 32).double(), positions=i(4))),
        (ValueError, dict(table=z(9, 32), positions=i(5))),
        (ValueError, dict(rotary_offset=1 << 40)),
    ]:
        with pytest.raises(err):
            append(**kw)
    for err, kw in [
        (TypeError, dict(q=None)), (ValueError, dict(q=z(4, 64))), (ValueError, dict(q=z(4, 7, 64))),
        (TypeError, dict(q=z(4, 8, 64).half())), (ValueError, dict(prefix_pages=i(4))),
        (ValueError, dict(prefix_len=i(1))), (ValueError, dict(prefix_pages=i(4, 1), prefix_len=i(1))),
        (ValueError, dict(prefix_pages=i(4), prefix_len=i(2))),
        (TypeError, dict(prefix_pages=z(4), prefix_len=i(1))),
        (ValueError, dict(out=z(4, 8, 32))), (TypeError, dict(out=z(4, 8, 64).bfloat16())),
        (ValueError, dict(lse=z(4, 7))), (TypeError, dict(lse=z(4, 8).double())),
        (ValueError, dict(v_dim=-1)), (ValueError, dict(v_dim=1 << 40)),
        (TypeError, dict(workspace=z(100))),
    ]:
        with pytest.raises(err):
            attend(**kw)
    # everything else is fine: what is missing is the GPU
    for f in (append, attend):
        with pytest.raises(ValueError, match="GPU"):
            f()


def test_python_sizes():
    size = lambda *a: kda.prefix_attention_workspace_size(*a, torch.bfloat16)
    assert size(12, 4, 8, 2, 64, 64, 16, 7, 30) > 0
    with pytest.raises(ValueError):
        size(12, 4, 7, 2, 64, 64, 16, 7, 30)
    with pytest.raises(ValueError):
        size(1 << 40, 4, 8, 2, 64, 64, 16, 7, 30)


def test_the_module_leaves_what_is_not_common():
    """None for anything it does not know: no tensors, too few, other types, CPU tensors."""
    m = _lib.cache_calls()
    t = tensors()
    cpu = [0, t["k"], t["v"], t["k_cache"], t["v_cache"], t["page_table"], t["lens"], None, None, None,
           None, 0, False]
    for args in (cpu, [], cpu[:5], [None] * 13, ["x"] * 13, cpu[:1] + [t["k"].half()] + cpu[2:]):
        assert m.append(*args) is None
    q = torch.zeros(4, 8, 64)
    cpu = [0, q, t["k_cache"], t["v_cache"], t["page_table"], t["lens"], None, None, None, 0.1, 64, True]
    for args in (cpu, [], [None] * 12, ["x"] * 12, cpu[:9] + ["x", 64, True]):
        assert m.attention(*args) is None
    with pytest.raises(TypeError):
        m.bind(1)
