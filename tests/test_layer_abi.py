"""The C ABI of include/kda_layer.h: exports, and the refusal of bad arguments on
the host before any device work; and the Python front end's own refusals (no GPU
needed).  Pointers are fake addresses far apart: validation never reads them.
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
GB = 1 << 30


def declared():
    text = open(os.path.join(ROOT, "include", "kda_layer.h")).read()
    text = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
    out = {}
    for name, args in re.findall(r"\b(kda_\w+)\s*\(([^)]*)\)\s*;", text):
        out[name] = [a.split()[-1].lstrip("*") for a in args.split(",")]
    return out


DECLARED = declared()


def test_library_exports_what_the_header_declares():
    handle = ctypes.CDLL(_lib.LIB_PATH)
    assert set(DECLARED) == set(_lib.LAYER_SIGNATURES)
    assert not set(_lib.LAYER_SIGNATURES) & set(_lib.SIGNATURES)
    for name, args in DECLARED.items():
        assert hasattr(handle, name), name
        assert len(_lib.LAYER_SIGNATURES[name][0]) == len(args), name


POINTERS = {"x", "weight", "bias", "initial_state", "cu_seqlens", "out", "final_state", "d_out",
            "d_final_state", "dx", "dweight", "dbias", "d_initial_state", "workspace", "state", "q",
            "k", "q_weight", "k_weight", "table", "positions", "out_q", "out_k", "d_out_q",
            "d_out_k", "dq", "dk", "dq_weight", "dk_weight", "dt", "A", "B", "C", "D", "ddt", "dA",
            "dB", "dC", "dD"}
SIZES = dict(batch=2, seq_len=50, channels=24, width=4, num_seqs=0, activation=1, dtype=BF16,
             workspace_bytes=1 << 40, stream=None, tokens=9, q_heads=4, k_heads=2, head_dim=64,
             rotary_dim=32, table_rows=100, eps=1e-6, norm=0, interleaved=0, num_heads=4,
             num_groups=2, state_dim=128)


def call(name, **kw):
    """Call `name` with valid arguments, those in kw in their places."""
    args, nxt = [], 1 << 40
    for a in DECLARED[name]:
        if a in kw:
            args.append(kw[a])
        elif a == "cu_seqlens":
            args.append(None)
        elif a in POINTERS:
            args.append(nxt)
        elif a in SIZES:
            args.append(SIZES[a])
        else:
            assert a.endswith("_stride"), a
            args.append({"kda_qk": 512, "kda_ss": 512}.get(name[:6], 24))
        nxt += 64 * GB
    return getattr(_lib.lib(), name)(*args)


CALLS = sorted(n for n in DECLARED if not n.endswith("_size"))


@pytest.mark.parametrize("name", CALLS)
def test_valid_arguments_reach_the_device_check(name):
    assert call(name) == DEVICE


REQUIRED = {
    "kda_short_conv_fwd": ["x", "weight", "out"],
    "kda_short_conv_bwd": ["x", "weight", "d_out", "dx", "dweight", "workspace"],
    "kda_short_conv_step": ["x", "weight", "state", "out"],
    "kda_qk_norm_fwd": ["q", "k", "table", "positions", "out_q", "out_k"],
    "kda_qk_norm_bwd": ["q", "k", "table", "positions", "d_out_q", "d_out_k", "dq", "dk",
                        "workspace"],
    "kda_ssm_chunk_fwd": ["x", "dt", "A", "B", "C", "out"],
    "kda_ssm_chunk_bwd": ["x", "dt", "A", "B", "C", "d_out", "dx", "ddt", "dA", "dB", "dC",
                          "workspace"],
    "kda_ssm_decode_step": ["x", "dt", "A", "B", "C", "state", "out"],
}


@pytest.mark.parametrize("name,arg", [(n, a) for n, v in REQUIRED.items() for a in v])
def test_required_pointers(name, arg):
    assert call(name, **{arg: None}) == NULL


OPTIONAL = {
    "kda_short_conv_fwd": ["bias", "initial_state", "final_state"],
    "kda_short_conv_bwd": ["bias", "initial_state", "d_final_state", "dbias", "d_initial_state"],
    "kda_short_conv_step": ["bias"],
    "kda_qk_norm_fwd": ["q_weight", "k_weight"],
    "kda_ssm_chunk_fwd": ["D", "initial_state", "final_state"],
    "kda_ssm_chunk_bwd": ["dD", "initial_state", "d_final_state", "d_initial_state"],
    "kda_ssm_decode_step": ["D"],
}


@pytest.mark.parametrize("name,arg", [(n, a) for n, v in OPTIONAL.items() for a in v])
def test_optional_pointers(name, arg):
    assert call(name, **{arg: None}) == DEVICE


def test_gradients_of_what_was_not_given():
    assert call("kda_qk_norm_bwd", q_weight=None) == NULL
    assert call("kda_qk_norm_bwd", q_weight=None, dq_weight=None) == DEVICE
    assert call("kda_ssm_chunk_bwd", D=None) == NULL
    assert call("kda_ssm_chunk_bwd", D=None, dD=None) == DEVICE


@pytest.mark.parametrize("name", CALLS)
@pytest.mark.parametrize("size", ["batch", "seq_len", "channels", "tokens", "q_heads", "k_heads",
                                  "num_heads", "num_groups"])
def test_negative_sizes(name, size):
    if size in DECLARED[name]:
        assert call(name, **{size: -1}) == SHAPE


@pytest.mark.parametrize("name", CALLS)
def test_types_and_configurations(name):
    assert call(name, dtype=2) == UNSUP
    if "width" in DECLARED[name]:
        assert call(name, width=1) == UNSUP and call(name, width=5) == UNSUP
        assert call(name, width=0) == SHAPE
        rows = {a: 1 << 30 for a in DECLARED[name] if a.endswith("_stride")}
        assert call(name, channels=(1 << 29) + 1, **rows) == UNSUP  # a row passes 2^31 bytes
        assert call(name, activation=2) == UNSUP
    if "head_dim" in DECLARED[name]:
        assert call(name, head_dim=96) == UNSUP
    if "state_dim" in DECLARED[name]:
        assert call(name, state_dim=32) == UNSUP and call(name, state_dim=0) == SHAPE
        assert call(name, num_groups=3) == SHAPE and call(name, num_groups=0) == SHAPE
    if "norm" in DECLARED[name]:
        assert call(name, norm=2) == UNSUP and call(name, rotary_dim=24) == UNSUP
        assert call(name, rotary_dim=80) == SHAPE and call(name, eps=-1.0) == SHAPE
        assert call(name, eps=float("nan")) == SHAPE and call(name, table_rows=0) == SHAPE


@pytest.mark.parametrize("name", CALLS)
def test_strides(name):
    for a in DECLARED[name]:
        if a.endswith("_stride"):
            assert call(name, **{a: 8}) == SHAPE, a
            if not name.startswith("kda_short_conv"):
                assert call(name, **{a: 516}) == ALIGN, a  # rows not on 16 bytes
            else:
                assert call(name, **{a: 25}) == DEVICE, a  # any distance
            if name.startswith("kda_ssm"):
                assert call(name, **{a: 1 << 25}) == UNSUP, a  # 64 rows pass 2^31 bytes


@pytest.mark.parametrize("name", CALLS)
def test_alignment(name):
    fine = {"x", "out", "initial_state", "final_state", "d_out", "d_final_state", "dx",
            "d_initial_state", "state"} if name.startswith("kda_short_conv") else set()
    for a in DECLARED[name]:
        if a in POINTERS and a != "cu_seqlens":
            assert call(name, **{a: (1 << 50) + 1}) == ALIGN, a
            four = {"weight", "bias", "dweight", "dbias", "q_weight", "k_weight", "dq_weight",
                    "dk_weight", "positions", "dt", "A", "D", "ddt", "dA", "dD"}
            want = DEVICE if a in fine or a in four else ALIGN
            assert call(name, **{a: (1 << 50) + 4}) == want, a
    if "cu_seqlens" in DECLARED[name]:
        assert call(name, batch=1, cu_seqlens=(1 << 50) + 2, num_seqs=3) == ALIGN


OUTPUTS = {
    "kda_short_conv_fwd": ["out", "final_state"],
    "kda_short_conv_bwd": ["dx", "dweight", "dbias", "d_initial_state", "workspace"],
    "kda_short_conv_step": ["out", "state"],
    "kda_qk_norm_fwd": ["out_q", "out_k"],
    "kda_qk_norm_bwd": ["dq", "dk", "dq_weight", "dk_weight", "workspace"],
    "kda_ssm_chunk_fwd": ["out", "workspace", "final_state"],
    "kda_ssm_chunk_bwd": ["dx", "ddt", "dA", "dB", "dC", "dD", "d_initial_state", "workspace"],
    "kda_ssm_decode_step": ["out", "state"],
}


@pytest.mark.parametrize("name", CALLS)
def test_outputs_overlap_nothing(name):
    at = 1 << 50
    big = dict(seq_len=2000) if name == "kda_ssm_chunk_fwd" else {}  # uses its workspace
    for o in OUTPUTS[name]:
        for a in DECLARED[name]:
            if a == o or a not in POINTERS:
                continue
            kw = dict(big)
            if a == "cu_seqlens":
                kw.update(batch=1, num_seqs=3)
            in_place = name == "kda_ssm_chunk_fwd" and {o, a} == {"final_state", "initial_state"}
            assert call(name, **{**kw, o: at, a: at}) == (DEVICE if in_place else ALIAS), (o, a)
    if name == "kda_ssm_chunk_fwd":  # in place, but not shifted
        assert call(name, initial_state=at, final_state=at + 64) == ALIAS


def test_slices_of_one_row_do_not_overlap():
    """dx | dB | dC side by side in rows of 512 + 2 * 256 + 8 elements (bf16), and
    the same shifted by one 16-byte piece into each other."""
    at, row = 1 << 50, 1032
    kw = dict(dx_stride=row, db_stride=row, dc_stride=row, head_dim=128, dx=at)
    assert call("kda_ssm_chunk_bwd", **kw, x_stride=512, dB=at + 1024, dC=at + 1536) == DEVICE
    assert call("kda_ssm_chunk_bwd", **kw, x_stride=512, dB=at + 1008, dC=at + 1536) == ALIAS
    assert call("kda_ssm_chunk_bwd", **kw, x_stride=512, dB=at + 1024, dC=at + 1520) == ALIAS
    # ... or past the row's end into the next token's dx
    assert call("kda_ssm_chunk_bwd", **kw, x_stride=512, dB=at + 1024, dC=at + 1568) == ALIAS
    # another distance between tokens: by first and last byte
    assert call("kda_ssm_chunk_bwd", **{**kw, "db_stride": row + 8}, dB=at + 1024) == ALIAS


@pytest.mark.parametrize("name", [n for n in CALLS if "cu_seqlens" in DECLARED[n]])
def test_packed_needs_one_row(name):
    assert call(name, cu_seqlens=1 << 50, num_seqs=3) == SHAPE
    assert call(name, batch=1, cu_seqlens=1 << 50, num_seqs=-1) == SHAPE
    assert call(name, batch=1, cu_seqlens=1 << 50, num_seqs=3) == DEVICE
    assert call(name, batch=1 << 16, seq_len=1 << 16) == SHAPE  # tokens pass int32
    assert call(name, batch=1, seq_len=2 ** 31 - 4095) == SHAPE


@pytest.mark.parametrize("name", [n for n in CALLS if "workspace" in DECLARED[n]])
def test_workspace_size(name):
    kw = dict(seq_len=2000) if name.startswith("kda_ssm") else {}
    size = getattr(_lib.lib(), name + "_workspace_size")(
        *[{**SIZES, **kw}[a] for a in DECLARED[name + "_workspace_size"]])
    assert size > 0
    assert call(name, **kw, workspace_bytes=size) == DEVICE
    assert call(name, **kw, workspace_bytes=size - 1) == SHAPE


def test_empty_work_needs_no_device():
    assert call("kda_short_conv_fwd", channels=0) == OK
    assert call("kda_short_conv_fwd", batch=0, x=None, out=None) == OK
    assert call("kda_short_conv_step", batch=0) == OK
    assert call("kda_qk_norm_fwd", tokens=0, q=None, k=None) == OK
    assert call("kda_qk_norm_fwd", q_heads=0, k_heads=0) == OK
    assert call("kda_qk_norm_bwd", tokens=0, dq_weight=None, dk_weight=None) == OK
    assert call("kda_ssm_chunk_fwd", batch=0) == OK
    assert call("kda_ssm_chunk_fwd", num_heads=0, num_groups=0) == OK
    assert call("kda_ssm_decode_step", batch=0) == OK
    # gradients of parameters are written all the same
    assert call("kda_short_conv_bwd", batch=0) == DEVICE
    assert call("kda_ssm_chunk_bwd", batch=0) == DEVICE


# ---------------------------------------------------------------- Python front end
def test_python_refusals():
    z = torch.zeros
    x, w = z(1, 4, 8), z(8, 4)
    for err, f in [
        (ValueError, lambda: kda.short_conv(x[0], w)),                      # 2-D
        (ValueError, lambda: kda.short_conv(x, z(7, 4))),                   # channels
        (TypeError, lambda: kda.short_conv(x, w.double())),
        (TypeError, lambda: kda.short_conv(x.half(), w)),
        (ValueError, lambda: kda.short_conv(x, w, activation="gelu")),
        (ValueError, lambda: kda.short_conv(x.transpose(1, 2), z(4, 4))),   # a token in pieces
        (ValueError, lambda: kda.short_conv(z(1, 1, 8).expand(1, 4, 8), w)),  # tokens overlap
        (ValueError, lambda: kda.short_conv(z(3, 4, 8)[:, :2], w)),         # uneven distances
        (ValueError, lambda: kda.short_conv(x, w, cu_seqlens=z(0, dtype=torch.int32))),
        (TypeError, lambda: kda.short_conv(x, w, cu_seqlens=z(2))),
        (ValueError, lambda: kda.short_conv(z(2, 4, 8), w, cu_seqlens=z(2, dtype=torch.int32))),
        (ValueError, lambda: kda.short_conv(x, w, initial_state=z(1, 4, 8))),
        (TypeError, lambda: kda.short_conv(x, w, initial_state=z(1, 3, 8).bfloat16())),
        (TypeError, lambda: kda.short_conv_step(z(2, 8), w, None)),
        (ValueError, lambda: kda.short_conv_bwd(x, w, z(1, 4, 9))),
        (ValueError, lambda: kda.qk_norm(z(1, 2, 3, 64), z(1, 3, 3, 64))),  # leading axes
        (ValueError, lambda: kda.qk_norm(z(1, 2, 3, 64), z(1, 2, 3, 64), kind="max")),
        (ValueError, lambda: kda.qk_norm(z(1, 2, 3, 64), z(1, 2, 3, 64), table=z(4, 32))),
        (TypeError, lambda: kda.qk_norm(z(1, 2, 3, 64), z(1, 2, 3, 64), table=z(4, 32),
                                        positions=z(1, 2, dtype=torch.int64))),
        (ValueError, lambda: kda.ssm_chunk_fwd(z(1, 2, 3, 64), z(1, 2, 3), z(3), z(1, 2, 2, 64),
                                               z(1, 2, 2, 64))),            # 3 heads, 2 groups
        (TypeError, lambda: kda.ssm_chunk_fwd(z(1, 2, 3, 64), None, z(3), z(1, 2, 1, 64),
                                              z(1, 2, 1, 64))),
        (ValueError, lambda: kda.ssm_chunk_fwd(z(1, 2, 3, 64), z(1, 2, 3), z(3), z(1, 2, 1, 64),
                                               z(1, 2, 1, 128))),
        (ValueError, lambda: kda.ssm_decode_step(z(2, 3, 64), z(2, 3), z(3), z(2, 1, 64),
                                                 z(2, 1, 64), z(2, 3, 64, 65))),
        (ValueError, lambda: kda.short_conv(x, w)),                         # not on a GPU
    ]:
        with pytest.raises(err):
            f()
