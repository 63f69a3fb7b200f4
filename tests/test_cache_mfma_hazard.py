"""The kernels on a paged cache chain no bf16 MFMA shape's result into the other's
accumulator too soon (tests/mfma_hazard.py), hold no packed fp32 instruction, and
set m0 right before each load from memory to LDS.  CPU only."""
import os
import re

import pytest

from mfma_hazard import find_chains
from test_mfma_hazard import CSRC, HIPCC, _asm

pytestmark = pytest.mark.skipif(not os.path.exists(HIPCC), reason="hipcc not available")


@pytest.mark.parametrize("src", ["attn.hip", "cache_append.hip"])
def test_cache_kernels(src, tmp_path):
    asm = _asm(os.path.join(CSRC, src), tmp_path)
    assert not find_chains(asm)
    for op in ("v_pk_add_f32", "v_pk_mul_f32", "v_pk_fma_f32"):
        assert op not in asm
    # the counter of loads on their way is the walks' own: what writes LDS from memory is in
    # assembly that the compiler does not count, each behind its own m0
    loads = [m.start() for m in re.finditer(r"^\s*global_load_lds_dwordx4", asm, re.M)]
    assert bool(loads) == (src == "attn.hip")
    for at in loads:
        before = [ln.strip() for ln in asm[max(0, at - 200): at].splitlines() if ln.strip()][-2:]
        assert before[0].startswith("s_mov_b32 m0,") and before[1] == "s_nop 0", before
