"""The scan's kernels chain no bf16 MFMA shape's result into the other's
accumulator too soon (tests/mfma_hazard.py): every kernel here uses one shape,
and the compiled assembly is scanned as for the rest of the library.  No packed
fp32 instruction is left in the layer operators' code either.  CPU only."""
import os

import pytest

from mfma_hazard import find_chains
from test_mfma_hazard import CSRC, HIPCC, _asm

pytestmark = pytest.mark.skipif(not os.path.exists(HIPCC), reason="hipcc not available")


@pytest.mark.parametrize("src", ["ssm_scan.hip", "ssm_bwd.hip", "ssm_step.hip", "conv.hip",
                                 "qk_norm.hip"])
def test_layer_kernels(src, tmp_path):
    asm = _asm(os.path.join(CSRC, src), tmp_path)
    assert not find_chains(asm)
    for op in ("v_pk_add_f32", "v_pk_mul_f32", "v_pk_fma_f32"):
        assert op not in asm
