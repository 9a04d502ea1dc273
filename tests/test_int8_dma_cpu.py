"""The int8 tiles' LDS DMA is inline asm like the prefill GEMM's: its generated code must
not read an SGPR base within five wait states of a VALU write either."""
import os
import subprocess
import tempfile

import pytest

from nvfp4_w4a4_gemm_quantize_amd import build as B
from tests.test_dma_hazard_cpu import WAIT_STATES, hazards


@pytest.mark.timeout(600)
def test_int8_dma_has_no_valu_sgpr_hazard():
    with tempfile.TemporaryDirectory() as d:
        out = os.path.join(d, "int8.s")
        cmd = [B.hipcc()] + B.COMMON + B.DEVICE + ["-x", "hip", "--cuda-device-only", "-S", os.path.join(B.CSRC, "int8.hip"), "-o", out]
        r = subprocess.run(cmd, capture_output=True, text=True)
        assert r.returncode == 0, r.stderr[-2000:]
        ndma, found = hazards(open(out).read())
    assert ndma > 50, "no LDS DMA instructions found: the scan would prove nothing"
    assert not found, "VALU write of an SGPR base within %d wait states of an LDS DMA: %s" % (WAIT_STATES, found[:3])
