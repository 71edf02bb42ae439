"""The microscaled products' global->LDS copies are inline assembly too: every copy in the
assembly of csrc/mx.hip is checked against the wait states that test_asm_hazards.py states
(a vector write of a scalar register before a copy reads it, a scalar write of M0)."""
import os
import re
import shutil
import subprocess
import tempfile

import pytest

from test_asm_hazards import hazards


def test_mx_copies_respect_sgpr_and_m0_wait_states():
    from dequant_matmul_iq4_amd import build as B
    if not (os.path.exists(B.HIPCC) or shutil.which(B.HIPCC)):
        pytest.skip("hipcc not available")
    flags = [f for f in B.FLAGS if f != "-fPIC"]
    with tempfile.TemporaryDirectory() as d:
        out = os.path.join(d, "mx.s")
        r = subprocess.run([B.HIPCC, *flags, "--offload-device-only", "-S", "-o", out, os.path.join(B.CSRC, "mx.hip")],
                           capture_output=True, text=True)
        assert r.returncode == 0, r.stderr[-2000:]
        lines = open(out).read().split("\n")
    assert sum("global_load_lds" in l for l in lines) > 50
    bad = hazards(lines)
    assert not bad, bad[:5]


def test_mx_copies_from_lane_addresses_respect_m0_wait_states():
    """The copies whose address is in a pair of vector registers read M0 alone."""
    from dequant_matmul_iq4_amd import build as B
    if not (os.path.exists(B.HIPCC) or shutil.which(B.HIPCC)):
        pytest.skip("hipcc not available")
    flags = [f for f in B.FLAGS if f != "-fPIC"]
    with tempfile.TemporaryDirectory() as d:
        out = os.path.join(d, "mx.s")
        r = subprocess.run([B.HIPCC, *flags, "--offload-device-only", "-S", "-o", out, os.path.join(B.CSRC, "mx.hip")],
                           capture_output=True, text=True)
        assert r.returncode == 0, r.stderr[-2000:]
        text = open(out).read()
    # s[200:201] exists in no kernel: what is left of the scan is M0
    far = r"(global_load_lds_dwordx4)\s+v\[\d+:\d+\],\s*off"
    lines = re.sub(far, r"\1 v0, s[200:201]", text).split("\n")
    assert sum("s[200:201]" in l for l in lines) > 20
    assert hazards(["s_mov_b32 m0, s9", "global_load_lds_dwordx4 v0, s[200:201]"])
    bad = hazards(lines)
    assert not bad, bad[:5]
