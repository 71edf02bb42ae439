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


def unfenced(lines):
    """LDS accesses of one function's lines that follow accesses of the other kind with no wave
    barrier between (in the order of the text): a write after a read, a read after a write."""
    out, last = [], None
    for n, l in enumerate(lines):
        if "wave barrier" in l or re.match(r"\s*s_barrier", l):
            last = None
        kind = re.match(r"\s*ds_(read|write)", l)
        if kind:
            if last and kind.group(1) != last:
                out.append((n, l.strip()))
            last = kind.group(1)
    return out


def test_results_pass_through_lds_between_wave_barriers():
    """A wave's results go to other lanes of it through LDS, without a workgroup barrier: behind the
    main loop of every tile kernel the writes and the reads stand between wave barriers."""
    assert unfenced(["ds_write_b64 v0, v[2:3]", "ds_read_b128 v[4:7], v1"])
    assert not unfenced(["ds_write_b64 v0, v[2:3]", "; wave barrier", "ds_read_b128 v[4:7], v1"])
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
    kernels = re.findall(r"^(_ZN3iq414mx_tile_kernel\w+):[^\n]*\n(.*?)^\.Lfunc_end", text, re.S | re.M)
    assert len(kernels) >= 11
    for name, body in kernels:
        lines = body.split("\n")
        end = max(n for n, l in enumerate(lines) if re.match(r"\s*s_barrier", l))
        assert sum("ds_write" in l for l in lines[end:]) >= 3, name
        assert not unfenced(lines[end:]), (name, unfenced(lines[end:])[:3])
