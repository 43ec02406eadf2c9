"""Audit of the KV cache attention's compiled code (no GPU needed).

The barriers between the tile kernel's phases wait for LDS accesses alone, so that
global loads stay in flight over them. That is only sound while the kernels reach LDS
by LDS instructions: a flat access, which the compiler chooses where it has lost sight
of the address space (in a function that it did not inline), is counted otherwise. So
this test compiles the source for gfx950 and checks that there are no flat accesses and
no calls."""
import os
import re
import subprocess

import pytest

from test_asm_audit import ROOT, _hipcc

SRC = os.path.join(ROOT, "rotation_w4a4_quantized_amd", "csrc", "kv_attention.hip")


@pytest.mark.skipif(_hipcc() is None, reason="hipcc not available")
def test_attention_has_no_flat_access_and_no_call(tmp_path):
    from rotation_w4a4_quantized_amd import build as B
    out = tmp_path / "kv_attention.s"
    cmd = [_hipcc(), "-x", "hip", *B.FLAGS, "--cuda-device-only", "-S", SRC, "-o", str(out)]
    p = subprocess.run(cmd, capture_output=True, text=True)
    assert p.returncode == 0, p.stderr[-2000:]
    lines = [ln.strip() for ln in out.read_text().splitlines()]
    code = [ln for ln in lines if ln and not ln.startswith((";", ".", "//")) and not ln.endswith(":")]
    bad = [ln for ln in code if re.match(r"flat_|s_swappc|s_setpc", ln)]
    assert not bad, bad[:4]
    assert sum(ln.startswith("ds_read") for ln in code) > 0     # the kernels were compiled
