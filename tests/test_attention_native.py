"""The attention kernels' gfx950 assembly (no GPU): what their hand-counted copies rely on.

Every direct-to-LDS copy comes right after the m0 write that gives its destination and wait states: s_nop 4, or, for the
second copy of a pair, whose operands were ready before the first one's wait, s_nop 0.  The kernel of few rows counts its
copies in flight, so none of its registers may be spilled to memory."""
from __future__ import annotations

import os
import re
import subprocess

import pytest

from fp8_block_scaled_a8w8_amd import build

DMA = re.compile(r"^\s*(buffer_load_dword\w*\s.*\blds\b|global_load_lds_dword\w*\s)")


@pytest.fixture(scope="module")
def assembly(tmp_path_factory):
    try:
        hipcc = build.hipcc()
    except RuntimeError:
        pytest.skip("hipcc not available")
    out = str(tmp_path_factory.mktemp("attention") / "attention.s")
    flags = [f for f in build.HIPCC_FLAGS if f != "-shared"]
    res = subprocess.run([hipcc, *flags, "-S", "--offload-device-only", "-I", os.path.join(build.ROOT, "include"), "-I",
                          os.path.join(build.HERE, "csrc"), os.path.join(build.HERE, "csrc", "a8w8_attention.hip"), "-o", out],
                         capture_output=True, text=True)
    assert res.returncode == 0, res.stderr[-2000:]
    with open(out) as f:
        return f.read()


def test_every_copy_is_padded_after_its_m0_write(assembly):
    lines = [ln.strip() for ln in assembly.splitlines() if ln.strip() and not ln.strip().startswith(";")]
    copies = [i for i, ln in enumerate(lines) if DMA.match(ln)]
    assert len(copies) > 200
    for i in copies:
        second = DMA.match(lines[i - 3]) is not None
        assert lines[i - 1] == "s_nop 4" or (second and lines[i - 1] == "s_nop 0"), (i, lines[i - 3:i + 1])
        assert re.match(r"s_mov_b32 m0, (s\d+|vcc_lo|vcc_hi)$", lines[i - 2]), (i, lines[i - 3:i + 1])


def test_the_kernel_of_few_rows_spills_nothing(assembly):
    found = re.findall(r"\.name:\s+(\S*few_kernel\S*).*?\.private_segment_fixed_size:\s+(\d+)", assembly, re.S)
    assert len(found) == 6
    assert all(int(size) == 0 for _, size in found), found
