"""No copy between registers is lost in the packed convolution's kernels.

The compiler has taken the upper half of a two-register value for undefined where a loop's body got
it from one of two places, a register or a load (the row of 8 bytes per lane that becomes the
window's newest): the copy that moves the window on was dropped from the machine code.  The
assembly names such a copy `kill: def $vgprA killed $vgprB` with two registers that have nothing
in common; where nothing has been dropped, both sides are the same register."""
import os
import re
import shutil
import subprocess

import pytest

from selective_state_space_20_amd import build

LOST = re.compile(r"; kill: def \$(\S+) killed (?:killed )?\$(\S+)")


def lost_copies(assembly):
    parts = lambda name: set(re.findall(r"[vsa]gpr\d+", name))
    return [line.strip() for line, m in ((line, LOST.search(line)) for line in assembly.splitlines())
            if m and not parts(m.group(1)) & parts(m.group(2))]


def test_the_search_finds_one():
    kept = "\t; kill: def $vgpr2 killed $vgpr2 killed $exec\n\t; kill: def $vgpr2_vgpr3 killed $vgpr2 killed $exec\n"
    assert lost_copies(kept) == []
    assert len(lost_copies(kept + "\t; kill: def $vgpr33 killed $vgpr37 killed $exec\n")) == 1


@pytest.mark.skipif(shutil.which("hipcc") is None, reason="needs hipcc")
def test_packed_convolution_keeps_its_copies(tmp_path):
    src, out = os.path.join(build.CSRC, "packed_conv.hip"), str(tmp_path / "packed_conv.s")
    subprocess.run(["hipcc", *build.FLAGS, "-I", os.path.join(build.ROOT, "include"), "-I", build.CSRC, "-S",
                    "--offload-device-only", src, "-o", out], check=True, capture_output=True)
    with open(out) as f:
        text = f.read()
    assert "packed_conv_kernel" in text
    assert lost_copies(text) == []
