"""Every HIP source under csrc/ passes the compiler's host pass without a
warning (a status that nothing looks at is one)."""

import os
import subprocess

import pytest

from bitlinear_w1_a8_amd import build

# the build's flags less the device's target features, which the host pass does not know
FLAGS = [f for f in build.FLAGS if f not in ("-Xclang", "-target-feature", "-packed-fp32-ops")]


@pytest.mark.parametrize("src", build.sources(), ids=os.path.basename)
def test_host_pass_has_no_warnings(src):
    r = subprocess.run([build.HIPCC, *FLAGS, "-Werror", "-Wno-unused-command-line-argument", "--cuda-host-only",
                        "-fsyntax-only", src], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
