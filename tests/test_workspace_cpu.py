"""Where the parts of a caller's workspace lie: csrc/workspace_check.cpp runs the library's own
carving (host code) for every start that the 16-byte rule allows."""
import os
import shutil
import subprocess

import pytest

from bit_nf4_quantized_19_b200 import build

HERE = os.path.dirname(os.path.abspath(__file__))


@pytest.mark.skipif(shutil.which("g++") is None, reason="needs g++")
def test_parts_lie_on_256_byte_addresses_inside_the_workspace(tmp_path):
    exe = str(tmp_path / "workspace_check")
    subprocess.run(["g++", "-std=c++17", "-O1", "-Wall", "-Werror", "-I", build.CSRC,
                    os.path.join(HERE, "csrc", "workspace_check.cpp"), "-o", exe], check=True)
    res = subprocess.run([exe], capture_output=True, text=True, timeout=60)
    assert res.returncode == 0, res.stdout + res.stderr
    assert int(res.stdout.split()[0]) == 4 * 32 * (6 * 3 + 1)
