"""The short division of the routing scores equals the IEEE division: built and run as a standalone CUDA program."""
import os
import re
import subprocess

import pytest

from mxfp8_precision_gemms_fp8bw_gb300 import build

pytestmark = pytest.mark.gpu

HERE = os.path.dirname(os.path.abspath(__file__))


def test_route_division(tmp_path):
    exe = str(tmp_path / "route_division")
    cmd = [build._nvcc(), *build.ARCH, "-O3", "-std=c++17", "-I" + build.CSRC,
           os.path.join(HERE, "cuda", "route_division.cu"), "-o", exe]
    subprocess.run(cmd, check=True, capture_output=True, text=True)
    r = subprocess.run([exe], capture_output=True, text=True, timeout=300)
    m = re.search(r"checked (\d+) mismatches (\d+)", r.stdout)
    assert m, r.stdout + r.stderr
    assert int(m.group(1)) == 24576 << 23 and int(m.group(2)) == 0, r.stdout
