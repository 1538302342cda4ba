"""The kernels of the operators around the layer, run on the CPU (cpu_kernels/).

The GPU's own sources are compiled for the host with bounds checks; every tensor
and workspace lies between unmapped pages, lanes run in three orders whose
results have to agree to the bit, and results are compared with the plain
64-bit forms. So an address out of range, a missing barrier or a result that
depends on timing shows here, on any machine."""
import os
import subprocess
import sys

import pytest

HERE = os.path.join(os.path.dirname(os.path.abspath(__file__)), "cpu_kernels")
sys.path.insert(0, HERE)
import cpu_build  # noqa: E402
sys.path.remove(HERE)


@pytest.fixture(scope="module")
def library(tmp_path_factory):
    if not os.path.exists(cpu_build.CLANG):
        pytest.skip("no ROCm clang here")
    return cpu_build.build(str(tmp_path_factory.mktemp("cpu_kernels")))


@pytest.mark.parametrize("which", ["norm", "conv", "selective"])
def test_kernels_on_cpu(library, which):
    r = subprocess.run([sys.executable, os.path.join(HERE, "cases.py"), library, which],
                       capture_output=True, text=True, timeout=600)
    assert r.returncode == 0 and "all cases done" in r.stdout, (r.returncode, r.stdout[-300:], r.stderr[-2000:])
