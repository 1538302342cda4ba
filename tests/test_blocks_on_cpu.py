"""The kernels of the recurrent block's operators, run on the CPU (cpu_kernels/) like
those in test_kernels_on_cpu.py: bounds, barriers and results that may not depend on the
lanes' order."""
import importlib.util
import os
import subprocess
import sys

import pytest

HERE = os.path.join(os.path.dirname(os.path.abspath(__file__)), "cpu_kernels")


@pytest.fixture(scope="module")
def library(tmp_path_factory):
    # a copy of the module of its own, whose lists grow
    spec = importlib.util.spec_from_file_location("cpu_build_blocks", os.path.join(HERE, "cpu_build.py"))
    build = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(build)
    if not os.path.exists(build.CLANG):
        pytest.skip("no ROCm clang here")
    build.SOURCES += ("recurrence.hip", "recurrence_bwd.hip", "dropout.hip", "block_norm.hip", "blocks_api.hip")
    build.HEADERS += ("recurrence.h", "dropout.h")
    # (workgroups run one after the other, so a word that one waits for is there, or never comes)
    flags = ("-D__builtin_amdgcn_sqrtf=sqrtf", "-D__builtin_amdgcn_s_sleep(x)=cpu::fail(\"waits for what does not come\")",
             "-D__hip_atomic_load(p,o,s)=(*(p))", "-D__hip_atomic_store(p,v,o,s)=(*(p)=(v))",
             "-D__hip_atomic_fetch_add(p,v,o,s)=((*(p)+=(v))-(v))", "-include", os.path.join(HERE, "vectors.h"))
    return build.build(str(tmp_path_factory.mktemp("cpu_blocks")), flags)


@pytest.mark.parametrize("which", ["recurrence", "dropout", "block"])
def test_blocks_on_cpu(library, which):
    r = subprocess.run([sys.executable, os.path.join(HERE, "cases_blocks.py"), library, which],
                       capture_output=True, text=True, timeout=900)
    assert r.returncode == 0 and "all cases done" in r.stdout, (r.returncode, r.stdout[-300:], r.stderr[-2000:])
