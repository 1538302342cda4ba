"""The kernels of the recurrent block's operators, run on the CPU (cpu_kernels/) like
those in test_kernels_on_cpu.py: bounds, barriers and results that may not depend on the
lanes' order."""
import importlib.util
import os
import subprocess
import sys

import pytest

HERE = os.path.join(os.path.dirname(os.path.abspath(__file__)), "cpu_kernels")


def builder():
    # a copy of the module of its own, whose lists change
    spec = importlib.util.spec_from_file_location("cpu_build_blocks", os.path.join(HERE, "cpu_build.py"))
    build = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(build)
    if not os.path.exists(build.CLANG):
        pytest.skip("no ROCm clang here")
    return build


@pytest.fixture(scope="module")
def library(tmp_path_factory):
    build = builder()
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


def test_growing_states_on_cpu(library):
    """The direct form's log-decays above 0, whose products over tiles are infinite."""
    r = subprocess.run([sys.executable, os.path.join(HERE, "cases_blocks.py"), library, "growth"],
                       capture_output=True, text=True, timeout=900)
    assert r.returncode == 0 and "all cases done" in r.stdout, (r.returncode, r.stdout[-300:], r.stderr[-2000:])


def test_dropped_values_on_cpu(library):
    """Infinities and NaN where the block norm's dropout drops, forward and back."""
    r = subprocess.run([sys.executable, os.path.join(HERE, "cases_blocks.py"), library, "dropped"],
                       capture_output=True, text=True, timeout=900)
    assert r.returncode == 0 and "all cases done" in r.stdout, (r.returncode, r.stdout[-300:], r.stderr[-2000:])


LOST = """
import ctypes, sys
import numpy as np
lib = ctypes.CDLL(sys.argv[1])
size = lib.ssd_recurrence_forward_workspace_size
size.restype = ctypes.c_size_t
L, E = 300, 32  # five tiles of 64 tokens
x, r = np.ones((L, E), np.float32), np.full((L, E), -0.5, np.float32)
y = np.full((L, E), 7, np.float32)
n = size(1, L, E, 0, 0)
ws = np.zeros(n + 256, np.uint8)
at = (ws.ctypes.data + 255) // 256 * 256
p = lambda a: ctypes.c_void_p(a.ctypes.data)
call = lib.ssd_recurrence_forward
assert call(p(x), p(r), None, None, ctypes.c_float(8), None, 1, L, E, 0, None, None, 0, p(y), None, None,
            ctypes.c_void_p(at), ctypes.c_size_t(n), None, None) == 0
if sys.argv[2] == "words":
    assert np.isfinite(y[:64]).all() and np.isnan(y[64:]).all()
else:
    assert (y == 7).all()
print("ended")
"""


@pytest.mark.parametrize("lost", ["words", "tickets"])
def test_waits_end_where_the_workspace_is_lost(tmp_path, lost):
    """Words that tiles wait for never come (as where another call has cleared them), or the
    count of tiles is none: every wait ends, and nothing is written out of its place."""
    build = builder()
    build.SOURCES = ("recurrence.hip", "recurrence_bwd.hip", "dropout.hip", "block_norm.hip", "norm.hip", "blocks_api.hip")
    build.HEADERS += ("recurrence.h", "dropout.h")
    flags = ("-D__builtin_amdgcn_sqrtf=sqrtf", "-D__builtin_amdgcn_s_sleep(x)=",
             "-D__hip_atomic_load(p,o,s)=(*(p))",
             "-D__hip_atomic_store(p,v,o,s)=" + ("(void)(v)" if lost == "words" else "(*(p)=(v))"),
             "-D__hip_atomic_fetch_add(p,v,o,s)=" + ("((*(p)+=(v))-(v))" if lost == "words" else "0x12345678u"),
             "-include", os.path.join(HERE, "vectors.h"))
    lib = build.build(str(tmp_path), flags, {"recurrence.h": lambda t: t.replace("kRecLooks = 1 << 20", "kRecLooks = 16")})
    r = subprocess.run([sys.executable, "-c", LOST, lib, lost], capture_output=True, text=True, timeout=120)
    assert r.returncode == 0 and "ended" in r.stdout, (r.returncode, r.stdout, r.stderr[-2000:])
