"""Builds the kernels of the operators around the layer for the CPU: the same
sources as the GPU's, with launches turned into calls (hip/hip_runtime.h here)
and the few lines that only the GPU's compiler takes replaced."""
import concurrent.futures as cf
import os
import re
import subprocess
import sys

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(os.path.dirname(HERE))
CSRC = os.path.join(ROOT, "structured_state_space_ssd_amd", "csrc")
CLANG = "/opt/rocm/llvm/bin/clang++"
SOURCES = ("conv.hip", "norm.hip", "selective.hip", "selective_bwd.hip", "layers_api.hip")
HEADERS = ("ssd_launch.h", "ssd_rows.h", "selective.h", "ssd_common.h")

ALLOC = r"""
#include <hip/hip_runtime.h>
// `bytes` between two unmapped pages, right before the second (right) or behind the first.
extern "C" void *cpu_alloc(size_t bytes, int right) {
    const size_t page = 4096, body = (bytes + page - 1) / page * page + (bytes == 0 ? page : 0);
    char *p = (char *)mmap(nullptr, body + 2 * page, PROT_NONE, MAP_PRIVATE | MAP_ANONYMOUS, -1, 0);
    if (p == MAP_FAILED || mprotect(p + page, body, PROT_READ | PROT_WRITE)) abort();
    return p + page + (right ? body - bytes : 0);
}
extern "C" void cpu_free(void *p, size_t bytes, int right) {
    const size_t page = 4096, body = (bytes + page - 1) / page * page + (bytes == 0 ? page : 0);
    munmap((char *)p - page - (right ? body - bytes : 0), body + 2 * page);
}
extern "C" void cpu_order(int order) { cpu::order = order; }
"""


def _closing(s, i):
    """Index after the parenthesis that closes the one before i."""
    depth = 1
    while depth:
        depth += {"(": 1, ")": -1}.get(s[i], 0)
        i += 1
    return i


def _split(s):
    """The parts of s between commas outside brackets."""
    parts, depth, part = [], 0, ""
    for c in s:
        if c == "," and depth == 0:
            parts.append(part)
            part = ""
            continue
        depth += (c in "([{<") - (c in ")]}>")
        part += c
    return parts + [part]


def transform(name, s):
    if name == "ssd_common.h":  # of it only what comes before the matrix fragments
        s = s[:s.index("// ---- MFMA operand fragments")]
        s = re.sub(r"typedef __bf16 \w+ __attribute__.*\n", "", s)
        s += ("inline int wave_id() { return threadIdx.x >> 6; }\n"
              "inline int lane_id() { return threadIdx.x & 63; }\n}  // namespace ssd\n")
    s = re.sub(r'asm volatile\("" : "\+[vs]"\(\w+\)\);', "", s)
    # (volatile: loads ahead of their use are made even where nothing uses them)
    s = s.replace("__attribute__((address_space(4)))", "volatile")
    s = s.replace("__builtin_bit_cast(uint32_t, __builtin_convertvector((f2{a, b}), b2))",
                  "static_cast<uint32_t>(from_f32<bf16_t>(a)) | static_cast<uint32_t>(from_f32<bf16_t>(b)) << 16")
    s = re.sub(r"typedef __bf16 b2 __attribute__.*\n|typedef float f2 __attribute__.*\n", "", s)
    launch = re.compile(r"(\w+_kernel(?:<[^;{}]*?>)?)(\s*\\?\s*)<<<(.*?)>>>\(", re.S)
    out, at = "", 0
    while m := launch.search(s, at):
        end = _closing(s, m.end())
        grid, threads = _split(m.group(3).replace("\\\n", ""))[:2]
        args = s[m.end():end - 1]
        out += (s[at:m.start()] + f"cpu::launch(dim3({grid}), {threads}, [=] {{ {m.group(1)}("
                + args + "); })")
        at = end
    return out + s[at:]


def build(out_dir, flags=(), patch=None):
    """Returns the path of the shared library. patch: name -> (text -> text)."""
    src = os.path.join(out_dir, "src")
    os.makedirs(src, exist_ok=True)
    for name in SOURCES + HEADERS:
        with open(os.path.join(CSRC, name)) as f:
            text = f.read()
        if patch and name in patch:
            text = patch[name](text)
        with open(os.path.join(src, name.replace(".hip", ".cpp")), "w") as f:
            f.write(transform(name, text))
    with open(os.path.join(src, "alloc.cpp"), "w") as f:
        f.write(ALLOC)
    # bounds of every array, shifts, divisions and int overflows trap
    checks = ["-fsanitize=bounds,shift,integer-divide-by-zero,signed-integer-overflow", "-fsanitize-trap=all"]
    common = [CLANG, "-std=c++20", "-O1", "-fPIC", "-w", "-U_FORTIFY_SOURCE", "-ffp-contract=off", *checks,
              *flags, f"-I{HERE}", f"-I{src}", f"-I{os.path.join(ROOT, 'include')}"]

    def one(name):
        cpp = os.path.join(src, name)
        r = subprocess.run([*common, "-c", cpp, "-o", cpp + ".o"], capture_output=True, text=True)
        if r.returncode:
            raise RuntimeError(r.stderr[-4000:])
        return cpp + ".o"

    names = [n.replace(".hip", ".cpp") for n in SOURCES] + ["alloc.cpp"]
    with cf.ThreadPoolExecutor(max_workers=6) as ex:
        objs = list(ex.map(one, names))
    lib = os.path.join(out_dir, "liblayers_cpu.so")
    subprocess.run([CLANG, "-shared", *objs, "-lm", "-o", lib], check=True)
    return lib


if __name__ == "__main__":
    print(build(sys.argv[1]))
