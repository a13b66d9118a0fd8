"""Builds and runs the programs of tests/cpu_wave: the library's kernel sources,
launches included, compiled for the host and run on guarded memory."""
import os
import shutil
import subprocess

import numpy as np
import pytest

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CLANG = next((c for c in ("/opt/rocm/llvm/bin/clang++", shutil.which("clang++")) if c and os.path.exists(c)), None)
STATUS = {-11: "an access outside a buffer", -7: "an access outside a buffer", 3: "a wait that never ends, or a copy out of place",
          6: "refused", 7: "the workspace's counters are not cleared", 8: "outputs differ between the turns"}


def build(folder, name):
    if CLANG is None:
        pytest.skip("no clang++ (ROCm's)")
    out = os.path.join(str(folder), name)
    subprocess.run([CLANG, "-x", "c++", "-std=c++17", "-O2", "-Wall", "-Wno-unused-function", "-Wno-psabi", "-Wno-pass-failed",
                    "-I", os.path.join(HERE, "cpu_wave"), "-I", os.path.join(ROOT, "block_scaled_fp4_gemv_amd", "csrc"),
                    "-I", os.path.join(ROOT, "include"), os.path.join(HERE, "cpu_wave", name + ".cpp"), "-o", out], check=True)
    return out


def run(program, folder, arrays):
    """Bytes of the program's output, and the kernels it launched, for the arrays' bytes in a row."""
    src, dst = os.path.join(str(folder), "in"), os.path.join(str(folder), "out")
    with open(src, "wb") as f:
        for a in arrays:
            f.write(np.ascontiguousarray(a).tobytes())
    done = subprocess.run([program, src, dst], capture_output=True, text=True, timeout=300)
    assert done.returncode == 0, f"status {done.returncode}: {STATUS.get(done.returncode, '')} {done.stderr}"
    return np.fromfile(dst, np.uint8), done.stdout
