"""What a launch that fails on the host leaves behind (kv_launch_check.cu)."""
from __future__ import annotations

import os
import subprocess

from entropy_coding_gb300 import build

FAKE_RUNTIME = """
static int last = 0;
int cudaLaunchKernelExC(const void *config, const void *kernel, void **arguments) { return last = 9; }
int cudaGetLastError(void) { int e = last; last = 0; return e; }
void **__cudaRegisterFatBinary(void *binary) { return 0; }
void __cudaRegisterFatBinaryEnd(void **handle) {}
void __cudaUnregisterFatBinary(void **handle) {}
"""


def test_a_failed_launch_leaves_no_error_behind(tmp_path):
    exe, fake = str(tmp_path / "check"), tmp_path / "fake.c"
    fake.write_text(FAKE_RUNTIME)
    src = os.path.join(os.path.dirname(os.path.abspath(__file__)), "kv_launch_check.cu")
    cmd = [build.nvcc(), *build.NVCC_FLAGS, "-cudart", "none", "-I", build.INCLUDE, "-I", build.CSRC, src, str(fake), "-o", exe]
    r = subprocess.run(cmd, capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    r = subprocess.run([exe], capture_output=True, text=True, timeout=60)
    assert r.returncode == 0, r.stdout + r.stderr
