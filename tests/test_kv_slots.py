"""The kernels' index arithmetic over ragged batches, compiled for the host (tests/kv_slots_check.cpp)."""
from __future__ import annotations

import os
import subprocess

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_slots_stay_in_range_whatever_the_counts_hold(tmp_path):
    exe = str(tmp_path / "kv_slots_check")
    subprocess.run(["g++", "-std=c++17", "-O2", "-I", os.path.join(ROOT, "entropy_coding_gb300", "csrc", "kv"),
                    os.path.join(ROOT, "tests", "kv_slots_check.cpp"), "-o", exe], check=True)
    r = subprocess.run([exe], capture_output=True, text=True)
    assert r.returncode == 0 and r.stdout == "ok\n", r.stdout
