"""Narrow tiles or split K for a gated block's linear of few rows: the rule against the
times that it was fitted to, on the CPU (tests/gated_plan_check.cu)."""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "smoothquant_w8a8_int8_gb300", "csrc")


def test_the_faster_way_is_taken(tmp_path):
    cands = (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc")
    nvcc = next((c for c in cands if c and os.path.exists(c)), None)
    if nvcc is None:
        pytest.skip("nvcc not found")
    exe = str(tmp_path / "gated_plan_check")
    subprocess.run([nvcc, "-std=c++17", "-O1", "-I", CSRC, "-o", exe,
                    os.path.join(ROOT, "tests", "gated_plan_check.cu")], check=True, timeout=300)
    p = subprocess.run([exe], capture_output=True, text=True, timeout=300)
    assert p.returncode == 0, p.stdout[-3000:]
    assert "0 failures" in p.stdout
