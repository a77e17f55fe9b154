"""The gated linear's grouped pair items, checked on the CPU: the schedule header is
compiled into a host-only program (tests/gated_schedule_check.cu) that checks that every
output column of every row block is covered once."""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "smoothquant_w8a8_int8_gb300", "csrc")


def test_gated_schedules_cover_every_tile_once(tmp_path):
    cands = (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc")
    nvcc = next((c for c in cands if c and os.path.exists(c)), None)
    if nvcc is None:
        pytest.skip("nvcc not found")
    exe = str(tmp_path / "gated_schedule_check")
    subprocess.run([nvcc, "-std=c++17", "-O1", "-I", CSRC, "-o", exe,
                    os.path.join(ROOT, "tests", "gated_schedule_check.cu")], check=True,
                   timeout=300)
    p = subprocess.run([exe], capture_output=True, text=True, timeout=300)
    assert p.returncode == 0, p.stdout[-3000:]
    assert "0 failures" in p.stdout
