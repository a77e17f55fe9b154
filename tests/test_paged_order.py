"""The paged attention's line of work for the row tiles that its launches have, and
for a q_start that decreases (tests/paged_order_check.cu, compiled for the host)."""
import os
import subprocess

import pytest

from test_paged_line import CSRC, ROOT, _nvcc


def test_row_tiles_and_decreasing_offsets(tmp_path):
    nvcc = _nvcc()
    if nvcc is None:
        pytest.skip("nvcc not found")
    exe = str(tmp_path / "paged_order_check")
    subprocess.run([nvcc, "-std=c++17", "-O1", "-I", CSRC, "-o", exe,
                    os.path.join(ROOT, "tests", "paged_order_check.cu")], check=True, timeout=300)
    p = subprocess.run([exe], capture_output=True, text=True, timeout=300)
    assert p.returncode == 0, p.stdout[-3000:]
    assert " 0 failures" in p.stdout
