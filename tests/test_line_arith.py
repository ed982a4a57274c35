"""CPU checks of the work line and workspace of the 4-bit store's split-K kernels, through a small host
program built with nvcc (tests/line_checks.cu)."""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_lines_and_workspaces_of_both_kernels(tmp_path):
    nvcc = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(nvcc):
        pytest.skip("nvcc not found")
    exe = str(tmp_path / "line_checks")
    subprocess.run([nvcc, "-std=c++17", "-O1", "--expt-relaxed-constexpr", "-gencode",
                    "arch=compute_103a,code=sm_103a", "-I", os.path.join(ROOT, "include"), "-o", exe,
                    os.path.join(ROOT, "tests", "line_checks.cu")], check=True, capture_output=True)
    out = subprocess.run([exe], capture_output=True, text=True)
    fails = [ln for ln in out.stdout.splitlines() if ln.startswith("FAIL")]
    assert out.returncode == 0 and not fails, "\n".join(fails[:20])
    assert "failures 0" in out.stdout
