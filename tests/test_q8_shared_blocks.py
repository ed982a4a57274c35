"""CPU checks of which segments of an 8-bit append share a block: the kernels' arithmetic (tests/block_checks_q8.cu)
and the oracle's statement of it."""
import os
import re
import shutil
import subprocess

import numpy as np
import pytest

import varlen_gqa_attention_gb300 as pkg
from oracle import step_oracle as S

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_runs_of_blocks_on_a_ring(tmp_path):
    nvcc = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(nvcc):
        pytest.skip("nvcc not found")
    exe = str(tmp_path / "block_checks_q8")
    subprocess.run([nvcc, "-std=c++17", "-O1", "--expt-relaxed-constexpr", "-gencode",
                    "arch=compute_103a,code=sm_103a", "-I", os.path.join(ROOT, "include"), "-o", exe,
                    os.path.join(ROOT, "tests", "block_checks_q8.cu")], check=True, capture_output=True)
    out = subprocess.run([exe], capture_output=True, text=True)
    assert out.returncode == 0 and "failures 0" in out.stdout, out.stdout


def test_the_oracle_names_the_segments_that_share_a_block():
    def shared(seq, T, rows, cols, window=0):
        live, _, _, _ = S.step_rows(seq, T, rows, cols, window)
        return S.q8_shared(seq, live, rows)

    # one block, other blocks, other columns, a ring that comes round, and a segment that overlaps
    assert shared([[0, 8, 0, 8], [8, 4, 0, 12]], 12, 32, 1) == [0, 1]
    assert shared([[0, 16, 0, 16], [16, 4, 0, 20]], 20, 32, 1) == []
    assert shared([[0, 8, 0, 8], [8, 4, 1, 12]], 12, 32, 2) == []
    assert shared([[0, 1, 0, 3], [1, 1, 0, 50]], 2, 48, 1, 1) == [0, 1]
    assert shared([[0, 9, 0, 8], [8, 4, 0, 12], [12, 1, 0, 14]], 13, 32, 1) == []
    assert shared([[0, 3, 0, 0], [3, 1, 0, 1]], 4, 32, 1) == []


def test_the_status_bit_is_the_headers():
    text = open(os.path.join(ROOT, "include", "sdpa_varlen.h")).read()
    assert re.search(r"#define SDPA_SEG_SHARED_BLOCK 128\b", text)
    assert pkg.SEG_SHARED_BLOCK == S.SHARED_BLOCK == 128 and "SEG_SHARED_BLOCK" in pkg.__all__
    others = [pkg.SEG_BAD_QRANGE, pkg.SEG_BAD_COL, pkg.SEG_BAD_KV, pkg.SEG_SPAN, pkg.SEG_OVERLAP, pkg.DEV_TIMEOUT,
              pkg.ROPE_BAD_POS]
    assert not np.bitwise_or.reduce(others) & pkg.SEG_SHARED_BLOCK
