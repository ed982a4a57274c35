"""CPU checks of 8-bit appends whose segments share blocks: the kernels' arithmetic (tests/block_checks_q8.cu) and the
oracle's statement of it."""
import os
import shutil
import subprocess

import numpy as np
import pytest

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


def test_the_oracle_names_the_blocks_that_segments_share():
    def shared(seq, T, rows, cols, window=0):
        live, _, _, _ = S.step_rows(seq, T, rows, cols, window)
        return {b: w for b, w in S.q8_blocks(seq, live, rows).items() if len(w) > 1}

    # one block, other blocks, other columns, a ring that comes round, and a segment that overlaps
    assert shared([[0, 8, 0, 8], [8, 4, 0, 12]], 12, 32, 1) == {(0, 0): [0, 1]}
    assert shared([[0, 16, 0, 16], [16, 4, 0, 20]], 20, 32, 1) == {}
    assert shared([[0, 8, 0, 8], [8, 4, 1, 12]], 12, 32, 2) == {}
    assert shared([[0, 1, 0, 3], [1, 1, 0, 50]], 2, 48, 1, 1) == {(0, 0): [0, 1]}
    assert shared([[0, 9, 0, 8], [8, 4, 0, 12], [12, 1, 0, 14]], 13, 32, 1) == {}
    assert shared([[0, 3, 0, 0], [3, 1, 0, 1]], 4, 32, 1) == {}


def test_the_oracle_codes_a_shared_block_once():
    """A prompt appended in parts by one call is what it is in one part, and a cell named twice takes the later segment's
    row whatever the order of the packed rows."""
    g = np.random.default_rng(1)
    x = g.normal(size=(40, 2, 64))
    codes, scales = np.full((1, 2, 48, 64), 128, dtype=np.uint8), np.zeros((1, 2, 3), dtype=np.uint8)

    def append(seq, x):
        live, p, col, _ = S.step_rows(seq, len(x), 48, 1, 0)
        return S.q8_append(codes, scales, x, [(t, int(p[t]), 0) for t in range(len(x))], seq, live, 48)

    whole = append([[0, 40, 0, 40]], x)
    for seq in ([[0, 7, 0, 7], [7, 33, 0, 40]], [[7, 33, 0, 40], [0, 7, 0, 7]]):
        parts = append(seq, x)
        assert all(np.array_equal(a, b) for a, b in zip(whole, parts))
    one = append([[0, 1, 0, 4]], x[1:2])
    twice = append([[1, 1, 0, 4], [0, 1, 0, 4]], np.stack([x[1], x[0]]))
    assert np.array_equal(one[0], twice[0])
