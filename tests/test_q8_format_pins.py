"""The 8-bit store's oracle against the statements of the header: scales, errors, rows coded again (CPU)."""
import math

import numpy as np
import pytest
import torch

from oracle import step_oracle as S

LARGEST = 127 * 512.0


def block(top, seed, D=64):
    """A block of 16 rows of bf16 values whose largest magnitude is `top` (a bf16 number)."""
    x = torch.rand(16, D, generator=torch.Generator().manual_seed(seed)) * 2 - 1
    x = (x * top).to(torch.bfloat16)
    x[5, 7] = top
    return S.f64(x)


@pytest.mark.parametrize("top", [2.0 ** -40, 2.0 ** -21, 1.5 * 2.0 ** -21, 127 * 2.0 ** -20, 2.0 ** -13, 1.0, 1.984375, 1.9921875,
                                 127.0, 127.5, 128.0, 60000.0, 65024.0])
def test_error_of_a_block(top):
    x = block(top, 1)
    codes, byte = S.q8_code_block(x)
    y = S.q8_unpack(codes[None, None], np.array([[[byte]]]))[0, 0]
    most, step = np.abs(x).max(), S.Q8_SCALES[byte]
    assert np.abs(y - x).max() <= step / 2
    assert most <= 127 * step and (byte == 0 or most > 127 * step / 2)
    if most >= 127 * 2.0 ** -20:
        assert step < most / 63
    assert np.array_equal(S.f64(S.to_bf16(y)), y)  # exact in bf16


def test_magnitudes_beyond_the_largest_scale_and_nan():
    x = block(65024.0, 2)
    x[3, :4] = [3e38, -np.inf, np.nan, -70000.0]
    codes, byte = S.q8_code_block(x)
    y = S.q8_unpack(codes[None, None], np.array([[[byte]]]))[0, 0]
    assert y[3, :4].tolist() == [LARGEST, -LARGEST, 0.0, -LARGEST]


def test_bytes_beyond_the_last_scale_stand_for_it():
    codes = np.arange(256, dtype=np.uint8).reshape(1, 1, 16, 16)
    ref = S.q8_unpack(codes, np.array([[[29]]]))
    for b in (30, 100, 255):
        assert np.array_equal(S.q8_unpack(codes, np.array([[[b]]])), ref)
    assert np.isfinite(ref).all()


def append_one_by_one(x, rows, n, first=0):
    """Tokens written one a step to column 0; yields the values of the store after each."""
    D = x.shape[-1]
    codes, scales = np.full((1, 1, rows, D), 77, dtype=np.uint8), np.full((1, 1, rows // 16), 200, dtype=np.uint8)
    for p in range(first, n):
        codes, scales = S.q8_append(codes, scales, x[p:p + 1, None], [(0, p % rows, 0)], [[0, 1, 0, p + 1]], [0], rows)
        yield S.q8_unpack(codes, scales)[0, 0], scales[0, 0]


def test_token_by_token_the_error_stays_below_a_step():
    g = np.random.default_rng(3)
    x = S.f64(torch.from_numpy(g.standard_normal((16, 64)) * np.exp2(np.arange(16))[:, None]).to(torch.bfloat16))
    kept = np.clip(x, -LARGEST, LARGEST)  # (the last rows have larger ones, which are taken as that)
    most = 0.0
    for p, (y, scales) in enumerate(append_one_by_one(x, 16, 16)):
        step = S.Q8_SCALES[scales[0]]
        most = max(most, step)
        assert np.abs(y[:p + 1] - kept[:p + 1]).max() < most
        assert np.abs(y[p] - kept[p]).max() <= step / 2


def test_a_block_forgets_an_outlier_once_it_is_overwritten():
    x = np.ones((48, 64))
    x[4] = 1000.0
    steps = [S.Q8_SCALES[s[0]] for _, s in append_one_by_one(x, 16, 48)]
    # 1 takes 2**-6 (127 * 2**-7 is less), 1000 takes 8 (127 * 4 is less)
    assert steps[3] == 2.0 ** -6 and steps[4] == steps[19] == 8.0 and steps[20] == 2.0 ** -6


def test_rows_without_a_position_count_for_nothing_and_keep_their_bytes():
    g = np.random.default_rng(5)
    codes = g.integers(0, 256, (2, 1, 32, 64)).astype(np.uint8)
    scales = np.full((2, 1, 2), 29, dtype=np.uint8)
    x = np.full((3, 1, 64), 0.5)
    c, s = S.q8_append(codes, scales, x, [(t, t, 1) for t in range(3)], [[0, 3, 1, 3]], [0, 0, 0], 32)
    assert math.isclose(S.Q8_SCALES[s[1, 0, 0]] * 127, 0.5, rel_tol=1.0) and s[1, 0, 1] == 29
    assert np.array_equal(c[1, :, 3:], codes[1, :, 3:]) and np.array_equal(c[0], codes[0])
    # the same rows a lap later: the other rows of the block now hold positions of the lap before
    _, s = S.q8_append(codes, scales, x, [(t, t, 1) for t in range(3)], [[0, 3, 1, 35]], [0, 0, 0], 32)
    assert s[1, 0, 0] == 29
