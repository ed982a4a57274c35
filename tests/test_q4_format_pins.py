"""How far a stored group of the 4-bit store may be from its values, as the header states it."""
import numpy as np
import pytest
import torch

from oracle import step_oracle as S


def groups(top, seed):
    """64 groups of 32 bf16 values whose largest magnitude is `top` (a bf16 number)."""
    x = torch.rand(64, 32, generator=torch.Generator().manual_seed(seed)) * 2 - 1
    x = (x * top).to(torch.bfloat16)
    x[:, 7] = top
    return x


@pytest.mark.parametrize("top", [2.0 ** -30, 2.0 ** -22, 1.5 * 2.0 ** -22, 2.0 ** -20, 7 * 2.0 ** -21, 2.0 ** -18, 0.01, 1.0,
                                 129.0, 13440.0])
def test_error_of_a_group(top):
    x = groups(top, 1)
    codes, scales = S.q4_pack(x)
    assert codes.shape == (64, 16) and scales.shape == (64, 1)
    y, v = S.q4_unpack(codes, scales), S.f64(x)
    err, most = np.abs(y - v), np.abs(v).max()
    assert most == S.f64(torch.tensor(top).to(torch.bfloat16))
    if most >= 7 * 2.0 ** -21:
        assert err.max() <= 0.54 / 7 * most
    else:
        assert err.max() <= 2.0 ** -22
        assert (most > 2.0 ** -22) or not y.any()


def test_larger_magnitudes_saturate_and_nan_is_0():
    x = groups(13440.0, 2)
    x[:, 3], x[:, 4], x[:, 5], x[:, 6] = 3e38, float("-inf"), float("nan"), -20000.0
    y = S.q4_unpack(*S.q4_pack(x))
    assert (y[:, 3] == 13440).all() and (y[:, 4] == -13440).all() and not y[:, 5].any() and (y[:, 6] == -13440).all()
