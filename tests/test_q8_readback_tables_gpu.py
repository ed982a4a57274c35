"""The read-back of an 8-bit store over tables of every length, on both sides of where the look-up of rows changes:
segments out of order, empty, invalid, overlapping and before their sequence's beginning, byte for byte."""
import numpy as np
import pytest
import torch

import varlen_gqa_attention_gb300 as pkg
from oracle import step_oracle as S

from test_q8_append_gpu import assert_read_back, random_store

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    torch.cuda.set_device(0)
    return torch.device("cuda:0")


def check(dev, seq, T, rows, cols, Hkv, D, window, modes, seed):
    live, p, col, st = S.step_rows(seq, T, rows, cols, window, modes)
    store = random_store(rows, cols, Hkv, D, seed)
    stored = pkg.Q8Store(*(t.to(dev) for t in store))
    status = torch.zeros(1, dtype=torch.int32, device=dev)
    out = [torch.full((T, Hkv, D), float("nan"), dtype=torch.bfloat16, device=dev) for _ in range(2)]
    ko, vo = pkg.sdpa_q8_unpack(stored, torch.tensor(seq, dtype=torch.int32, device=dev), T, window=window,
                                seg_mode=None if modes is None else torch.tensor(modes, dtype=torch.int32, device=dev),
                                k_out=out[0], v_out=out[1], status=status)
    assert int(status) == st
    there = (live >= 0) & (p >= 0)
    assert_read_back(ko, store.k_codes.numpy(), store.k_scales.numpy(), col, p, there, rows)
    assert_read_back(vo, store.v_codes.numpy(), store.v_scales.numpy(), col, p, there, rows)
    return st


@pytest.mark.parametrize("S_", [1, 2, 31, 32, 33, 34, 64, 256, 257, 600])
@pytest.mark.parametrize("D,Hkv", [(64, 3), (128, 2), (256, 1)])
def test_tables_of_every_length(dev, S_, D, Hkv):
    rng = np.random.default_rng(S_ + D)
    cols, rows = 9, 48
    for most, window in ((1, 0), (5, 20), (30, 9)):
        seq, t = [], 1
        for s in range(S_):
            n = int(rng.integers(0 if s else 1, most + 1))
            kv = int(rng.integers(0, rows + 1 if window == 0 else 400))
            seq.append([t, n, int(rng.integers(0, cols)), kv])
            t += n + int(rng.integers(0, 2))
        rng.shuffle(seq)
        check(dev, seq, t + 3, rows, cols, Hkv, D, window, None, S_)
        if S_ > 8:
            seq[3][2], seq[4][3], seq[5][0] = cols, -2, -1
            seq[6] = [1, t, 0, 9]  # over all the others
            assert check(dev, seq, t + 3, rows, cols, Hkv, D, window, None, S_) & pkg.SEG_OVERLAP
            seq[6][1] = 0
            seq[7][1] += 1  # may meet its neighbour
            modes = [[1, int(rng.choice([0, 9, 20]))] for _ in seq]
            check(dev, seq, t + 3, rows, cols, Hkv, D, 0, modes, S_)
