"""The append into an 8-bit store leaves out segments that write to one block of a column, and says so: the others are
appended as a table without those appends them, byte for byte."""
import numpy as np
import pytest
import torch

import varlen_gqa_attention_gb300 as pkg
from oracle import step_oracle as S

from test_q8_append_gpu import random_store
from test_rope_gpu import assert_rotated

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    torch.cuda.set_device(0)
    return torch.device("cuda:0")


def check(dev, seq, T, rows, cols, *, D=64, Hq=4, Hkv=2, window=0, positions=None, P=2000, shared=None, seed=0):
    g = torch.Generator().manual_seed(seed)
    q, k, v = (torch.randn(T, h, D, generator=g).to(torch.bfloat16) for h in (Hq, Hkv, Hkv))
    seq = np.asarray(seq, dtype=np.int32).reshape(-1, 4)
    live, _, _, _ = S.step_rows(seq, T, rows, cols, window)
    out = S.q8_shared(seq, live, rows)
    if shared is not None:
        assert out == shared
    left = seq.copy()
    left[out] = 0  # without rows
    table = pkg.rope_table(P, D)
    pos = None if positions is None else np.asarray(positions, dtype=np.int32)
    qr, kb, wrote, st = S.rope_append(q, k, v, rows, cols, left, window, table, (D // 2,),
                                      None if pos is None else pos[None])
    live, _, _, _ = S.step_rows(left, T, rows, cols, window)
    store = random_store(rows, cols, Hkv, D, seed + 1, 10, 20)
    ref = []
    for codes, scales, x in ((store.k_codes, store.k_scales, kb), (store.v_codes, store.v_scales, v)):
        ref += S.q8_append(codes.numpy(), scales.numpy(), x, wrote, left, live, rows)
    stored = pkg.Q8Store(*(t.to(dev) for t in store))
    status = torch.zeros(1, dtype=torch.int32, device=dev)
    qd = pkg.sdpa_rope_append_q8(q.to(dev), k.to(dev), v.to(dev), stored, torch.from_numpy(seq).to(dev), table.to(dev),
                                 positions=None if pos is None else torch.from_numpy(pos).to(dev), window=window,
                                 status=status)
    assert int(status) == st | (pkg.SEG_SHARED_BLOCK if out else 0)
    for name, a, b in zip(pkg.Q8Store._fields, stored, ref):
        assert torch.equal(a.cpu(), torch.from_numpy(b)), name
    assert_rotated(qd, qr, q, D, False)
    gone = sorted(set(range(T)) - {t for t, _, _ in wrote})
    assert not bool(qd[gone].any())


@pytest.mark.parametrize("D", [64, 128, 256])
def test_two_parts_of_a_prompt(dev, D):
    # a prompt in two segments that meet inside a block, and in two that meet where one begins
    check(dev, [[0, 40, 1, 40], [40, 30, 1, 70], [70, 9, 0, 9]], 80, 96, 2, D=D, shared=[0, 1], seed=D)
    check(dev, [[0, 48, 1, 48], [48, 30, 1, 78], [78, 2, 0, 9]], 80, 96, 2, D=D, shared=[], seed=D)


def test_tokens_of_one_column(dev):
    # the same token twice, two neighbours, two in neighbouring blocks, and another column's
    check(dev, [[0, 1, 0, 5], [1, 1, 0, 5]], 2, 32, 2, shared=[0, 1])
    check(dev, [[0, 1, 0, 15], [1, 1, 0, 16], [2, 1, 1, 16]], 3, 32, 2, shared=[0, 1])
    check(dev, [[0, 1, 0, 16], [1, 1, 0, 17], [2, 1, 1, 16]], 3, 32, 2, shared=[])


def test_rings_on_which_two_segments_come_together(dev):
    check(dev, [[0, 1, 0, 3], [1, 1, 0, 50], [2, 20, 1, 100]], 22, 48, 2, window=1, shared=[0, 1])
    check(dev, [[0, 40, 0, 100], [40, 1, 0, 141]], 41, 48, 1, window=1, shared=[0, 1])
    check(dev, [[0, 17, 0, 81], [17, 14, 0, 127]], 31, 48, 1, window=1, shared=[0, 1])
    check(dev, [[0, 16, 0, 80], [16, 14, 0, 143]], 30, 48, 1, window=1, shared=[])
    check(dev, [[0, 5, 0, 20], [5, 7, 0, 90]], 12, 16, 1, window=1, shared=[0, 1])  # a ring of one block


def test_segments_that_write_nothing_share_nothing(dev):
    # overlapping ones, invalid ones, empty ones, and one before its sequence's beginning
    check(dev, [[0, 4, 0, 4], [3, 3, 0, 9], [6, 2, 0, 12]], 8, 32, 1, shared=[])
    check(dev, [[0, 4, 0, 4], [4, 3, 0, -1], [7, 0, 0, 9], [7, 2, 0, 40], [9, 2, 0, 0]], 11, 32, 1, shared=[])
    # places outside the rotation table count all the same
    live = [[0, 4, 0, 4], [4, 3, 0, 12]]
    pos = [5, 1, 2, 3, 2000, 2000, -1]
    check(dev, live, 7, 32, 1, positions=pos, shared=[0, 1])


@pytest.mark.parametrize("S_", [40, 300, 700])
def test_random_tables(dev, S_):
    rng = np.random.default_rng(S_)
    seq, t = [], 0
    for s in range(S_):
        n = int(rng.integers(0, 24))
        seq.append([t, n, int(rng.integers(0, S_ // 3)), int(rng.integers(0, 1000))])
        t += n + int(rng.integers(0, 2))
    seq[5][0] += 1  # meets the next one
    rng.shuffle(seq)
    check(dev, seq, t + 2, 80, S_ // 3, window=40, P=1001, seed=S_)
    out = [s for s in seq]
    live, _, _, _ = S.step_rows(out, t + 2, 80, S_ // 3, 40)
    assert 4 < len(S.q8_shared(out, live, 80)) < S_
