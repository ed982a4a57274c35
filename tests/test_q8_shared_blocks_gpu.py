"""The append into an 8-bit store where segments of one call write to one block of a column: it is coded once, with the rows
of all of them, byte for byte as the oracle has it."""
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


def check(dev, seq, T, rows, cols, *, D=64, Hq=4, Hkv=2, window=0, positions=None, P=2000, shared=None, seed=0, modes=None):
    g = torch.Generator().manual_seed(seed)
    q, k, v = (torch.randn(T, h, D, generator=g).to(torch.bfloat16) for h in (Hq, Hkv, Hkv))
    seq = np.asarray(seq, dtype=np.int32).reshape(-1, 4)
    live, _, _, _ = S.step_rows(seq, T, rows, cols, window, modes)
    both = [w for w in S.q8_blocks(seq, live, rows).values() if len(w) > 1]
    if shared is not None:
        assert sorted({s for w in both for s in w}) == shared
    table = pkg.rope_table(P, D)
    pos = None if positions is None else np.asarray(positions, dtype=np.int32)
    qr, kb, wrote, st = S.rope_append(q, k, v, rows, cols, seq, window, table, (D // 2,),
                                      None if pos is None else pos[None], seg_mode=modes)
    store = random_store(rows, cols, Hkv, D, seed + 1, 10, 20)
    ref = []
    for codes, scales, x in ((store.k_codes, store.k_scales, kb), (store.v_codes, store.v_scales, v)):
        ref += S.q8_append(codes.numpy(), scales.numpy(), x, wrote, seq, live, rows)
    stored = pkg.Q8Store(*(t.to(dev) for t in store))
    status = torch.zeros(1, dtype=torch.int32, device=dev)
    qd = pkg.sdpa_rope_append_q8(q.to(dev), k.to(dev), v.to(dev), stored, torch.from_numpy(seq).to(dev), table.to(dev),
                                 positions=None if pos is None else torch.from_numpy(pos).to(dev), window=window,
                                 seg_mode=None if modes is None else torch.tensor(modes, dtype=torch.int32, device=dev),
                                 status=status)
    assert int(status) == st
    for name, a, b in zip(pkg.Q8Store._fields, stored, ref):
        assert torch.equal(a.cpu(), torch.from_numpy(b)), name
    assert_rotated(qd, qr, q, D, False)
    return len(both)


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


def test_more_parts_than_a_block_has_rows(dev):
    # a prompt token by token in one call, in order and out of it, and twice over
    for n, order in ((40, 1), (40, -1), (17, 1)):
        seq = [[t, 1, 0, t + 1] for t in range(n)][::order]
        assert check(dev, seq, n, 48, 1, seed=n) == n // 16 + (n % 16 > 1)
    seq = [[t, 1, 0, 1 + t % 20] for t in range(40)]
    check(dev, seq, 40, 48, 1, D=128, shared=list(range(40)))
    check(dev, seq[::-1], 40, 48, 1, D=256, shared=list(range(40)))


def test_segments_that_write_nothing_share_nothing(dev):
    # overlapping ones, invalid ones, empty ones, and one before its sequence's beginning
    check(dev, [[0, 4, 0, 4], [3, 3, 0, 9], [6, 2, 0, 12]], 8, 32, 1, shared=[])
    check(dev, [[0, 4, 0, 4], [4, 3, 0, -1], [7, 0, 0, 9], [7, 2, 0, 40], [9, 2, 0, 0]], 11, 32, 1, shared=[])


def test_places_outside_the_rotation_table(dev):
    # a row that is not written leaves its cell to the other segment's, which keeps it or writes it
    live = [[0, 4, 0, 4], [4, 3, 0, 12]]
    check(dev, live, 7, 32, 1, positions=[5, 1, 2, 3, 2000, 2000, -1], shared=[0, 1])
    check(dev, live, 7, 32, 1, positions=[5, 2000, 2, -1, 7, 2000, 0], shared=[0, 1])
    check(dev, [[0, 4, 0, 100], [4, 4, 0, 100]], 8, 48, 1, window=1, positions=[1, 2000, 2, 3, 2000, 2000, 5, -1], shared=[0, 1])
    check(dev, [[0, 1, 0, 4], [1, 1, 0, 9]], 2, 32, 1, positions=[-1, -1], shared=[0, 1])


def test_modes_decide_which_segments_share(dev):
    seq = [[0, 4, 0, 100], [4, 4, 0, 102], [8, 4, 0, 30]]
    check(dev, seq, 12, 32, 1, modes=[[1, 16], [1, 0], [0, 0]], shared=[])
    check(dev, seq, 12, 32, 1, modes=[[1, 16], [1, 9], [0, 0]], shared=[0, 1])


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
    assert check(dev, seq, t + 2, 80, S_ // 3, window=40, P=1001, seed=S_) > S_ // 4


def test_padding_tokens_of_one_scratch_column(dev):
    # a batch of 24 sequences padded to 200 tokens, whose scratch cells lie in one block; captured and replayed
    n, T, D = 24, 200, 128
    seq = np.array([[i, 1, i, 1 + 3 * i] if i < n else [i, 1, n, 1 + i % 2] for i in range(T)], dtype=np.int32)
    check(dev, seq, T, 96, n + 1, D=D, shared=list(range(n, T)))
    q, k, v = (torch.randn(T, h, D, device=dev).to(torch.bfloat16) for h in (4, 2, 2))
    table, seqd = pkg.rope_table(100, D, device=dev), torch.from_numpy(seq).to(dev)
    store = pkg.q8_store(96, n + 1, 2, D, device=dev)
    out = torch.empty_like(q)
    pkg.sdpa_rope_append_q8(q, k, v, store, seqd, table, q_out=out)
    want = [t.clone() for t in store]
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        pkg.sdpa_rope_append_q8(q, k, v, store, seqd, table, q_out=out)
    for _ in range(5):
        for t, x in zip(store, pkg.q8_store(96, n + 1, 2, D, device=dev)):
            t.copy_(x)
        graph.replay()
        for t, w in zip(store, want):
            assert torch.equal(t, w)
