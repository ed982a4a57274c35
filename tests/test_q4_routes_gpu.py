"""Which kernels an automatically routed 4-bit attention call takes, and their results.

The scheduler's header opens the workspace (SchedHdr in csrc/common.cuh, 64-bit words): units of the split-K
and the prefill route are words 4 and 5, the packed rows of a split-K unit word 119.  A call that is not
scheduled writes its status only.
"""
import numpy as np
import pytest
import torch

import varlen_gqa_attention_gb300 as pkg
from oracle import sdpa_varlen_oracle as O

from test_q4_attention_gpu import check, queries, random_store

pytestmark = pytest.mark.gpu

FEW, TILE = 32, 128  # rows of a split-K unit: mma.sync kernel, tensor-memory kernel


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    torch.cuda.set_device(0)
    return torch.device("cuda:0")


def run(q, store, seq, dev, **kw):
    """Output, status bits and header words of the call on a workspace of 0xFF bytes."""
    T, Hq, D = q.shape
    stored = pkg.Q4Store(*(t.to(dev) for t in store))
    seqd = torch.from_numpy(np.ascontiguousarray(seq, dtype=np.int32)).to(dev)
    ws = torch.full((pkg.q4_workspace_bytes(T, Hq, stored, len(seqd)),), 255, dtype=torch.uint8, device=dev)
    out = torch.full((T, Hq, D), float("nan"), dtype=torch.bfloat16, device=dev)
    status = torch.zeros(1, dtype=torch.int32, device=dev)
    pkg.sdpa_varlen_q4(q.to(dev), stored, seqd, out=out, workspace=ws, status=status, **kw)
    torch.cuda.synchronize()
    return out, int(status), ws[:960].cpu().view(torch.int64).tolist()


def units(seq, which, group, Hkv, rows):
    return sum(Hkv * -(-seq[i][1] * group // rows) for i in which)


# lens: (tokens, keys) of each segment, chunks first; staged: how many of them take the staged route
@pytest.mark.parametrize("D,Hq,Hkv,rows,window,lens,staged,sk_rows", [
    # 800 packed rows (512 to 1023) beside single tokens: the kernel for few rows takes the tokens
    (128, 32, 4, 10496, 0, [(100, 10496), (1, 10000), (1, 77), (1, 10496)], 1, FEW),
    (64, 32, 4, 20992, 0, [(100, 20992), (1, 20000), (1, 77), (1, 1)], 1, FEW),
    # 1040 packed rows beside blocks of 128, which the tensor-memory kernel takes
    (128, 32, 4, 8192, 0, [(130, 8192)] + [(16, 500 + 9 * i) for i in range(8)], 1, TILE),
    (64, 32, 4, 16384, 0, [(130, 16384)] + [(16, 500 + 9 * i) for i in range(8)], 1, TILE),
    # two chunks, each on a ring that has wrapped, within a window
    (128, 32, 4, 9008, 8063, [(130, 30000), (131, 9011), (1, 12345), (3, 40)], 2, FEW),
    # more segments than the small scheduler takes
    (128, 32, 4, 10496, 0, [(100, 10496)] + [(1, 300 + 11 * i) for i in range(40)], 1, FEW),
    # a chunk on its own; D = 256, where the tensor-memory kernel of few-row segments does not exist
    (128, 16, 2, 4096, 0, [(530, 4000)], 1, TILE),
    (256, 16, 2, 2064, 0, [(130, 2064), (1, 2000), (2, 33)], 1, FEW),
])
def test_a_long_chunk_is_staged(dev, D, Hq, Hkv, rows, window, lens, staged, sk_rows):
    group, cols = Hq // Hkv, 3
    seq, t = [], 0
    for i, (n, kv) in enumerate(lens):
        seq.append([t, n, i % cols, kv])
        t += n + (i == 1)  # one row of no segment
    store, q = random_store(rows, cols, Hkv, D, D + len(lens)), queries(t + 1, Hq, D, 80)
    got, st, words = run(q, store, seq, dev, causal=True, window=window)
    assert words[119] == sk_rows
    assert words[5] == units(seq, range(staged), group, Hkv, 128 if D == 256 else 256)
    assert words[4] == units(seq, range(staged, len(seq)), group, Hkv, sk_rows)
    n = lens[0][0]
    rows_subset = sorted({0, 1, 31, 32, 33, n // 2, n - 1, n, min(n + 1, t), t - 1, t} | {s[0] for s in seq[-3:]})
    check(got, st, q, store, seq, True, window, p_step=2.0 ** -8, rows_subset=rows_subset)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("S_", [24, 70])
@pytest.mark.parametrize("chunk,kv,long,sk_rows", [
    (120, 130, 1500, FEW),  # a chunk over few keys among tokens over many
    (120, 1500, 40, TILE),  # over many keys among tokens over few
])
def test_a_chunk_among_single_tokens_takes_the_kernel_that_costs_less(dev, D, S_, chunk, kv, long, sk_rows):
    seq, t = [], 0
    for i in range(S_):
        n = chunk if i == S_ // 2 else 1
        seq.append([t, n, i % 5, kv if n > 1 else long - i % 9])
        t += n
    store, q = random_store(1504, 5, 4, D, D + S_), queries(t + 1, 32, D, 81)
    got, st, words = run(q, store, seq, dev, causal=True)
    assert words[119] == sk_rows and words[5] == 0 and words[4] == units(seq, range(S_), 8, 4, sk_rows)
    c = S_ // 2
    check(got, st, q, store, seq, True, rows_subset=sorted({0, c - 1, c, c + 31, c + chunk - 1, c + chunk, t - 1, t}))


def test_single_tokens_are_not_scheduled(dev):
    store, q = random_store(512, 4, 2, 128, 5), queries(4, 8, 128, 82)
    seq = [[i, 1, 3 - i, 500 - i] for i in range(4)]
    got, st, words = run(q, store, seq, dev, causal=True)
    assert words[119] == -1 and words[9] == 0  # the bytes that were there, and the status
    check(got, st, q, store, seq, True)
