"""Which kernels an automatically routed 8-bit attention call takes, and their results.

The scheduler's header opens the workspace (SchedHdr in csrc/common.cuh, 64-bit words): units of the split-K
and the prefill route are words 4 and 5, the packed rows of a split-K unit word 119.  A call that is not
scheduled writes its status only.
"""
import numpy as np
import pytest
import torch

import varlen_gqa_attention_gb300 as pkg

from test_q4_attention_gpu import queries
from test_q4_routes_gpu import units
from test_q8_attention_gpu import check, random_store

pytestmark = pytest.mark.gpu

FEW, TILE = 32, 128  # rows of a split-K unit: mma.sync kernel, tensor-memory kernel
UNTOUCHED = -1       # a workspace of 0xFF bytes


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    torch.cuda.set_device(0)
    return torch.device("cuda:0")


@pytest.fixture(autouse=True)
def automatic():
    pkg.set_route_policy(pkg.ROUTE_AUTO)
    yield


def run(q, store, seq, dev, **kw):
    """Output, status bits and header words of the call on a workspace of 0xFF bytes."""
    T, Hq, D = q.shape
    stored = pkg.Q8Store(*(t.to(dev) for t in store))
    seqd = torch.from_numpy(np.ascontiguousarray(seq, dtype=np.int32)).to(dev)
    ws = torch.full((pkg.q8_workspace_bytes(T, Hq, stored, len(seqd)),), 255, dtype=torch.uint8, device=dev)
    out = torch.full((T, Hq, D), float("nan"), dtype=torch.bfloat16, device=dev)
    status = torch.zeros(1, dtype=torch.int32, device=dev)
    pkg.sdpa_varlen_q8(q.to(dev), stored, seqd, out=out, workspace=ws, status=status, **kw)
    torch.cuda.synchronize()
    return out, int(status), ws[:960].cpu().view(torch.int64).tolist()


def table(lens):
    seq, t = [], 0
    for i, (n, kv) in enumerate(lens):
        seq.append([t, n, i, kv])
        t += n
    return seq, t


# lens: (tokens, keys) of each segment, chunks first; staged: how many of them take the staged route
@pytest.mark.parametrize("D,Hq,Hkv,rows,window,lens,staged,sk_rows", [
    (128, 32, 4, 10496, 0, [(100, 10496), (1, 10000), (1, 77), (1, 10496)], 1, FEW),
    (128, 32, 4, 8192, 0, [(130, 8192)] + [(16, 500 + 9 * i) for i in range(8)], 1, TILE),
    (64, 32, 4, 16384, 0, [(130, 16384)] + [(16, 500 + 9 * i) for i in range(8)], 1, TILE),
    # two chunks, each on a ring that has wrapped, within a window
    (128, 32, 4, 9008, 8063, [(130, 30000), (131, 9011), (1, 12345), (3, 40)], 2, FEW),
    # more segments than the small scheduler takes
    (128, 32, 4, 10496, 0, [(100, 10496)] + [(1, 300 + 11 * i) for i in range(40)], 1, FEW),
    # a chunk on its own (the small scheduler, whose units are then of 128 rows); D = 256
    (128, 16, 2, 4096, 0, [(530, 4000)], 1, TILE),
    (128, 16, 2, 4096, 0, [(700, 4000)], 1, TILE),
    (256, 16, 2, 2064, 0, [(130, 2064), (1, 2000), (2, 33)], 1, FEW),
])
def test_a_long_chunk_is_staged(dev, D, Hq, Hkv, rows, window, lens, staged, sk_rows):
    seq, t = table(lens)
    store, q = random_store(rows, len(lens), Hkv, D, D + t), queries(t, Hq, D, 7)
    out, st, hdr = run(q, store, seq, dev, causal=True, window=window)
    subset = sorted({r for s in seq for r in (s[0], s[0] + s[1] // 2, s[0] + s[1] - 1)})
    check(out, st, q, store, seq, True, window, rows_subset=subset)
    unit = 128 if D == 256 else 256
    assert hdr[5] == units(seq, range(staged), Hq // Hkv, Hkv, unit)
    assert hdr[4] == units(seq, range(staged, len(seq)), Hq // Hkv, Hkv, sk_rows) and hdr[119] == sk_rows


# (as long as a CTA for every token and KV head fits the SMs at once, 1400 keys need no schedule)
@pytest.mark.parametrize("D,n,sk_rows", [(128, 3, UNTOUCHED), (128, 16, TILE), (64, 16, UNTOUCHED), (64, 32, TILE),
                                         (256, 3, UNTOUCHED), (256, 16, FEW)])
def test_blocks_of_rows_take_the_kernel_that_costs_less(dev, D, n, sk_rows):
    # 12 segments of n tokens of 4 heads a KV head over up to 1500 keys
    seq, t = table([(n, 1500 - 31 * i) for i in range(12)])
    store, q = random_store(1504, 12, 2, D, n), queries(t, 8, D, n)
    out, st, hdr = run(q, store, seq, dev, causal=True, window=1400)
    check(out, st, q, store, seq, True, 1400)
    assert hdr[119] == sk_rows


@pytest.mark.parametrize("D,Hkv,S_,rows,direct", [
    (128, 2, 32, 8192, True), (128, 8, 32, 4096, True), (128, 8, 32, 8192, False), (128, 8, 1, 16384, True),
    (128, 8, 1, 32768, False), (64, 8, 32, 8192, True), (64, 8, 16, 16384, False), (256, 4, 16, 8192, True),
    (256, 4, 4, 16384, False),
])
def test_single_tokens_are_scheduled_only_over_long_ranges(dev, D, Hkv, S_, rows, direct):
    # short sequences in stores of these rows: the host sees the rows only
    cols = 3
    store = pkg.q8_store(rows, cols, Hkv, D, device=dev)
    small = random_store(320, cols, Hkv, D, 9)
    for big, s in zip(store, small):
        big[:, :, :s.shape[2]] = s.to(dev)
    seq = [[i, 1, i % cols, 300 - 7 * i] for i in range(S_)]
    q = queries(S_, 2 * Hkv, D, 10)
    ws = torch.full((pkg.q8_workspace_bytes(S_, 2 * Hkv, store, S_),), 255, dtype=torch.uint8, device=dev)
    out = pkg.sdpa_varlen_q8(q.to(dev), store, torch.tensor(seq, dtype=torch.int32, device=dev), causal=True, workspace=ws)
    check(out, 0, q, small, seq, True)
    assert (ws[:960].cpu().view(torch.int64)[119] == UNTOUCHED) == direct
