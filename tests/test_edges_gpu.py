"""Calls at the ends of what the arguments allow, on every route, over the bf16 and the 4-bit store."""
import math

import numpy as np
import pytest
import torch

import varlen_gqa_attention_gb300 as pkg
from oracle import step_oracle as S

from test_q4_attention_gpu import check, queries, random_store, run_q4
from test_rope_gpu import assert_rotated

pytestmark = pytest.mark.gpu
LAST = 2 ** 31 - 1


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    torch.cuda.set_device(0)
    return torch.device("cuda:0")


@pytest.fixture(params=["auto", "splitk", "prefill"])
def route(request):
    pkg.set_route_policy({"auto": pkg.ROUTE_AUTO, "splitk": pkg.ROUTE_SPLITK, "prefill": pkg.ROUTE_PREFILL}[request.param])
    yield request.param
    pkg.set_route_policy(pkg.ROUTE_AUTO)


def both(dev, q, store, seq, causal, window, modes=None, rows_subset=None):
    """The 4-bit call and, over the same values, the bf16 one."""
    kw = dict(causal=causal, window=window)
    got, st = run_q4(q, store, seq, dev, seg_mode=modes, **kw)
    check(got, st, q, store, seq, causal, window, modes, rows_subset=rows_subset)
    k, v = (S.to_bf16(S.column_store(c.numpy(), b.numpy()).numpy()).to(dev)
            for c, b in ((store.k_codes, store.k_scales), (store.v_codes, store.v_scales)))
    seqd, status = torch.tensor(seq, dtype=torch.int32, device=dev), torch.zeros(1, dtype=torch.int32, device=dev)
    if modes is None:
        bf = pkg.sdpa_varlen(q.to(dev), k, v, seqd, status=status, **kw)
    else:
        bf = pkg.sdpa_varlen_modes(q.to(dev), k, v, seqd, torch.tensor(modes, dtype=torch.int32, device=dev), status=status)
    check(bf, int(status), q, store, seq, causal, window, modes, p_step=2.0 ** -8, rows_subset=rows_subset)


@pytest.mark.parametrize("D", [64, 128, 256])
def test_the_widest_window_hides_no_key(dev, route, D):
    # a window of 2^31 - 1 and rows before their sequence's beginning
    seq = [[0, 20, 0, 10], [20, 3, 1, 1], [23, 1, 2, 30]]
    store, q = random_store(32, 3, 2, D, D), queries(25, 8, D, 1)
    for causal in (False, True):
        both(dev, q, store, seq, causal, LAST)
        both(dev, q, store, seq, causal, LAST - 1)
    both(dev, q, store, seq, True, 0, [[0, LAST], [1, LAST], [0, LAST - 5]])


@pytest.mark.parametrize("D", [64, 128, 256])
def test_the_last_positions_on_a_ring(dev, route, D):
    seq = [[0, 1, 0, LAST], [1, 7, 1, LAST - 3], [8, 90, 2, LAST], [98, 2, 3, LAST - 127]]
    store, q = random_store(256, 4, 1, D, D), queries(101, 8, D, 2)
    for causal in (True, False):
        both(dev, q, store, seq, causal, 150)


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("lens", [[(1, 700)], [(1, 700), (1, 3), (5, 99)], [(40, 300), (1, 20)]])
def test_128_query_heads_for_one(dev, route, D, lens):
    seq, t = [], 0
    for i, (n, kv) in enumerate(lens):
        seq.append([t, n, i, kv])
        t += n
    both(dev, queries(t, 128, D, 3), random_store(704, len(lens), 1, D, D), seq, True, 0)


@pytest.mark.parametrize("D", [64, 128, 256])
def test_one_query_head_for_all_and_rows_shared(dev, route, D):
    # strides of 0: every head, then every row, the same
    seq, store = [[0, 1, 1, 300], [1, 150, 0, 200]], random_store(304, 2, 2, D, D)
    q = queries(151, 8, D, 4)
    for shared in (q[:, :1].expand(151, 8, D), q[:1].expand(151, 8, D)):
        stored = pkg.Q4Store(*(t.to(dev) for t in store))
        status = torch.zeros(1, dtype=torch.int32, device=dev)
        qd = shared[:, :1].contiguous().to(dev).expand(151, 8, D) if shared.stride(1) == 0 else \
            shared[:1].contiguous().to(dev).expand(151, 8, D)
        got = pkg.sdpa_varlen_q4(qd, stored, torch.tensor(seq, dtype=torch.int32, device=dev), causal=True, status=status)
        check(got, int(status), shared.contiguous(), store, seq, True)


@pytest.mark.parametrize("D", [64, 128, 256])
def test_parts_of_one_projections_rows(dev, route, D):
    # q, k and v rows beside each other in one tensor, the rotated queries over the queries, and the attention's
    # output over rows with space between them
    T, Hq, Hkv, rows = 33, 6, 2, 64
    seq = [[0, 20, 1, 50], [21, 12, 0, 12]]
    qkv = queries(T, Hq + 2 * Hkv + 1, D, 5)
    table = pkg.rope_table(64, D)
    q, k, v = qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:Hq + 2 * Hkv]
    qr, kb, wrote, st = S.rope_append(q, k, v, rows, 2, np.array(seq), 0, table, (D // 2,))
    ref_q = qkv.clone()
    store = random_store(rows, 2, Hkv, D, 6)
    stored = pkg.Q4Store(*(t.to(dev) for t in store))
    x = qkv.to(dev)
    seqd = torch.tensor(seq, dtype=torch.int32, device=dev)
    status = torch.zeros(1, dtype=torch.int32, device=dev)
    out = pkg.sdpa_rope_append_q4(x[:, :Hq], x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:Hq + 2 * Hkv], stored, seqd, table.to(dev),
                                  q_out=x[:, :Hq], status=status)
    assert int(status) == st
    assert_rotated(out, qr, q, D, False)
    assert torch.equal(x[:, Hq:].cpu().view(torch.int16), ref_q[:, Hq:].view(torch.int16))
    (kc, ks), (vc, vs) = S.q4_pack(kb), S.q4_pack(v)
    for t, row, col in wrote:
        for dst, src in zip(store, (kc, ks, vc, vs)):
            dst[col, :, row] = torch.from_numpy(src[t])
    assert all(torch.equal(a.cpu(), b) for a, b in zip(stored, store))
    wide = torch.full((T, Hq + 1, D + 8), 7.0, dtype=torch.bfloat16, device=dev)
    got = pkg.sdpa_varlen_q4(out, stored, seqd, causal=True, out=wide[:, :Hq, :D], status=status)
    check(got, int(status), out.cpu(), store, seq, True)
    assert bool((wide[:, Hq] == 7).all()) and bool((wide[:, :, D:] == 7).all())


@pytest.mark.parametrize("T,Hkv", [(20000, 1), (5000, 8)])
def test_thousands_of_single_tokens(dev, T, Hkv):
    D, cols, rows = 64, 50, 64
    rng = np.random.default_rng(T)
    seq = np.stack([rng.permutation(T), np.ones(T), np.arange(T) % cols, rng.integers(0, rows + 1, T)], axis=1).astype(np.int32)
    seq[17, 2], seq[18, 3], seq[19, 1] = cols, -1, 0
    store, q = random_store(rows, cols, Hkv, D, T), queries(T, 2 * Hkv, D, 7)
    got, st = run_q4(q, store, seq, dev, causal=True)
    pick = sorted({int(seq[i, 0]) for i in (0, 17, 18, 19, 20, T - 1)} | set(range(0, T, T // 40)))
    # the oracle on the picked rows' own table
    sub = seq[np.isin(seq[:, 0], pick)]
    at = {t: i for i, t in enumerate(pick)}
    sub[:, 0] = [at[int(t)] for t in sub[:, 0]]
    assert st == pkg.SEG_BAD_COL | pkg.SEG_BAD_KV
    check(got[torch.tensor(pick, device=dev)], st, q[pick], store, sub, True)


def test_the_scale_of_a_caller(dev, route):
    store, q = random_store(304, 2, 2, 128, 8), queries(40, 8, 128, 8)
    seq = [[0, 30, 0, 300], [30, 1, 1, 17], [31, 9, 1, 9]]
    for scale in (1e-30, 0.5 / math.sqrt(128), 1.0):
        got, st = run_q4(q, store, seq, dev, causal=True, scale=scale)
        check(got, st, q, store, seq, True, scale=scale)


@pytest.mark.parametrize("window", [2 ** 31, 2 ** 32 + 5, 2 ** 63 - 1, -2 ** 32 + 5])
def test_windows_beyond_32_bits_are_refused(dev, window):
    # 2^32 + 5 would be cut to 5
    store = pkg.q4_store(64, 1, 2, 64, device=dev)
    q, k = queries(3, 4, 64, 9).to(dev), queries(3, 2, 64, 10).to(dev)
    seq, table = torch.tensor([[0, 3, 0, 40]], dtype=torch.int32, device=dev), pkg.rope_table(64, 64, device=dev)
    cols = [torch.zeros(64, 1, 2, 64, dtype=torch.bfloat16, device=dev) for _ in range(2)]
    for call in (lambda: pkg.sdpa_varlen(q, *cols, seq, causal=True, window=window),
                 lambda: pkg.sdpa_varlen_append(q, k, k, *cols, seq, causal=True, window=window),
                 lambda: pkg.sdpa_varlen_splitk_static(q, *cols, seq, causal=True, window=window),
                 lambda: pkg.sdpa_rope_append(q, k, k, *cols, seq, table, window=window),
                 lambda: pkg.sdpa_rope_append_q4(q, k, k, store, seq, table, window=window),
                 lambda: pkg.sdpa_q4_unpack(store, seq, 3, window=window),
                 lambda: pkg.sdpa_varlen_q4(q, store, seq, causal=True, window=window)):
        with pytest.raises(ValueError, match="beyond 32 bits"):
            call()
