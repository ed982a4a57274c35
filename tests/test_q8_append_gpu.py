"""GPU parity of the rotated append into an 8-bit store and of its read-back.

Rotated keys are the 64-bit ones rounded to fp32 and bf16, scales are powers of two and a code is one exact
product rounded to an integer, so stores and read-backs are compared byte for byte.  Rotated queries are held to
the bound of the rotation itself (tests/test_rope_gpu.py)."""
import numpy as np
import pytest
import torch

import varlen_gqa_attention_gb300 as pkg
from oracle import step_oracle as S

from test_rope_append_gpu import bits
from test_rope_gpu import assert_rotated

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    torch.cuda.set_device(0)
    return torch.device("cuda:0")


def random_store(rows, cols, Hkv, D, seed, lo=0, hi=256):
    """Codes of every kind, scale bytes in [lo, hi)."""
    g = torch.Generator().manual_seed(seed)
    out = []
    for _ in range(2):
        out.append(torch.randint(0, 256, (cols, Hkv, rows, D), generator=g, dtype=torch.uint8))
        out.append(torch.randint(lo, hi, (cols, Hkv, rows // 16), generator=g, dtype=torch.uint8))
    return pkg.Q8Store(*out)


def assert_read_back(got, codes, scales, col, p, there, rows):
    r = np.maximum(p, 0) % rows
    ref = S.q8_unpack(codes, scales)[col, :, r]
    ref[~there] = 0.0
    assert torch.equal(bits(got), bits(S.to_bf16(ref)))


def check(dev, *, D, Hq, Hkv, T, rows, cols, seq, window=0, R=None, sections=None, axes=1, interleaved=False,
          explicit=False, modes=None, P=None, seed=0, spread=1.0, lo=10, hi=20):
    R = D if R is None else R
    g = torch.Generator().manual_seed(seed)
    # parts of one projection's rows
    qkv = (torch.randn(T, Hq + 2 * Hkv, D, generator=g) * torch.exp(spread * torch.randn(T, Hq + 2 * Hkv, 1, generator=g)))
    qkv = qkv.to(torch.bfloat16)
    q, k, v = qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:]
    seq = np.asarray(seq, dtype=np.int32).reshape(-1, 4)
    P = max(int(seq[:, 3].max(initial=1)) + 1, 2) if P is None else P
    table = pkg.rope_table(P, R)
    sections = (R // 2,) if sections is None else sections
    pos = torch.randint(0, P, (axes, T), generator=g, dtype=torch.int32) if explicit or axes > 1 else None
    qr, kb, wrote, st = S.rope_append(q, k, v, rows, cols, seq, window, table, sections,
                                      None if pos is None else pos.numpy(), interleaved, modes)
    live, p, col, st_rows = S.step_rows(seq, T, rows, cols, window, modes)
    qkvd = qkv.to(dev)
    kw = dict(positions=None if pos is None else pos.to(dev), sections=sections, interleaved=interleaved,
              window=window, seg_mode=None if modes is None else torch.tensor(modes, dtype=torch.int32, device=dev))
    seqd = torch.from_numpy(seq).to(dev)
    store = random_store(rows, cols, Hkv, D, seed + 1, lo, hi)
    stored = pkg.Q8Store(*(t.to(dev) for t in store))
    status = torch.zeros(1, dtype=torch.int32, device=dev)
    qd = pkg.sdpa_rope_append_q8(qkvd[:, :Hq], qkvd[:, Hq:Hq + Hkv], qkvd[:, Hq + Hkv:], stored, seqd, table.to(dev),
                                 status=status, **kw)
    assert int(status) == st
    assert_rotated(qd, qr, q, R, interleaved)
    gone = sorted(set(range(T)) - {t for t, _, _ in wrote})
    assert not bool(qd[gone].any())
    ref = []
    for codes, scales, x in ((store.k_codes, store.k_scales, kb), (store.v_codes, store.v_scales, v)):
        ref += S.q8_append(codes.numpy(), scales.numpy(), x, wrote, seq, live, rows)
    for name, a, b in zip(pkg.Q8Store._fields, stored, ref):
        assert torch.equal(a.cpu(), torch.from_numpy(b)), name

    # read back what the step's rows have become
    status.zero_()
    ko, vo = pkg.sdpa_q8_unpack(stored, seqd, T, window=window, seg_mode=kw["seg_mode"], status=status)
    assert int(status) == st_rows
    there = (live >= 0) & (p >= 0)
    assert_read_back(ko, ref[0], ref[1], col, p, there, rows)
    assert_read_back(vo, ref[2], ref[3], col, p, there, rows)


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("interleaved", [False, True])
def test_single_tokens_of_every_head_layout(dev, D, interleaved):
    for n, (Hq, Hkv) in enumerate([(1, 1), (8, 2), (15, 3), (32, 8), (40, 20)]):
        seq = [[i, 1, 6 - i, [1, 16, 7, 48, 33, 2, 40][i]] for i in range(7)]
        check(dev, D=D, Hq=Hq, Hkv=Hkv, T=7, rows=48, cols=7, seq=seq, interleaved=interleaved, seed=n, spread=2.0)


@pytest.mark.parametrize("D,R,sections,axes", [(64, 32, (3, 5, 8), 3), (128, 128, (16, 24, 24), 3), (128, 48, (24,), 1),
                                               (256, 256, (64, 0, 32, 32), 4), (128, 96, (47, 1), 2)])
def test_axes_and_partial_rotations(dev, D, R, sections, axes):
    for il in (False, True):
        check(dev, D=D, Hq=6, Hkv=2, T=70, rows=80, cols=3, seq=[[1, 40, 1, 61], [45, 20, 0, 20]], R=R,
              sections=sections, axes=axes, explicit=True, interleaved=il, seed=axes, P=777)


@pytest.mark.parametrize("n,kv", [(1, 17), (15, 15), (16, 16), (17, 33), (31, 47), (33, 40), (3, 48), (48, 48)])
def test_blocks_begun_ended_and_filled(dev, n, kv):
    check(dev, D=64, Hq=2, Hkv=2, T=n + 2, rows=64, cols=2, seq=[[1, n, 1, kv]], seed=n, spread=3.0, lo=0, hi=30)


@pytest.mark.parametrize("n,kv", [(1, 81), (5, 70), (5, 64), (32, 100), (47, 99), (48, 112), (48, 100), (48, 97), (48, 95), (40, 1000)])
def test_rings_of_three_blocks(dev, n, kv):
    # steps up to the whole ring, which come back to the block they began in
    check(dev, D=128, Hq=2, Hkv=1, T=n, rows=48, cols=2, seq=[[0, n, 0, kv]], window=1, seed=n + kv, spread=2.0)


def test_a_ring_of_one_block(dev):
    for n, kv in ((1, 1), (1, 40), (7, 20), (16, 16), (16, 21), (9, 31)):
        check(dev, D=64, Hq=1, Hkv=1, T=n, rows=16, cols=1, seq=[[0, n, 0, kv]], window=1, seed=kv, spread=2.0)


def test_long_chunk_on_a_ring_wraps(dev):
    # 700 rows on a 1024-row ring whose positions pass a multiple of 1024
    check(dev, D=128, Hq=4, Hkv=2, T=705, rows=1024, cols=3, seq=[[2, 700, 2, 5300]], window=300, seed=5)


def test_chunks_and_single_tokens_at_once(dev):
    seq, t = [], 0
    for i, (n, kv) in enumerate([(1, 200), (130, 300), (1, 16), (1, 17), (60, 60), (2, 400), (1, 33), (77, 303)]):
        seq.append([t, n, 7 - i, kv])
        t += n + i % 2
    check(dev, D=256, Hq=8, Hkv=4, T=t + 3, rows=400, cols=8, seq=seq, seed=3)


def test_tables_with_invalid_overlapping_and_early_segments(dev):
    seq = [[0, 3, 0, 10], [3, 2, 5, 10], [5, 2, 1, 10], [6, 2, 2, 10], [9, 4, 3, 2], [13, 0, 1, 5], [14, 2, 1, 60],
           [-1, 2, 1, 9], [20, 9, 0, 9], [17, 1, 1, -4], [16, 1, 2, 0]]
    check(dev, D=64, Hq=2, Hkv=1, T=25, rows=48, cols=4, seq=seq, seed=6)
    # a segment that overlaps another one far from its other rows is not live anywhere
    check(dev, D=64, Hq=2, Hkv=1, T=400, rows=400, cols=3, seq=[[0, 300, 0, 300], [299, 60, 1, 60], [360, 40, 2, 40]],
          seed=7)


def test_modes_per_segment_decide_validity(dev):
    seq = [[0, 4, 0, 100], [4, 4, 1, 100], [8, 4, 2, 30]]
    check(dev, D=128, Hq=4, Hkv=2, T=12, rows=32, cols=3, seq=seq, modes=[[1, 16], [1, 0], [0, 0]], seed=8)


def test_many_segments_and_no_segment(dev):
    seq = [[2 * i, 1 + i % 2, (i * 11) % 700, 1 + (i * 5) % 30] for i in range(700)]
    check(dev, D=64, Hq=2, Hkv=1, T=1400, rows=32, cols=700, seq=seq, seed=9)
    check(dev, D=64, Hq=2, Hkv=1, T=5, rows=32, cols=2, seq=np.zeros((0, 4)), seed=10)


def test_positions_outside_the_table_store_nothing(dev):
    # rows 1 and 3 of every four are outside; blocks with no row inside keep every byte
    for n, kv, window, rows in ((8, 12, 0, 32), (20, 40, 0, 48), (20, 100, 1, 48)):
        g = torch.Generator().manual_seed(n)
        q, k, v = (torch.randn(n, h, 64, generator=g).to(torch.bfloat16) for h in (2, 1, 1))
        seq = np.array([[0, n, 0, kv]], dtype=np.int32)
        table = pkg.rope_table(10, 64)
        pos = torch.tensor([10 if i % 2 or i >= n - 3 else i % 10 for i in range(n)], dtype=torch.int32)
        qr, kb, wrote, st = S.rope_append(q, k, v, rows, 1, seq, window, table, (32,), pos.numpy()[None])
        live, _, _, _ = S.step_rows(seq, n, rows, 1, window)
        store = random_store(rows, 1, 1, 64, n, 0, 40)
        stored = pkg.Q8Store(*(t.to(dev) for t in store))
        status = torch.zeros(1, dtype=torch.int32, device=dev)
        pkg.sdpa_rope_append_q8(q.to(dev), k.to(dev), v.to(dev), stored, torch.from_numpy(seq).to(dev), table.to(dev),
                                positions=pos.to(dev), window=window, status=status)
        assert int(status) == st == pkg.ROPE_BAD_POS
        ref = S.q8_append(store.k_codes.numpy(), store.k_scales.numpy(), kb, wrote, seq, live, rows)
        assert torch.equal(stored.k_codes.cpu(), torch.from_numpy(ref[0]))
        assert torch.equal(stored.k_scales.cpu(), torch.from_numpy(ref[1]))


def test_extreme_values_take_their_codes(dev):
    k = torch.zeros(80, 1, 64, dtype=torch.bfloat16)
    k[0, 0, :5] = torch.tensor([127.0, 0.5, 1.5, -0.5, 2.5], dtype=torch.bfloat16)
    k[16, 0, :3] = torch.tensor([3e38, float("inf"), float("-inf")], dtype=torch.bfloat16)
    k[32, 0, 0], k[33, 0, 1] = float("nan"), 7.0
    k[48, 0, :4] = torch.tensor([2.0 ** -21, -1.5 * 2.0 ** -20, 1e-38, -0.0], dtype=torch.bfloat16)
    k[64:, 0, :] = torch.linspace(-65536, 65536, 64).to(torch.bfloat16)
    store = pkg.q8_store(80, 1, 1, 64, device=dev)
    pkg.sdpa_rope_append_q8(torch.zeros(80, 1, 64, dtype=torch.bfloat16, device=dev), torch.zeros_like(k).to(dev),
                            k.to(dev), store, torch.tensor([[0, 80, 0, 80]], dtype=torch.int32, device=dev),
                            pkg.rope_table(80, 64, device=dev))
    for b in range(5):
        c, s = S.q8_code_block(S.f64(k[16 * b:16 * b + 16, 0]))
        assert int(store.v_scales[0, 0, b]) == s
        assert torch.equal(store.v_codes[0, 0, 16 * b:16 * b + 16].cpu(), torch.from_numpy(c))
    assert bool((store.k_codes == 128).all()) and not bool(store.k_scales.any())


def test_every_largest_magnitude_takes_the_oracles_scale(dev):
    # all 2^15 - 2^7 finite bf16 magnitudes, each the largest of a block of one row that holds its fractions
    mag = torch.arange(0x7F80, dtype=torch.int16).view(torch.bfloat16)
    x = (mag.float()[:, None] * torch.linspace(-1, 1, 64)).to(torch.bfloat16)
    x[:, 5] = mag
    n = mag.numel()
    store = pkg.q8_store(16, n, 1, 64, device=dev)
    flat = torch.tensor([1.0, 0.0], device=dev).expand(2, 32, 2).contiguous()
    i = torch.arange(n, dtype=torch.int32)
    seq = torch.stack([i, torch.ones_like(i), i, torch.ones_like(i)], dim=1).to(dev)
    xd = x.view(n, 1, 64).to(dev)
    half = n // 2  # (a table's segments are looked through by every CTA)
    for a in range(0, n, half):
        part = seq[:half].clone()
        part[:, 2] += a
        pkg.sdpa_rope_append_q8(xd[a:a + half], torch.zeros_like(xd[:half]), xd[a:a + half], store, part, flat)
    ref = [S.q8_code_block(S.f64(x[t:t + 1])) for t in range(n)]
    assert torch.equal(store.v_scales[:, 0, 0].cpu(), torch.tensor([s for _, s in ref], dtype=torch.uint8))
    assert torch.equal(store.v_codes[:, 0, 0].cpu(), torch.from_numpy(np.concatenate([c for c, _ in ref])))


def test_token_by_token_as_the_oracle_has_it(dev):
    # one captured step, replayed for every position of a ring's three laps
    D, Hkv, rows = 128, 2, 32
    g = torch.Generator().manual_seed(11)
    store = random_store(rows, 2, Hkv, D, 12)
    stored = pkg.Q8Store(*(t.to(dev) for t in store))
    kc, ks, vc, vs = (t.numpy() for t in store)
    table = pkg.rope_table(128, D)
    tabled, seqd = table.to(dev), torch.zeros(2, 4, dtype=torch.int32, device=dev)
    q, k, v = (torch.zeros(2, h, D, dtype=torch.bfloat16, device=dev) for h in (4, Hkv, Hkv))
    out = torch.empty_like(q)
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        pkg.sdpa_rope_append_q8(q, k, v, stored, seqd, tabled, window=8, q_out=out)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        pkg.sdpa_rope_append_q8(q, k, v, stored, seqd, tabled, window=8, q_out=out)
    for p in range(0, 96):
        seq = np.array([[0, 1, 1, p + 1], [1, 1, 0, max(1, p - 40)]], dtype=np.int32)
        scale = 2.0 ** (p % 7 - 3)
        new = [(scale * torch.randn(2, Hkv, D, generator=g)).to(torch.bfloat16) for _ in range(2)]
        k.copy_(new[0]), v.copy_(new[1]), seqd.copy_(torch.from_numpy(seq))
        graph.replay()
        _, kb, wrote, _ = S.rope_append(q.cpu(), new[0], new[1], rows, 2, seq, 8, table, (D // 2,))
        live, _, _, _ = S.step_rows(seq, 2, rows, 2, 8)
        kc, ks = S.q8_append(kc, ks, kb, wrote, seq, live, rows)
        vc, vs = S.q8_append(vc, vs, new[1], wrote, seq, live, rows)
    for name, a, b in zip(pkg.Q8Store._fields, stored, (kc, ks, vc, vs)):
        assert torch.equal(a.cpu(), torch.from_numpy(b)), name


def test_queries_in_place_and_other_streams(dev):
    g = torch.Generator().manual_seed(3)
    q, k, v = (torch.randn(6, h, 128, generator=g).to(torch.bfloat16) for h in (4, 2, 2))
    seq = np.array([[0, 5, 1, 30]], dtype=np.int32)
    table = pkg.rope_table(32, 128)
    qr, kb, wrote, _ = S.rope_append(q, k, v, 32, 2, seq, 0, table, (64,))
    qd, kd, vd, tabled, seqd = (t.to(dev) for t in (q, k, v, table, torch.from_numpy(seq)))
    store = pkg.q8_store(32, 2, 2, 128, device=dev)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    assert pkg.sdpa_rope_append_q8(qd, kd, vd, store, seqd, tabled, q_out=qd, stream=side) is qd
    ko, vo = pkg.sdpa_q8_unpack(store, seqd, 6, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert_rotated(qd, qr, q, 128, False)
    assert not bool(qd[5].any()) and not bool(ko[5].any())
    live, p, col, _ = S.step_rows(seq, 6, 32, 2, 0)
    empty = pkg.q8_store(32, 2, 2, 128)
    c, s = S.q8_append(empty.v_codes.numpy(), empty.v_scales.numpy(), v, wrote, seq, live, 32)
    assert_read_back(vo, c, s, col, p, live >= 0, 32)


def test_strided_rows_and_outputs(dev):
    # rows shared by every head (stride 0), rows far apart, and read-backs into part of a larger tensor
    D, Hkv, T = 64, 3, 21
    g = torch.Generator().manual_seed(4)
    base = torch.randn(T, 4, D, generator=g).to(torch.bfloat16)
    k, v, q = base[:, 1:2].expand(T, Hkv, D), base[:, 2:3].expand(T, Hkv, D), base[:, :1].expand(T, 6, D)
    seq = np.array([[0, 20, 0, 25]], dtype=np.int32)
    table = pkg.rope_table(32, D)
    _, kb, wrote, _ = S.rope_append(q, k, v, 32, 1, seq, 0, table, (32,))
    live, p, col, _ = S.step_rows(seq, T, 32, 1, 0)
    bd, seqd = base.to(dev), torch.from_numpy(seq).to(dev)
    store = pkg.q8_store(32, 1, Hkv, D, device=dev)
    out = torch.full((T, 9, 2 * D), 5.0, dtype=torch.bfloat16, device=dev)
    pkg.sdpa_rope_append_q8(bd[:, :1].expand(T, 6, D), bd[:, 1:2].expand(T, Hkv, D), bd[:, 2:3].expand(T, Hkv, D), store,
                            seqd, table.to(dev))
    back = torch.full((T, 2 * Hkv + 1, 2 * D), 5.0, dtype=torch.bfloat16, device=dev)
    ko, vo = pkg.sdpa_q8_unpack(store, seqd, T, k_out=back[:, :Hkv, :D], v_out=back[:, Hkv:2 * Hkv, D:])
    empty = pkg.q8_store(32, 1, Hkv, D)
    for got, x in ((ko, kb), (vo, v)):
        c, s = S.q8_append(empty.k_codes.numpy(), empty.k_scales.numpy(), x, wrote, seq, live, 32)
        assert_read_back(got, c, s, col, p, live >= 0, 32)
    assert bool((back[:, 2 * Hkv] == 5).all()) and bool((back[:, :Hkv, D:] == 5).all()) and \
        bool((back[:, Hkv:2 * Hkv, :D] == 5).all()) and bool((out == 5).all())
