"""GPU parity of the rotated append (bf16 and 4-bit stores) and of the 4-bit read-back.

Rotated keys are the 64-bit ones rounded to fp32 and bf16, and a code is decided by comparisons that
fp32 makes exactly, so stores and read-backs are compared bit for bit.  Rotated queries are held to
the bound of the rotation itself (tests/test_rope_gpu.py)."""
import numpy as np
import pytest
import torch

import varlen_gqa_attention_gb300 as pkg
from oracle import sdpa_varlen_oracle as O
from oracle import step_oracle as S

from test_rope_gpu import assert_rotated

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    torch.cuda.set_device(0)
    return torch.device("cuda:0")


def bits(t):
    return t.detach().cpu().view(torch.int16)


def random_store(rows, cols, Hkv, D, seed):
    g = torch.Generator().manual_seed(seed)
    return pkg.Q4Store(*(torch.randint(0, 256, (cols, Hkv, rows, n), generator=g, dtype=torch.uint8)
                         for n in (D // 2, D // 32, D // 2, D // 32)))


def check(dev, *, D, Hq, Hkv, T, rows, cols, seq, window=0, R=None, sections=None, axes=1, interleaved=False,
          explicit=False, modes=None, P=None, seed=0, spread=1.0):
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
    qkvd = qkv.to(dev)
    args = (qkvd[:, :Hq], qkvd[:, Hq:Hq + Hkv], qkvd[:, Hq + Hkv:])
    kw = dict(positions=None if pos is None else pos.to(dev), sections=sections, interleaved=interleaved,
              window=window, seg_mode=None if modes is None else torch.tensor(modes, dtype=torch.int32, device=dev))
    seqd = torch.from_numpy(seq).to(dev)

    def assert_queries(got):
        assert_rotated(got, qr, q, R, interleaved)
        gone = sorted(set(range(T)) - {t for t, _, _ in wrote})
        assert not bool(got[gone].any())

    # the bf16 store
    ks = torch.randn(rows, cols, Hkv, D, generator=g).to(torch.bfloat16)
    vs = torch.randn(rows, cols, Hkv, D, generator=g).to(torch.bfloat16)
    kd, vd = ks.to(dev), vs.to(dev)
    status = torch.zeros(1, dtype=torch.int32, device=dev)
    qd = pkg.sdpa_rope_append(*args, kd, vd, seqd, table.to(dev), status=status, **kw)
    for t, row, col in wrote:
        ks[row, col], vs[row, col] = kb[t], v[t]
    assert int(status) == st
    assert_queries(qd)
    assert torch.equal(bits(kd), bits(ks)) and torch.equal(bits(vd), bits(vs))

    # the 4-bit store
    store = random_store(rows, cols, Hkv, D, seed + 1)
    stored = pkg.Q4Store(*(t.to(dev) for t in store))
    status.zero_()
    qd = pkg.sdpa_rope_append_q4(*args, stored, seqd, table.to(dev), status=status, **kw)
    (kc, kscale), (vc, vscale) = S.q4_pack(kb), S.q4_pack(v)
    for t, row, col in wrote:
        for dst, src in zip(store, (kc, kscale, vc, vscale)):
            dst[col, :, row] = torch.from_numpy(src[t])
    assert int(status) == st
    assert_queries(qd)
    for name, a, b in zip(pkg.Q4Store._fields, stored, store):
        assert torch.equal(a.cpu(), b), name

    # read back what the step's rows have become
    live, p, col, st_rows = S.step_rows(seq, T, rows, cols, window, modes)
    status.zero_()
    ko, vo = pkg.sdpa_q4_unpack(stored, seqd, T, window=window, seg_mode=kw["seg_mode"], status=status)
    assert int(status) == st_rows
    there = (live >= 0) & (p >= 0)
    for got, codes, scales in ((ko, store.k_codes, store.k_scales), (vo, store.v_codes, store.v_scales)):
        ref = S.q4_unpack(codes.numpy()[col, :, np.maximum(p, 0) % rows], scales.numpy()[col, :, np.maximum(p, 0) % rows])
        ref[~there] = 0.0
        assert torch.equal(bits(got), bits(S.to_bf16(ref)))


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("interleaved", [False, True])
def test_decode_rows_of_every_head_layout(dev, D, interleaved):
    for n, (Hq, Hkv) in enumerate([(1, 1), (8, 2), (15, 3), (32, 8)]):
        seq = [[i, 1, 6 - i, [1, 16, 7, 48, 33, 2, 40][i]] for i in range(7)]
        check(dev, D=D, Hq=Hq, Hkv=Hkv, T=7, rows=48, cols=7, seq=seq, interleaved=interleaved, seed=n, spread=2.0)


@pytest.mark.parametrize("D,R,sections,axes", [(64, 32, (3, 5, 8), 3), (128, 128, (16, 24, 24), 3), (128, 48, (24,), 1),
                                               (256, 256, (64, 0, 32, 32), 4), (128, 96, (47, 1), 2)])
def test_axes_and_partial_rotations(dev, D, R, sections, axes):
    for il in (False, True):
        check(dev, D=D, Hq=6, Hkv=2, T=70, rows=80, cols=3, seq=[[1, 40, 1, 61], [45, 20, 0, 20]], R=R,
              sections=sections, axes=axes, explicit=True, interleaved=il, seed=axes, P=777)


def test_long_chunk_on_a_ring_wraps(dev):
    # 700 rows on a 1024-row ring whose positions pass a multiple of 1024
    check(dev, D=128, Hq=4, Hkv=2, T=705, rows=1024, cols=3, seq=[[2, 700, 2, 5300]], window=300, seed=5)


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
    g = torch.Generator().manual_seed(1)
    q, k, v = (torch.randn(4, h, 64, generator=g).to(torch.bfloat16) for h in (2, 1, 1))
    seq = np.array([[0, 4, 0, 12]], dtype=np.int32)
    table = pkg.rope_table(10, 64)  # positions 8, 9, 10, 11: the last two are not in it
    qr, kb, wrote, st = S.rope_append(q, k, v, 16, 1, seq, 0, table, (32,))
    assert st == pkg.ROPE_BAD_POS and [w[0] for w in wrote] == [0, 1]
    ks = torch.zeros(16, 1, 1, 64, dtype=torch.bfloat16, device=dev)
    vs = torch.zeros_like(ks)
    status = torch.zeros(1, dtype=torch.int32, device=dev)
    qd = pkg.sdpa_rope_append(q.to(dev), k.to(dev), v.to(dev), ks, vs, torch.from_numpy(seq).to(dev), table.to(dev),
                              status=status)
    assert int(status) == st and not bool(qd[2:].any())
    assert_rotated(qd, qr, q, 64, False)
    assert torch.equal(bits(ks[8:10, 0]), bits(kb[:2])) and int(ks.count_nonzero()) == int(kb[:2].count_nonzero())
    assert torch.equal(bits(vs[8:10, 0]), bits(v[:2])) and int(vs.count_nonzero()) == int(v[:2].count_nonzero())


def test_extreme_values_take_their_codes(dev):
    k = torch.zeros(8, 1, 64, dtype=torch.bfloat16)
    k[0, 0, :5] = torch.tensor([7.0, 0.5, 1.5, -0.5, 2.5], dtype=torch.bfloat16)
    k[1] = 3e38
    k[2, 0, 0], k[2, 0, 1] = float("inf"), 2.0
    k[3, 0, 0], k[3, 0, 1] = float("nan"), 7.0
    k[4] = 1e-20
    k[5, 0, :] = torch.tensor([7 * (1 + 1 / 16)] * 32 + [7 * (1 + 3 / 16)] * 32, dtype=torch.bfloat16)
    k[6, 0, ::2], k[6, 0, 1::2] = -0.0, 1e-38
    k[7, 0, :] = torch.linspace(-30, 30, 64).to(torch.bfloat16)
    store = pkg.q4_store(16, 1, 1, 64, device=dev)
    pkg.sdpa_rope_append_q4(torch.zeros(8, 1, 64, dtype=torch.bfloat16, device=dev), torch.zeros_like(k).to(dev),
                            k.to(dev), store, torch.tensor([[0, 8, 0, 8]], dtype=torch.int32, device=dev),
                            pkg.rope_table(8, 64, device=dev))
    c, s = S.q4_pack(k)
    assert torch.equal(store.v_codes[0, :, :8].cpu(), torch.from_numpy(c).transpose(0, 1))
    assert torch.equal(store.v_scales[0, :, :8].cpu(), torch.from_numpy(s).transpose(0, 1))
    assert bool((store.v_codes[0, :, 8:] == 0x88).all()) and bool((store.k_codes[0, :, :8] == 0x88).all())


def test_queries_in_place(dev):
    g = torch.Generator().manual_seed(3)
    q, k, v = (torch.randn(6, h, 128, generator=g).to(torch.bfloat16) for h in (4, 2, 2))
    seq = np.array([[0, 5, 1, 30]], dtype=np.int32)
    table = pkg.rope_table(32, 128)
    qr, _, _, _ = S.rope_append(q, k, v, 32, 2, seq, 0, table, (64,))
    qd = q.to(dev)
    store = pkg.q4_store(32, 2, 2, 128, device=dev)
    assert pkg.sdpa_rope_append_q4(qd, k.to(dev), v.to(dev), store, torch.from_numpy(seq).to(dev), table.to(dev),
                                   q_out=qd) is qd
    assert_rotated(qd, qr, q, 128, False)
    assert not bool(qd[5].any())


def test_every_largest_magnitude_takes_the_oracles_scale(dev):
    # all 2^15 - 2^7 bf16 magnitudes, each the largest of a group whose other values are its fractions
    mag = torch.arange(0x7F80, dtype=torch.int16).view(torch.bfloat16)
    frac = torch.linspace(-1, 1, 32)
    x = (mag.float()[:, None] * frac).to(torch.bfloat16)
    x[:, 5] = mag
    T = mag.numel() // 2
    x = x.view(T, 1, 64)
    rows = -(-T // 16) * 16
    store = pkg.q4_store(rows, 1, 1, 64, device=dev)
    xd = x.to(dev)
    flat = torch.tensor([1.0, 0.0], device=dev).expand(T, 32, 2).contiguous()
    seq = torch.tensor([[0, T, 0, T]], dtype=torch.int32, device=dev)
    pkg.sdpa_rope_append_q4(xd, torch.zeros_like(xd), xd, store, seq, flat)
    c, s = S.q4_pack(x)
    assert torch.equal(store.v_scales[0, 0, :T].cpu(), torch.from_numpy(s[:, 0]))
    assert torch.equal(store.v_codes[0, 0, :T].cpu(), torch.from_numpy(c[:, 0]))
