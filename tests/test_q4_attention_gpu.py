"""GPU parity of attention over the 4-bit column store against the 64-bit oracle.

The oracle attends over the values the codes stand for, laid out as the bf16 column store.  What the
kernels round: the probabilities (to fp16 on the split-K route, half a step 2^-11; to bf16 on the
tensor-memory route, 2^-8), a score in fp32 (each of its D products and sums at most 2^-23 of the sum
of magnitudes, taken twice for the softmax's two ends, and 2^-20 for exp2 and its argument's
rounding), sums in fp32, and the output (bf16, 2^-8).  fp16 probabilities are held so that a row's
largest is at least 2^7: one too small for a full step of them (2^-24) is off by 2^-25, which is 2^-32
of the row's sum, times its value."""
import math

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


@pytest.fixture(params=["auto", "splitk"], autouse=True)
def route(request):
    """Every test under the automatic routes (short key ranges without a schedule) and with a schedule."""
    pkg.set_route_policy(pkg.ROUTE_AUTO if request.param == "auto" else pkg.ROUTE_SPLITK)
    yield request.param
    pkg.set_route_policy(pkg.ROUTE_AUTO)


def random_store(rows, cols, Hkv, D, seed, lo=150, hi=170):
    """Codes of every kind (0 among them), scale bytes in [lo, hi)."""
    g = torch.Generator().manual_seed(seed)
    out = []
    for _ in range(2):
        out.append(torch.randint(0, 256, (cols, Hkv, rows, D // 2), generator=g, dtype=torch.uint8))
        out.append(torch.randint(lo, hi, (cols, Hkv, rows, D // 32), generator=g, dtype=torch.uint8))
    return pkg.Q4Store(*out)


def run_q4(q, store, seq, dev, **kw):
    """The call with a workspace of 0xFF bytes and an output full of NaN, and its status bits."""
    T, Hq, D = q.shape
    stored = pkg.Q4Store(*(t.to(dev) for t in store))
    seqd = torch.from_numpy(np.ascontiguousarray(seq, dtype=np.int32).reshape(-1, 4)).to(dev)
    ws = torch.full((pkg.q4_workspace_bytes(T, Hq, stored, len(seqd)),), 255, dtype=torch.uint8, device=dev)
    out = torch.full((T, Hq, D), float("nan"), dtype=torch.bfloat16, device=dev)
    status = torch.zeros(1, dtype=torch.int32, device=dev)
    if kw.get("seg_mode") is not None:
        kw["seg_mode"] = torch.tensor(kw["seg_mode"], dtype=torch.int32, device=dev)
    pkg.sdpa_varlen_q4(q.to(dev), stored, seqd, out=out, workspace=ws, status=status, **kw)
    torch.cuda.synchronize()
    return out, int(status)


def check(got, st, q, store, seq, causal, window=0, modes=None, scale=None, p_step=2.0 ** -11, rows_subset=None, tag=""):
    T, Hq, D = q.shape
    cols, Hkv, rows, _ = store.k_codes.shape
    scale = 1 / math.sqrt(D) if scale is None else scale
    k, v = (S.column_store(c.numpy(), b.numpy()) for c, b in ((store.k_codes, store.k_scales),
                                                             (store.v_codes, store.v_scales)))
    ref, seg_id, st_ref = O.sdpa_varlen(q, k, v, seq, causal, window, scale, rows_subset, modes)
    assert st == st_ref, f"{tag}: status {st}, not {st_ref}"
    mag, _, _ = O.sdpa_varlen(q, k, v.abs(), seq, causal, window, scale, rows_subset, modes)
    _, lo, hi, _ = O.visible_interval(seq, T, causal, window, rows, cols, modes)
    kmax = float(k.abs().sum(-1).max())
    qmax = np.abs(S.f64(q)).max(-1)  # sum |q_d k_d| <= max|q| sum|k|
    s_err = (2 * D * 2.0 ** -23 * scale * qmax * kmax + 2.0 ** -20)[..., None]
    small = 2.0 ** -32 * float(v.abs().max()) * np.maximum(hi - lo, 0)[:, None, None]
    bound = 2.0 ** -8 * np.abs(ref) + (p_step + 2 * s_err) * mag + small + 1e-30
    g = got.double().cpu().numpy()
    wanted = np.arange(T) if rows_subset is None else np.asarray(sorted(rows_subset))
    live = wanted[(seg_id[wanted] >= 0)]
    err = np.abs(g[live] - ref[live])
    assert np.isfinite(g[live]).all(), f"{tag}: not finite"
    assert (err <= bound[live]).all(), f"{tag}: {err.max()} at {np.argwhere(err > bound[live])[:3]}"
    zero = wanted[(seg_id[wanted] == O.UNCOVERED) | ((seg_id[wanted] >= 0) & (hi[wanted] <= lo[wanted]))]
    assert bool((got[torch.as_tensor(zero, device=got.device)].view(torch.int16) == 0).all()), tag


def queries(T, Hq, D, seed):
    return torch.randn(T, Hq, D, generator=torch.Generator().manual_seed(seed)).to(torch.bfloat16)


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("Hq,Hkv", [(1, 1), (8, 2), (15, 3), (16, 1), (40, 2)])
def test_single_tokens(dev, D, Hq, Hkv):
    kv = [1, 16, 17, 63, 64, 65, 128, 129, 300, 320, 2, 0]
    seq = [[i, 1, 11 - i, n] for i, n in enumerate(kv)]
    store, q = random_store(320, 12, Hkv, D, D + Hq), queries(12, Hq, D, 1)
    got, st = run_q4(q, store, seq, dev, causal=True)
    check(got, st, q, store, seq, True)


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("causal", [True, False])
def test_blocks_of_rows_and_gaps(dev, D, causal):
    seq = [[1, 3, 0, 3], [5, 17, 2, 100], [22, 40, 1, 47], [70, 5, 3, 2]]  # the last sees keys from its fourth row on
    store, q = random_store(112, 4, 2, D, D), queries(78, 6, D, 2)
    got, st = run_q4(q, store, seq, dev, causal=causal)
    check(got, st, q, store, seq, causal)


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("rows,window", [(16, 9), (48, 33), (128, 100), (144, 129), (272, 256)])
def test_windows_on_rings(dev, D, rows, window):
    rng = np.random.default_rng(rows + D)
    seq, t = [], 0
    for s in range(9):
        n = int(rng.integers(1, rows - window + 2))
        seq.append([t, n, s, int(rng.integers(1, 9 * rows))])
        t += n
    store, q = random_store(rows, 9, 2, D, rows), queries(t + 2, 8, D, 3)
    for causal in (True, False):
        got, st = run_q4(q, store, seq, dev, causal=causal, window=window)
        check(got, st, q, store, seq, causal, window)


@pytest.mark.parametrize("S_", [5, 60])
def test_random_tables_with_modes_invalid_and_overlapping_segments(dev, S_):
    rng = np.random.default_rng(S_)
    for trial, D in enumerate((64, 128, 256)):
        seq, t = [], 0
        for s in range(S_):
            t += int(rng.integers(0, 2))
            n = int(rng.integers(0, 9))
            seq.append([t, n, s % 7, int(rng.integers(0, 400))])
            t += n
        seq[1][1] += 2            # may meet the next one
        seq[2][2] = 7             # no such column
        seq[3][3] = -1
        modes = [[int(rng.integers(0, 2)), int(rng.choice([0, 1, 20, 90]))] for _ in seq]
        store, q = random_store(96, 7, 2, D, trial), queries(t + 4, 4, D, 4)
        got, st = run_q4(q, store, seq, dev, causal=True, seg_mode=modes)
        check(got, st, q, store, seq, True, 0, modes)


def test_long_contexts_split_over_many_ctas(dev):
    seq = [[0, 1, 0, 6000], [1, 2, 1, 6144], [3, 1, 2, 33]]
    for D in (64, 128, 256):
        store, q = random_store(6144, 3, 1, D, 5 + D), queries(4, 8, D, 5)
        got, st = run_q4(q, store, seq, dev, causal=True)
        check(got, st, q, store, seq, True)


def test_every_scale_byte(dev):
    # a store of one scale: the output scales with it, from the smallest to the largest byte
    q = queries(1, 2, 64, 6)
    for b in (0, 1, 30, 63, 64, 120, 168, 200, 255):
        store = random_store(48, 1, 1, 64, b, 168, 169)
        store.v_scales.fill_(b)
        got, st = run_q4(q, store, [[0, 1, 0, 41]], dev, causal=True)
        check(got, st, q, store, [[0, 1, 0, 41]], True, tag=f"V scale {b}")
        store = random_store(48, 1, 1, 64, b, 150, 160)
        store.k_scales.fill_(b)
        scale = 1 / float(S.scale_of(b)) / 64  # scores of order one
        got, st = run_q4(q, store, [[0, 1, 0, 41]], dev, causal=True, scale=scale)
        check(got, st, q, store, [[0, 1, 0, 41]], True, scale=scale, tag=f"K scale {b}")


def test_one_visible_key_returns_its_values_exactly(dev):
    for D in (64, 128, 256):
        store, q = random_store(64, 2, 2, D, D, 0, 256), queries(3, 4, D, 7)
        seq = [[0, 1, 0, 1], [1, 2, 1, 50]]
        got, _ = run_q4(q, store, seq, dev, causal=True, window=1)
        v = S.to_bf16(S.q4_unpack(store.v_codes.numpy(), store.v_scales.numpy()))
        want = torch.stack([v[0, :, 0], v[1, :, 48], v[1, :, 49]]).repeat_interleave(2, dim=1)
        assert torch.equal(got.cpu().view(torch.int16), want.view(torch.int16)), D


def test_keys_outside_the_visible_ones_do_not_matter(dev):
    rows, window = 160, 70
    seq = [[0, 2, 0, 1000], [2, 1, 2, 40]]
    store, q = random_store(rows, 4, 2, 128, 8), queries(3, 8, 128, 8)
    a, _ = run_q4(q, store, seq, dev, causal=True, window=window)
    seen = torch.zeros(4, rows, dtype=torch.bool)
    seen[0, torch.arange(1000 - 71, 1000) % rows] = True
    seen[2, :40] = True
    other = pkg.Q4Store(*(torch.where(seen[:, None, :, None], t, 255 - t) for t in store))
    b, _ = run_q4(q, other, seq, dev, causal=True, window=window)
    assert torch.equal(a.view(torch.int16), b.view(torch.int16))


def test_a_row_of_nan_or_infinity_stays_alone(dev):
    q = queries(6, 4, 128, 9)
    store = random_store(256, 1, 1, 128, 9)
    clean, _ = run_q4(q, store, [[0, 6, 0, 200]], dev, causal=True)
    q[2, 1, 5], q[4, 3, 100] = float("nan"), float("inf")
    got, _ = run_q4(q, store, [[0, 6, 0, 200]], dev, causal=True)
    assert bool(got[2, 1].isnan().any()) and bool(got[4, 3].isnan().any())
    got[2, 1], got[4, 3] = clean[2, 1], clean[4, 3]
    assert torch.equal(got.view(torch.int16), clean.view(torch.int16))


def test_strided_rows_no_rows_and_no_segments(dev):
    store = random_store(64, 2, 2, 64, 10)
    wide = queries(8, 12, 64, 10)
    q = wide[::2, 4:8]
    out = torch.full((4, 9, 64), 3.0, dtype=torch.bfloat16, device=dev)
    stored = pkg.Q4Store(*(t.to(dev) for t in store))
    seq = torch.tensor([[0, 4, 1, 60]], dtype=torch.int32, device=dev)
    pkg.sdpa_varlen_q4(wide.to(dev)[::2, 4:8], stored, seq, causal=True, out=out[:, ::2][:, :4])
    check(out[:, ::2][:, :4], 0, q, store, [[0, 4, 1, 60]], True)
    assert bool((out[:, 1::2] == 3).all()) and bool((out[:, 8] == 3).all())
    assert pkg.sdpa_varlen_q4(wide[:0].to(dev), stored, seq[:0], causal=True).shape == (0, 12, 64)
    got = pkg.sdpa_varlen_q4(wide.to(dev), stored, seq[:0], causal=True)
    assert not bool(got.any())


def test_a_column_beyond_two_gibibytes(dev):
    # the last column's codes begin past 2^31 bytes, its rows past 2^31 of them in dims
    rows, cols, Hkv, D = 1 << 18, 9, 8, 256
    store = pkg.q4_store(rows, cols, Hkv, D, device=dev)
    assert store.k_codes.numel() > 1 << 31
    kv, window, n = rows - 3, 90, 4
    small = random_store(128, 1, Hkv, D, 11)
    at = torch.arange(kv - window - n + 1, kv)
    for big, s in zip(store, small):
        big[cols - 1, :, at.to(dev)] = s[0, :, at % 128].to(dev)
    q = queries(n, 8, D, 11)
    seq = torch.tensor([[0, n, cols - 1, kv]], dtype=torch.int32, device=dev)
    got = pkg.sdpa_varlen_q4(q.to(dev), store, seq, causal=True, window=window)
    check(got, 0, q, small, [[0, n, 0, kv]], True, window)


def test_two_calls_at_once_on_two_streams(dev):
    store = random_store(512, 4, 2, 128, 12)
    stored = pkg.Q4Store(*(t.to(dev) for t in store))
    q = [queries(4, 8, 128, 20 + i) for i in range(2)]
    seq = [[i, 1, i, 500 - i] for i in range(4)]
    seqd = torch.tensor(seq, dtype=torch.int32, device=dev)
    qd = [x.to(dev) for x in q]
    streams = [torch.cuda.Stream(dev) for _ in range(2)]
    torch.cuda.synchronize()
    outs = [[pkg.sdpa_varlen_q4(qd[i], stored, seqd, causal=True, stream=streams[i]) for i in range(2)]
            for _ in range(20)]
    torch.cuda.synchronize()
    for pair in outs:
        for i in range(2):
            check(pair[i], 0, q[i], store, seq, True)


def test_a_decode_loop_in_one_captured_graph(dev):
    """Rotate and append a step's rows, then attend, captured once and replayed with new lengths."""
    Hq, Hkv, D, rows, cols, T = 8, 2, 128, 64, 4, 3
    table = pkg.rope_table(400, D)
    tab = table.to(dev)
    store = random_store(rows, cols, Hkv, D, 13)
    stored = pkg.Q4Store(*(t.to(dev) for t in store))
    q, k, v = (torch.zeros(T, h, D, dtype=torch.bfloat16, device=dev) for h in (Hq, Hkv, Hkv))
    seqd = torch.zeros(T, 4, dtype=torch.int32, device=dev)
    ws = torch.empty(pkg.q4_workspace_bytes(T, Hq, stored, T), dtype=torch.uint8, device=dev)
    qr, out = torch.empty_like(q), torch.empty_like(q)

    def step():
        pkg.sdpa_rope_append_q4(q, k, v, stored, seqd, tab, window=50, q_out=qr)
        pkg.sdpa_varlen_q4(qr, stored, seqd, causal=True, window=50, out=out, workspace=ws)

    keep = [t.clone() for t in stored]
    step()
    torch.cuda.synchronize()
    for t, old in zip(stored, keep):
        t.copy_(old)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    gen = torch.Generator().manual_seed(14)
    for n in range(6):
        new = [torch.randn(T, h, D, generator=gen).to(torch.bfloat16) for h in (Hq, Hkv, Hkv)]
        seq = np.array([[i, 1, (i + n) % cols, 1 + n + 60 * i] for i in range(T)], dtype=np.int32)
        for a, b in zip((q, k, v), new):
            a.copy_(b)
        seqd.copy_(torch.from_numpy(seq))
        g.replay()
        torch.cuda.synchronize()
        ref_q, kb, wrote, _ = S.rope_append(*new, rows, cols, seq, 50, table, (D // 2,))
        packed = S.q4_pack(kb) + S.q4_pack(new[2])
        for t, row, col in wrote:
            for dst, src in zip(store, packed):
                dst[col, :, row] = torch.from_numpy(src[t])
        for a, b in zip(stored, store):
            assert torch.equal(a.cpu(), b)
        assert_rotated(qr, ref_q, new[0], D, False)
        check(out, 0, qr.cpu(), store, seq, True, 50)


def test_the_bf16_store_agrees_with_the_4_bit_one_on_its_values(dev):
    # the values are exact in bf16: the bf16 entry over them and this one differ by rounding only
    store, q = random_store(512, 2, 2, 128, 15), queries(20, 8, 128, 15)
    seq = [[0, 1, 1, 512], [1, 19, 0, 300]]
    got, st = run_q4(q, store, seq, dev, causal=True)
    k, v = (S.to_bf16(S.column_store(c.numpy(), b.numpy()).numpy()).to(dev)
            for c, b in ((store.k_codes, store.k_scales), (store.v_codes, store.v_scales)))
    bf = pkg.sdpa_varlen(q.to(dev), k, v, torch.tensor(seq, dtype=torch.int32, device=dev), causal=True)
    check(got, st, q, store, seq, True)
    check(bf, st, q, store, seq, True, p_step=2.0 ** -8)


# ------------------------------------------- the tensor-memory route: columns staged in bf16 first

@pytest.fixture
def prefill_route(route):
    if route != "auto":
        pytest.skip("one policy at a time")
    pkg.set_route_policy(pkg.ROUTE_PREFILL)
    yield
    pkg.set_route_policy(pkg.ROUTE_AUTO)


@pytest.mark.parametrize("D", [64, 128, 256])
def test_staged_route_small_shapes(dev, prefill_route, D):
    seq = [[0, 1, 3, 100], [1, 70, 1, 300], [75, 130, 0, 131], [210, 5, 2, 2]]
    store, q = random_store(304, 4, 2, D, D), queries(218, 4, D, 30)
    for causal in (True, False):
        got, st = run_q4(q, store, seq, dev, causal=causal)
        check(got, st, q, store, seq, causal, p_step=2.0 ** -8)


@pytest.mark.parametrize("D", [64, 128, 256])
def test_staged_route_on_rings(dev, prefill_route, D):
    rows, window = 272, 150
    rng = np.random.default_rng(D)
    seq, t = [], 0
    for s in range(6):
        n = int(rng.integers(1, rows - window + 2))
        seq.append([t, n, s, int(rng.integers(1, 9 * rows))])
        t += n
    store, q = random_store(rows, 6, 1, D, rows + D), queries(t, 8, D, 31)
    got, st = run_q4(q, store, seq, dev, causal=True, window=window)
    check(got, st, q, store, seq, True, window, p_step=2.0 ** -8)
    modes = [[s % 2, [window, 40, 1][s % 3]] for s in range(6)]
    got, st = run_q4(q, store, seq, dev, causal=True, seg_mode=modes)
    check(got, st, q, store, seq, True, 0, modes, p_step=2.0 ** -8)


def test_staged_route_many_segments(dev, prefill_route):
    # more segments than the small scheduler takes, two of them on one column, some not live
    seq = [[3 * i, 3, i % 37, 20 + i] for i in range(45)]
    seq[4][2], seq[9][1] = 99, 5
    store, q = random_store(80, 40, 1, 64, 32), queries(136, 4, 64, 32)
    got, st = run_q4(q, store, seq, dev, causal=True)
    check(got, st, q, store, seq, True, p_step=2.0 ** -8)


@pytest.mark.parametrize("S_", [11, 40])
def test_segments_beyond_the_staged_columns_take_the_other_route(dev, prefill_route, S_):
    # 2^20 rows of 64 dims are 256 MiB of bf16 K and V a column: eight are staged
    rows = 1 << 20
    store = pkg.q4_store(rows, 12, 1, 64, device=dev)
    small = random_store(320, 12, 1, 64, 33)
    for big, s in zip(store, small):
        big[:, :, :320] = s.to(dev)
    q = queries(9 * S_, 8, 64, 33)
    seq = [[9 * i, 8 + (i % 2), (5 * i) % 12, 300 - 7 * (i % 40)] for i in range(S_)]
    seq[2][1] = 0
    seqd = torch.tensor(seq, dtype=torch.int32, device=dev)
    status = torch.zeros(1, dtype=torch.int32, device=dev)
    got = pkg.sdpa_varlen_q4(q.to(dev), store, seqd, causal=True, status=status)
    check(got, int(status), q, small, seq, True, p_step=2.0 ** -8)


def test_a_long_chunk_beside_single_tokens(dev):
    # automatic routing: the chunk goes through staged columns, the tokens do not
    store = random_store(4096, 4, 2, 128, 34)
    seq = [[0, 1, 3, 4096], [1, 700, 1, 4090], [701, 1, 0, 77], [705, 300, 2, 301]]
    q = queries(1006, 8, 128, 34)
    rows = [0, 1, 2, 128, 333, 700, 701, 702, 704, 705, 706, 900, 1004, 1005]
    got, st = run_q4(q, store, seq, dev, causal=True)
    check(got, st, q, store, seq, True, p_step=2.0 ** -8, rows_subset=rows)
    got, st = run_q4(q, store, seq, dev, causal=True, window=100)
    check(got, st, q, store, seq, True, 100, p_step=2.0 ** -8, rows_subset=rows)


# ----------------------------------------- both split-K kernels over their whole range of segments

@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("Hq,Hkv,lens", [
    (8, 2, [(32, 6000)]),                        # one unit of 128 rows, its keys cut over many CTAs
    (8, 1, [(17, 5003), (16, 4096), (1, 6143)]),  # 136, 128 and 8 packed rows: a block of 8 rows, a full one
    (128, 1, [(1, 4500), (2, 130), (3, 129)]),   # a token's heads fill a unit
    (8, 8, [(129, 3000), (128, 2999), (5, 5)]),  # no shared heads, rows that no block divides
    (24, 2, [(40, 2111), (11, 64), (10, 63)]),   # 12 rows a token: tokens end inside a unit
])
def test_tile_kernel_pieces(dev, D, Hq, Hkv, lens):
    seq, t = [], 1
    for i, (n, kv) in enumerate(lens):
        seq.append([t, n, i, kv])
        t += n + i
    rows = -(-max(kv for _, kv in lens) // 16) * 16
    store, q = random_store(rows, len(lens), Hkv, D, D + Hq), queries(t + 1, Hq, D, 40)
    subset = sorted({0, t} | {r for s in seq for r in (s[0], s[0] + 1, s[0] + s[1] // 2, s[0] + s[1] - 1, s[0] + s[1])
                              if r <= t})
    for causal, window in ((True, 0), (False, 0), (True, 700)):
        got, st = run_q4(q, store, seq, dev, causal=causal, window=window)
        check(got, st, q, store, seq, causal, window, rows_subset=subset, tag=f"{causal} {window}")


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("blocks", [[12, 9, 1, 1, 1, 1, 1, 1], [70, 3, 2, 1, 1, 1, 1, 1], [40, 40]])
def test_few_rows_on_average_with_longer_blocks_among_them(dev, D, blocks):
    # 8 x 2 packed rows a token: blocks of 17 to 32 rows and several units of 32 in the split-K kernel
    seq, t = [], 0
    for i, n in enumerate(blocks):
        seq.append([t, n, i, 900 + 37 * i])
        t += n
    pad = len(blocks)
    seq += [[t, 0, 0, 1]] * max(0, t * 2 - 16 * pad)  # (empty segments count towards the average)
    store, q = random_store(1200, 8, 2, D, D), queries(t, 4, D, 41)
    got, st = run_q4(q, store, seq, dev, causal=True)
    check(got, st, q, store, seq, True)


def test_many_segments_of_several_rows(dev):
    # more segments than the small scheduler takes, on the tensor-memory kernel: several units a CTA
    seq = [[6 * i, 5 + i % 2, (3 * i) % 44, 130 + 9 * (i % 50)] for i in range(88)]
    store, q = random_store(608, 44, 4, 128, 42), queries(6 * 88, 16, 128, 42)
    assert 6 * 88 * 4 > 16 * 88
    for modes in (None, [[i % 2, [0, 1, 64, 200][i % 4]] for i in range(88)]):
        got, st = run_q4(q, store, seq, dev, causal=True, seg_mode=modes)
        check(got, st, q, store, seq, True, 0, modes)


def test_a_scale_of_zero_is_the_mean_of_the_visible_values(dev):
    store = random_store(512, 2, 2, 128, 43)
    for seq in ([[0, 1, 0, 500], [1, 1, 1, 3]], [[0, 30, 0, 500], [30, 30, 1, 31]]):
        T = seq[-1][0] + seq[-1][1]
        q = queries(T, 8, 128, 43)
        got, st = run_q4(q, store, seq, dev, causal=True, scale=0.0)
        check(got, st, q, store, seq, True, scale=0.0)


@pytest.mark.parametrize("D", [64, 128])
def test_tile_kernel_keeps_a_row_of_nan_or_infinity_alone(dev, D):
    seq = [[0, 24, 0, 3000], [24, 24, 1, 90]]
    q, store = queries(48, 8, D, 44), random_store(3008, 2, 1, D, 44)
    clean, _ = run_q4(q, store, seq, dev, causal=True)
    for t, h, d, x in ((2, 1, 5, "nan"), (17, 7, 63, "inf"), (30, 3, 0, "nan"), (47, 0, 1, "-inf")):
        q[t, h, d] = float(x)
    got, _ = run_q4(q, store, seq, dev, causal=True)
    for t, h in ((2, 1), (17, 7), (30, 3), (47, 0)):
        assert bool(got[t, h].isnan().any()), (t, h)
        got[t, h] = clean[t, h]
    assert torch.equal(got.view(torch.int16), clean.view(torch.int16))


def test_the_same_call_gives_the_same_bits(dev):
    store = random_store(4096, 6, 2, 128, 45)
    for seq, Hq in (([[i, 1, i, 4000 - i] for i in range(6)], 16), ([[40 * i, 40, i, 4000 - i] for i in range(6)], 8)):
        q = queries(seq[-1][0] + seq[-1][1], Hq, 128, 45)
        first, _ = run_q4(q, store, seq, dev, causal=True)
        for _ in range(10):
            again, _ = run_q4(q, store, seq, dev, causal=True)
            assert torch.equal(first.view(torch.int16), again.view(torch.int16))


def test_one_workspace_for_calls_of_different_sizes(dev):
    # the workspace of the largest call serves the smaller ones, whichever kernel they take
    store = random_store(2048, 6, 2, 128, 46)
    stored = pkg.Q4Store(*(t.to(dev) for t in store))
    ws = torch.full((pkg.q4_workspace_bytes(240, 16, stored, 6),), 255, dtype=torch.uint8, device=dev)
    for n, S_ in ((40, 6), (1, 6), (3, 6), (2, 6), (17, 6), (240, 1), (1, 1), (70, 2), (200, 1)):
        seq = [[n * i, n, i, 2000 - 300 * i] for i in range(S_)]
        q = queries(S_ * n, 16, 128, 46)
        got = pkg.sdpa_varlen_q4(q.to(dev), stored, torch.tensor(seq, dtype=torch.int32, device=dev), causal=True,
                                 workspace=ws)
        check(got, 0, q, store, seq, True, p_step=2.0 ** -8, rows_subset=sorted({0, S_ * n // 2, S_ * n - 1}))


def test_two_captured_graphs_of_one_workspace_replayed_in_turn(dev):
    store = random_store(1024, 4, 2, 128, 47)
    stored = pkg.Q4Store(*(t.to(dev) for t in store))
    ws = torch.empty(pkg.q4_workspace_bytes(120, 8, stored, 4), dtype=torch.uint8, device=dev)
    sides = []
    for n in (1, 30):
        seq = [[n * i, n, i, 1000 - 99 * i] for i in range(4)]
        q = queries(4 * n, 8, 128, 47 + n)
        qd, seqd = q.to(dev), torch.tensor(seq, dtype=torch.int32, device=dev)
        out = torch.empty_like(qd)
        call = lambda qd=qd, seqd=seqd, out=out: pkg.sdpa_varlen_q4(qd, stored, seqd, causal=True, out=out, workspace=ws)
        call()
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            call()
        sides.append((g, q, seq, out))
    for _ in range(3):
        for g, q, seq, out in sides:
            out.fill_(float("nan"))
            g.replay()
            check(out, 0, q, store, seq, True)


def test_python_entries_refuse_mixed_devices_and_foreign_streams(dev):
    store = pkg.q4_store(64, 2, 2, 64, device=dev)
    q, seq = queries(3, 4, 64, 48).to(dev), torch.tensor([[0, 3, 0, 5]], dtype=torch.int32, device=dev)
    k = queries(3, 2, 64, 49).to(dev)
    table = pkg.rope_table(16, 64, device=dev)

    class Foreign:
        device_index, cuda_stream = 7, 0

    with pytest.raises(ValueError, match="stream is on device 7"):
        pkg.sdpa_rope(q, table, seq[0, :3].contiguous(), out=torch.empty_like(q), stream=Foreign())
    for call in (lambda: pkg.sdpa_rope(q, table.cpu(), seq[0, :3].contiguous()),
                 lambda: pkg.sdpa_rope_append_q4(q, k, k.cpu(), store, seq, table),
                 lambda: pkg.sdpa_rope_append_q4(q, k, k, store, seq.cpu(), table),
                 lambda: pkg.sdpa_q4_unpack(store._replace(v_scales=store.v_scales.cpu()), seq, 3),
                 lambda: pkg.sdpa_varlen_q4(q, store, seq, causal=True, out=torch.empty(3, 4, 64, dtype=q.dtype))):
        with pytest.raises(ValueError, match="same CUDA device"):
            call()
    with pytest.raises(pkg.SdpaError, match="workspace of"):
        pkg.sdpa_varlen_q4(q, store, seq, causal=True, workspace=torch.empty(1024, dtype=torch.uint8, device=dev))
    with pytest.raises(pkg.SdpaError, match="16-byte aligned|multiples of 8"):
        pkg.sdpa_rope(torch.empty(3, 4 * 64 + 2, dtype=q.dtype, device=dev)[:, 2:].unflatten(1, (4, 64)), table,
                      seq[0, :3].contiguous())
    small = pkg.Q4Store(*(t[:, :, :24].contiguous() for t in store))
    with pytest.raises(pkg.SdpaError, match="multiple of 16 rows"):
        pkg.sdpa_varlen_q4(q, small, seq, causal=True)


@pytest.mark.parametrize("S_", [20, 70])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("chunk,kv,long", [
    (120, 130, 1500),   # a chunk over few keys among tokens over many: the split-K kernel for few rows
    (120, 1500, 40),    # over many keys: the tensor-memory one
    (400, 1500, 1500),  # long enough to be staged in bf16, tokens beside it
])
def test_a_chunk_among_single_tokens_takes_the_cheaper_kernel(dev, S_, D, chunk, kv, long):
    seq, t = [], 0
    for i in range(S_):
        n = chunk if i == S_ // 2 else 1
        seq.append([t, n, i, max(n, kv) if n > 1 else long - i % 9])
        t += n
    seq[3][2] = S_ + 5  # one segment of no column
    store, q = random_store(1504, S_, 2, D, D + S_), queries(t + 2, 32, D, 50)
    rows = sorted({0, 1, 3, t - 1, t, t + 1} | {S_ // 2 + i for i in (-1, 0, 1, chunk // 2, chunk - 1, chunk)})
    for causal in (True, False):
        got, st = run_q4(q, store, seq, dev, causal=causal)
        check(got, st, q, store, seq, causal, p_step=2.0 ** -8, rows_subset=rows)
    got, st = run_q4(q, store, seq, dev, causal=True, window=100)
    check(got, st, q, store, seq, True, 100, p_step=2.0 ** -8, rows_subset=rows)


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("S_,Hq,Hkv", [(300, 8, 2), (512, 2, 1), (513, 2, 1), (170, 64, 2)])
def test_tables_of_many_single_tokens(dev, D, S_, Hq, Hkv):
    # with columns shared, empty and invalid entries, tokens out of order, and two that overlap
    rng = np.random.default_rng(S_ + D)
    order = rng.permutation(S_)
    seq = [[int(order[i]), 1, i % 23, int(rng.integers(0, 129))] for i in range(S_)]
    seq[5][1], seq[9][2], seq[11][3] = 0, 23, -4
    seq[17][0] = seq[40][0]
    seq[60][0] = -1
    store, q = random_store(128, 23, Hkv, D, S_), queries(S_, Hq, D, 60)
    modes = [[i % 2, [0, 1, 20, 128][i % 4]] for i in range(S_)]
    rows = sorted({int(order[i]) for i in (0, 5, 9, 11, 17, 40, 60, 61, S_ - 1)} | set(range(0, S_, 37)))
    for m in (None, modes):
        got, st = run_q4(q, store, seq, dev, causal=True, seg_mode=m)
        check(got, st, q, store, seq, True, 0, m, rows_subset=rows)


def test_the_workspace_status_of_a_call_without_a_schedule(dev):
    store = pkg.q4_store(64, 2, 1, 64, device=dev)
    ws = torch.full((pkg.q4_workspace_bytes(4, 2, store, 3),), 255, dtype=torch.uint8, device=dev)
    q = queries(4, 2, 64, 61).to(dev)
    for seq in ([[0, 1, 0, 5], [1, 1, 1, 6], [2, 1, 0, 7]], [[0, 2, 0, 5], [1, 1, 1, 6], [3, 1, 7, 9]],
                [[0, 2, 0, 5], [0, 0, 1, 6], [3, 1, 1, -9]]):
        pkg.sdpa_varlen_q4(q, store, torch.tensor(seq, dtype=torch.int32, device=dev), causal=True, workspace=ws)
        _, _, _, want = O.visible_interval(np.array(seq), 4, True, 0, 64, 2, None)
        assert pkg.workspace_status(ws) == want


@pytest.mark.parametrize("n,Hq", [(1, 4), (5, 4), (3, 8)])
def test_more_segments_than_the_scheduler_keeps_in_shared_memory(dev, n, Hq):
    # 1100 segments, columns shared by many, one of them longer, some invalid, two overlapping
    S_ = 1100
    seq, t = [], 0
    for i in range(S_):
        m = 150 if i == 700 else n
        seq.append([t, m, (7 * i) % 31, max(m, 1 + (13 * i) % 160)])
        t += m
    seq[3][2], seq[500][3], seq[900][0] = 31, -1, seq[899][0]
    store, q = random_store(160, 31, 1, 64, n), queries(t, Hq, 64, 70)
    chunk = seq[700][0]
    rows = sorted({0, t - 1, chunk - 1, chunk, chunk + 77, chunk + 149, chunk + 150} |
                  {seq[i][0] + j for i in (3, 4, 500, 501, 898, 899, 901, 1099) for j in range(n)} |
                  {seq[900][0], seq[901][0] - 1})
    for causal, window in ((True, 0), (False, 0), (True, 11)):
        got, st = run_q4(q, store, seq, dev, causal=causal, window=window)
        check(got, st, q, store, seq, causal, window, p_step=2.0 ** -8, rows_subset=rows)


def test_staged_route_more_segments_than_the_scheduler_keeps_in_shared_memory(dev, prefill_route):
    seq = [[2 * i, 2, (5 * i) % 29, 2 + (11 * i) % 150] for i in range(1100)]
    seq[8][2] = 40
    store, q = random_store(160, 29, 1, 64, 71), queries(2200, 2, 64, 71)
    got, st = run_q4(q, store, seq, dev, causal=True)
    check(got, st, q, store, seq, True, p_step=2.0 ** -8, rows_subset=[0, 1, 15, 16, 17, 1000, 1001, 2198, 2199])
