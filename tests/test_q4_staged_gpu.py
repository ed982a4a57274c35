"""What the staged route of the 4-bit attention (long chunks, keys and values brought to 16 bits in the
workspace) has to keep like the other routes: probabilities of fp16, and rows of NaN or infinity.

Keys here are small (scale bytes 120 to 127, at most 0.24 in magnitude), so that a score's rounding does not
hide a probability's: 2 * 2 D 2^-23 scale max|q| max sum|k| comes to about 2^-13 of a row's magnitudes at
D = 64 (max|q| 4.2, sum|k| 7) and 2^-10 at D = 256 (4.5, 26)."""
import pytest
import torch

import varlen_gqa_attention_gb300 as pkg

from test_q4_attention_gpu import check, queries, random_store, run_q4

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    torch.cuda.set_device(0)
    return torch.device("cuda:0")


@pytest.fixture
def staged():
    pkg.set_route_policy(pkg.ROUTE_PREFILL)
    yield
    pkg.set_route_policy(pkg.ROUTE_AUTO)


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("seq,rows,window", [
    ([[0, 40, 1, 40], [42, 3, 0, 2]], 48, 0),         # rows that see one key, two keys, ...; one that sees none
    ([[0, 150, 1, 2000], [150, 300, 0, 300]], 2000, 0),  # units cut over several CTAs
    ([[0, 200, 1, 1000], [200, 30, 0, 40]], 272, 40),  # a ring that has wrapped
])
def test_probabilities_keep_fp16(dev, staged, D, seq, rows, window):
    store, q = random_store(rows, 2, 2, D, D, lo=120, hi=128), queries(seq[-1][0] + seq[-1][1] + 1, 8, D, 90)
    subset = None if rows < 1000 else list(range(0, 152, 3)) + list(range(152, 460, 7))
    subset = subset and [t for t in subset if t < q.shape[0]]
    got, st = run_q4(q, store, seq, dev, causal=True, window=window)
    check(got, st, q, store, seq, True, window, p_step=2.0 ** -11, rows_subset=subset)


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("kv", [50, 3000])  # one CTA a unit, and several
def test_a_row_of_nan_or_infinity_stays_alone(dev, staged, D, kv):
    seq = [[0, 48, 1, kv]]
    store, q = random_store(3008, 2, 2, D, D), queries(48, 8, D, 91)
    want, _ = run_q4(q, store, seq, dev, causal=False)
    bad = {(2, 1): "nan", (17, 7): "inf", (30, 3): "nan", (47, 0): "-inf"}
    for (t, h), x in bad.items():
        q[t, h, 5 * h] = float(x)
    got, st = run_q4(q, store, seq, dev, causal=False)
    assert st == 0
    for t, h in bad:
        assert bool(got[t, h].isnan().all()), (t, h)
        got[t, h] = want[t, h]
    assert bool((got.view(torch.int16) == want.view(torch.int16)).all())
