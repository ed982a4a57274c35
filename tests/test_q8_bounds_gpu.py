"""GPU parity of attention over the 8-bit store where scales differ most, held row by row to what its roundings allow
(tests/q8_bounds.py, whose bound tests/test_q8_bounds.py tries on wrong outputs)."""
import pytest
import torch

import q8_bounds as B
import varlen_gqa_attention_gb300 as pkg
from test_q4_attention_gpu import queries
from test_q8_append_gpu import random_store
from test_q8_attention_gpu import run_q8
from test_q8_bounds import SEQ, cases

pytestmark = pytest.mark.gpu


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


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("window", [0, 24])
@pytest.mark.parametrize("which", ["values", "keys"])
def test_blocks_of_the_smallest_and_the_largest_scale(dev, route, D, window, which):
    store, scale = cases(D)[which]
    q = queries(24, 4, D, 8)
    got, st = run_q8(q, store, SEQ, dev, causal=True, window=window, scale=scale)
    assert st == 0
    B.hold(got, q, store, SEQ, True, window, scale)
    one = [[0, 24, 1, 140]]  # one segment, whose rows see more and more of them
    got, st = run_q8(q, store, one, dev, causal=True, window=window, scale=scale)
    assert st == 0
    B.hold(got, q, store, one, True, window, scale)


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("n", [1, 7, 40])
def test_values_of_every_byte_pattern(dev, route, D, n):
    # codes and scale bytes of all kinds, code 0 under the largest scale among them
    store = random_store(272, 3, 2, D, D + n, 0, 256)
    for s in (store.k_scales, store.v_scales):
        s.copy_(torch.where(torch.rand(s.shape, generator=torch.Generator().manual_seed(n)) < 0.3, s % 30, s))
    store.k_scales.copy_(12 + store.k_scales % 3)
    seq = [[0, n, 2, 270], [n, n, 0, 100], [2 * n + 1, n, 1, max(n, 17)]]
    q = queries(3 * n + 2, 8, D, n)
    for causal, window in ((True, 0), (False, 0), (True, 33)):
        got, st = run_q8(q, store, seq, dev, causal=causal, window=window)
        assert st == 0
        B.hold(got, q, store, seq, causal, window, tag=f"{causal} {window}")


@pytest.mark.parametrize("D", [64, 128, 256])
def test_blocks_that_no_row_sees(dev, route, D):
    # of the largest scale, or ordinary: the same bits, whatever shares a tile with them
    ordinary = random_store(192, 2, 2, D, 9, 10, 14)
    store = pkg.Q8Store(*(t.clone() for t in ordinary))
    seq, window = [[0, 3, 0, 70], [3, 20, 1, 128], [23, 1, 0, 31]], 40
    seen = torch.zeros(2, 12, dtype=torch.bool)
    for q_start, n, col, kv in seq:
        seen[col, max(0, kv - n - window + 1) // 16:(kv - 1) // 16 + 1] = True
    for c, s in ((store.k_codes, store.k_scales), (store.v_codes, store.v_scales)):
        for col in range(2):
            s[col, :, ~seen[col]] = 29
            c[col].view(2, 12, 16, D)[:, ~seen[col]] = 0
    assert not seen[0].all() and not seen[1].all()
    q = queries(24, 4, D, 9)
    a, _ = run_q8(q, ordinary, seq, dev, causal=True, window=window)
    b, _ = run_q8(q, store, seq, dev, causal=True, window=window)
    assert torch.equal(a.view(torch.int16), b.view(torch.int16))
    B.hold(b, q, store, seq, True, window)
