"""The rows that pad a unit of the prefill kernels: what lies behind a segment in q, and what such rows make of the
keys, leaves the segment's own rows as they are, bit for bit.

A unit holds 128 packed rows (D = 256) or 256; 21 tokens of 8 heads a KV head fill 168.  What follows the segment in q
belongs to no segment or to another one."""
import pytest
import torch

import varlen_gqa_attention_gb300 as pkg

from test_q4_attention_gpu import queries, random_store as random_q4
from test_q8_attention_gpu import random_store as random_q8

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    torch.cuda.set_device(0)
    return torch.device("cuda:0")


@pytest.fixture(autouse=True)
def staged():
    pkg.set_route_policy(pkg.ROUTE_PREFILL)
    yield
    pkg.set_route_policy(pkg.ROUTE_AUTO)


def calls(D, rows, Hkv, dev):
    """The three stores' attention over stores of their own."""
    g = torch.Generator().manual_seed(D)
    k, v = (torch.randn(rows, 2, Hkv, D, generator=g).to(torch.bfloat16).to(dev) for _ in range(2))
    q4, q8 = (type(s)(*(t.to(dev) for t in s)) for s in (random_q4(rows, 2, Hkv, D, D), random_q8(rows, 2, Hkv, D, D)))
    return {"bf16": lambda q, seq, **kw: pkg.sdpa_varlen(q, k, v, seq, **kw),
            "q4": lambda q, seq, **kw: pkg.sdpa_varlen_q4(q, q4, seq, **kw),
            "q8": lambda q, seq, **kw: pkg.sdpa_varlen_q8(q, q8, seq, **kw)}, (k, v)


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("n,kv", [(21, 1000), (21, 130), (1, 700), (50, 3000)])
def test_what_lies_behind_a_segment_in_q(dev, D, n, kv):
    Hq, Hkv, T = 16, 2, n + 40
    run, _ = calls(D, 3008, Hkv, dev)
    seq = torch.tensor([[0, n, 1, kv]], dtype=torch.int32, device=dev)
    q = queries(T, Hq, D, n).to(dev)
    for name, call in run.items():
        for kw in (dict(causal=True), dict(causal=False), dict(causal=True, window=500)):
            plain = call(q, seq, **kw)
            assert bool(plain[:n].isfinite().all()) and not bool(plain[n:].any())
            for x in (0.0, float("nan"), float("inf"), float("-inf"), 3e38, None):
                other = q.clone()
                other[n:] = x if x is not None else 200 * q[n:]
                got = call(other, seq, **kw)
                assert torch.equal(got.view(torch.int16), plain.view(torch.int16)), (name, kw, x)


@pytest.mark.parametrize("D", [64, 128, 256])
def test_another_segments_rows_behind_one(dev, D):
    # the second segment's rows pad the first one's unit, over a column that is not theirs
    n, Hq, Hkv = 21, 16, 2
    run, _ = calls(D, 1008, Hkv, dev)
    seq = torch.tensor([[0, n, 1, 1000], [n, 40, 0, 900]], dtype=torch.int32, device=dev)
    q = queries(n + 40, Hq, D, n).to(dev)
    other = q.clone()
    other[n:] = float("nan")
    for name, call in run.items():
        plain, got = call(q, seq, causal=True), call(other, seq, causal=True)
        assert torch.equal(got[:n].view(torch.int16), plain[:n].view(torch.int16)), name
        assert bool(plain.isfinite().all()), name
        if name != "bf16":  # (whose entry leaves the outputs of rows that are NaN themselves open)
            assert bool(got[n:].isnan().all()), name


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("x", [float("nan"), float("inf"), float("-inf")])
def test_keys_that_only_the_last_row_and_the_padding_see(dev, D, x):
    n, kv, Hq, Hkv = 21, 1000, 16, 2
    run, (k, _) = calls(D, 1008, Hkv, dev)
    seq = torch.tensor([[0, n, 1, kv]], dtype=torch.int32, device=dev)
    q = queries(n + 40, Hq, D, n).to(dev)
    plain = run["bf16"](q, seq, causal=True)
    k[kv - 1, 1] = x
    got = run["bf16"](q, seq, causal=True)
    assert torch.equal(got[:n - 1].view(torch.int16), plain[:n - 1].view(torch.int16))
    k[kv:, 1] = x  # behind the last position: nobody's
    assert torch.equal(run["bf16"](q, seq, causal=True)[:n - 1].view(torch.int16), plain[:n - 1].view(torch.int16))
