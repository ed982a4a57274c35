"""Attention over codes that no append writes: code 0 under the largest scales stands for -65536, on every route.

Keys of 0 give every visible key the same weight, 2^-6 of 64 keys, and the values are whole numbers whose sums fp32
holds, so the outputs are known to the bit."""
import pytest
import torch

import varlen_gqa_attention_gb300 as pkg

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    torch.cuda.set_device(0)
    return torch.device("cuda:0")


@pytest.fixture(params=["auto", "splitk", "prefill"], autouse=True)
def route(request):
    pkg.set_route_policy({"auto": pkg.ROUTE_AUTO, "splitk": pkg.ROUTE_SPLITK, "prefill": pkg.ROUTE_PREFILL}[request.param])
    yield request.param
    pkg.set_route_policy(pkg.ROUTE_AUTO)


@pytest.mark.parametrize("byte", [29, 30, 255])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("n", [1, 3, 150])
def test_values_of_the_lowest_code(dev, byte, D, n):
    Hq, Hkv, rows = 8, 2, 64
    store = pkg.q8_store(rows, 2, Hkv, D, device=dev)
    store.v_scales.fill_(byte)
    store.v_codes[0] = 0
    store.v_codes[1, :, ::2], store.v_codes[1, :, 1::2] = 0, 255
    q = torch.randn(2 * n, Hq, D, generator=torch.Generator().manual_seed(n)).to(torch.bfloat16).to(dev)
    seq = torch.tensor([[0, n, 0, rows], [n, n, 1, rows]], dtype=torch.int32, device=dev)
    out = pkg.sdpa_varlen_q8(q, store, seq, causal=False)
    assert bool((out[:n] == -65536).all())
    assert bool((out[n:] == (65024 - 65536) / 2).all())
    one = pkg.sdpa_varlen_q8(q, store, seq, causal=True, window=1)  # (rows before the beginning see nothing)
    p = rows - n + torch.arange(n, device=dev)
    want = torch.where(p < 0, 0, torch.where(p % 2 == 1, 65024, -65536)).to(torch.bfloat16)
    assert bool((one[:n] == torch.where(p < 0, 0, -65536).to(torch.bfloat16)[:, None, None]).all())
    assert bool((one[n:] == want[:, None, None]).all())
