"""Outputs of calls on a given stream: their memory stays theirs until both that stream and the one that was
current at the call have done what was queued before they were dropped."""
import pytest
import torch

import varlen_gqa_attention_gb300 as pkg

from test_q4_attention_gpu import queries

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    torch.cuda.set_device(0)
    return torch.device("cuda:0")


@pytest.mark.parametrize("entry", ["rope", "append", "append_q4", "unpack", "attention"])
def test_a_dropped_output_is_not_written_again_while_it_is_read(dev, entry):
    T, D = 512, 128
    side = torch.cuda.Stream(dev)
    x, k = queries(T, 4, D, 1).to(dev), queries(T, 4, D, 2).to(dev)
    table = pkg.rope_table(T, D, device=dev)
    pos = torch.arange(T, dtype=torch.int32, device=dev)
    seq = torch.tensor([[0, T, 0, T]], dtype=torch.int32, device=dev)
    store = pkg.q4_store(T, 1, 4, D, device=dev)
    cols = [torch.zeros(T, 1, 4, D, dtype=torch.bfloat16, device=dev) for _ in range(2)]
    calls = {
        "rope": lambda **kw: pkg.sdpa_rope(x, table, pos, **kw),
        "append": lambda **kw: pkg.sdpa_rope_append(x, k, k, *cols, seq, table, **kw),
        "append_q4": lambda **kw: pkg.sdpa_rope_append_q4(x, k, k, store, seq, table, **kw),
        "unpack": lambda **kw: pkg.sdpa_q4_unpack(store, seq, T, **kw)[0],
        "attention": lambda **kw: pkg.sdpa_varlen_q4(x, store, seq, causal=True, **kw),
    }
    want = calls[entry]().clone()
    seen = torch.empty_like(want)
    torch.cuda.synchronize()
    side.wait_stream(torch.cuda.current_stream())
    out = calls[entry](stream=side)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda._sleep(200_000_000)  # a tenth of a second before the current stream reads it
    seen.copy_(out)
    del out
    with torch.cuda.stream(side):
        others = [torch.full_like(want, 7.0) for _ in range(8)]
    torch.cuda.synchronize()
    assert bool((seen.view(torch.int16) == want.view(torch.int16)).all())
    del others


@pytest.mark.parametrize("entry", ["varlen", "varlen_append", "modes", "dense", "static", "rope", "append", "append_q4",
                                   "unpack", "attention"])
def test_an_output_takes_no_memory_that_the_current_stream_still_reads(dev, entry):
    T, D = 512, 128
    side = torch.cuda.Stream(dev)
    x, k = queries(T, 4, D, 1).to(dev), queries(T, 4, D, 2).to(dev)
    table = pkg.rope_table(T, D, device=dev)
    pos = torch.arange(T, dtype=torch.int32, device=dev)
    seq = torch.tensor([[0, T, 0, T]], dtype=torch.int32, device=dev)
    mode = torch.tensor([[1, 0]], dtype=torch.int32, device=dev)
    store = pkg.q4_store(T, 1, 4, D, device=dev)
    cols = [torch.zeros(T, 1, 4, D, dtype=torch.bfloat16, device=dev) for _ in range(2)]
    call = {
        "varlen": lambda: pkg.sdpa_varlen(x, *cols, seq, causal=True, stream=side),
        "varlen_append": lambda: pkg.sdpa_varlen_append(x, k, k, *cols, seq, causal=True, stream=side),
        "modes": lambda: pkg.sdpa_varlen_modes(x, *cols, seq, mode, stream=side),
        "dense": lambda: pkg.sdpa_causal_prefill(x, k, k, stream=side),
        "static": lambda: pkg.sdpa_varlen_splitk_static(x, *cols, seq, causal=True, stream=side),
        "rope": lambda: pkg.sdpa_rope(x, table, pos, stream=side),
        "append": lambda: pkg.sdpa_rope_append(x, k, k, *cols, seq, table, stream=side),
        "append_q4": lambda: pkg.sdpa_rope_append_q4(x, k, k, store, seq, table, stream=side),
        "unpack": lambda: pkg.sdpa_q4_unpack(store, seq, T, stream=side),
        "attention": lambda: pkg.sdpa_varlen_q4(x, store, seq, causal=True, stream=side),
    }[entry]
    call()  # (kernels loaded, workspaces of this size known to the allocator)
    torch.cuda.synchronize()
    side.wait_stream(torch.cuda.current_stream())
    # blocks of an output's size and of larger ones, read by the current stream a tenth of a second from now
    sizes = [T * 4 * D * 2] * 4 + [1 << 21, 1 << 22, 1 << 23, 1 << 24, 1 << 25]
    read = [torch.full((n,), 5, dtype=torch.uint8, device=dev) for n in sizes]
    seen = [torch.empty_like(t) for t in read]
    torch.cuda._sleep(200_000_000)
    for a, b in zip(seen, read):
        a.copy_(b)
    del read, b
    out = call()
    torch.cuda.synchronize()
    assert all(bool((t == 5).all()) for t in seen)
    del out
