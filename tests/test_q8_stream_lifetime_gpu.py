"""Outputs of 8-bit calls on a given stream: their memory stays theirs until both that stream and the one that was
current at the call have done what was queued before they were dropped."""
import pytest
import torch

import varlen_gqa_attention_gb300 as pkg

from test_q4_attention_gpu import queries

pytestmark = pytest.mark.gpu
T, D = 512, 128


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    torch.cuda.set_device(0)
    return torch.device("cuda:0")


def entry_call(dev, entry):
    x, k = queries(T, 4, D, 1).to(dev), queries(T, 4, D, 2).to(dev)
    table = pkg.rope_table(T, D, device=dev)
    seq = torch.tensor([[0, T, 0, T]], dtype=torch.int32, device=dev)
    store = pkg.q8_store(T, 1, 4, D, device=dev)
    pkg.sdpa_rope_append_q8(x, k, k, store, seq, table)
    return {
        "append": lambda **kw: pkg.sdpa_rope_append_q8(x, k, k, store, seq, table, **kw),
        "unpack_k": lambda **kw: pkg.sdpa_q8_unpack(store, seq, T, **kw)[0],
        "unpack_v": lambda **kw: pkg.sdpa_q8_unpack(store, seq, T, **kw)[1],
        "attention": lambda **kw: pkg.sdpa_varlen_q8(x, store, seq, causal=True, **kw),
    }[entry]


@pytest.mark.parametrize("entry", ["append", "unpack_k", "unpack_v", "attention"])
def test_a_dropped_output_is_not_written_again_while_it_is_read(dev, entry):
    side = torch.cuda.Stream(dev)
    call = entry_call(dev, entry)
    want = call().clone()
    seen = torch.empty_like(want)
    torch.cuda.synchronize()
    side.wait_stream(torch.cuda.current_stream())
    out = call(stream=side)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda._sleep(200_000_000)  # a tenth of a second before the current stream reads it
    seen.copy_(out)
    del out
    with torch.cuda.stream(side):
        others = [torch.full_like(want, 7.0) for _ in range(8)]
    torch.cuda.synchronize()
    assert bool((seen.view(torch.int16) == want.view(torch.int16)).all())
    del others


@pytest.mark.parametrize("entry", ["append", "unpack_k", "attention"])
def test_an_output_takes_no_memory_that_the_current_stream_still_reads(dev, entry):
    side = torch.cuda.Stream(dev)
    call = entry_call(dev, entry)
    call(stream=side)  # (kernels loaded, workspaces of this size known to the allocator)
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
    out = call(stream=side)
    torch.cuda.synchronize()
    assert all(bool((t == 5).all()) for t in seen)
    del out
