"""Buffers that a call would write through or read beyond are refused before anything is launched."""
import pytest
import torch

import varlen_gqa_attention_gb300 as pkg

from test_q4_attention_gpu import queries

pytestmark = pytest.mark.gpu


@pytest.fixture
def call():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    dev = torch.device("cuda:0")
    torch.cuda.set_device(0)
    q, k = queries(3, 4, 64, 1).to(dev), queries(3, 2, 64, 2).to(dev)
    cols = [torch.zeros(64, 1, 2, 64, dtype=torch.bfloat16, device=dev) for _ in range(2)]
    seq = torch.tensor([[0, 3, 0, 40]], dtype=torch.int32, device=dev)
    mode, store = torch.tensor([[1, 0]], dtype=torch.int32, device=dev), pkg.q4_store(64, 1, 2, 64, device=dev)
    return {
        "varlen": lambda **kw: pkg.sdpa_varlen(q, *cols, seq, causal=True, **kw),
        "append": lambda **kw: pkg.sdpa_varlen_append(q, k, k, *cols, seq, causal=True, **kw),
        "modes": lambda **kw: pkg.sdpa_varlen_modes(q, *cols, seq, mode, **kw),
        "q4": lambda **kw: pkg.sdpa_varlen_q4(q, store, seq, causal=True, **kw),
        "dense": lambda **kw: pkg.sdpa_causal_prefill(q, k, k, **kw),
    }


@pytest.mark.parametrize("entry", ["varlen", "append", "modes", "q4", "dense"])
def test_workspaces_and_outputs(call, entry):
    byte = dict(dtype=torch.uint8, device="cuda")
    for ws in (torch.empty(1 << 24, dtype=torch.uint8), torch.empty(1, **byte).expand(1 << 24),
               torch.empty(1 << 25, **byte)[::2]):
        with pytest.raises(ValueError, match="workspace must be contiguous|workspace must be a contiguous|same CUDA device"):
            call[entry](workspace=ws)
    rows = dict(dtype=torch.bfloat16, device="cuda")
    for out in (torch.empty(3, 4, 64, dtype=torch.bfloat16), torch.empty(2, 4, 64, **rows), torch.empty(3, 4, 32, **rows),
                torch.empty(3, 4, 64, dtype=torch.float32, device="cuda"), torch.empty(3, 4, 128, **rows)[:, :, ::2]):
        with pytest.raises(ValueError):
            call[entry](out=out)


@pytest.mark.parametrize("entry", ["varlen", "append", "modes", "q4"])
@pytest.mark.parametrize("status", ["host", "int64", "none"])
def test_status_words(call, entry, status):
    word = {"host": torch.zeros(1, dtype=torch.int32), "int64": torch.zeros(1, dtype=torch.int64, device="cuda"),
            "none": torch.zeros(0, dtype=torch.int32, device="cuda")}[status]
    with pytest.raises(ValueError, match="status must be an int32 tensor|same CUDA device"):
        call[entry](status=word)


def test_shapes_of_dense_keys_and_values(call):
    q, k = queries(3, 4, 64, 1).cuda(), queries(5, 2, 64, 2).cuda()
    for kk, vv in ((k, k[:4].contiguous()), (k, k[:, :1].contiguous()), (k[:, :, :32].contiguous(),) * 2):
        with pytest.raises(ValueError, match=r"\[Lkv, Hkv, D\]"):
            pkg.sdpa_causal_prefill(q, kk, vv)
    assert call["dense"](out=torch.empty_like(q)).shape == q.shape
