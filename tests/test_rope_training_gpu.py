"""The rotation inside a training step's own autograd function."""
import numpy as np
import pytest
import torch

import varlen_gqa_attention_gb300 as pkg
from oracle import step_oracle as S

pytestmark = pytest.mark.gpu


class Rotate(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, table, positions):
        ctx.save_for_backward(table, positions)
        return pkg.sdpa_rope(x, table, positions)

    @staticmethod
    def backward(ctx, dy):
        return pkg.sdpa_rope(dy, *ctx.saved_tensors, inverse=True), None, None


@pytest.mark.parametrize("shared", [False, True])  # one head's rows, broadcast to four
def test_gradients_reach_the_rows(shared):
    dev, T, H, D = torch.device("cuda:0"), 21, 4, 64
    g = torch.Generator().manual_seed(3)
    x = torch.randn(T, 1 if shared else H, D, generator=g).to(torch.bfloat16).to(dev).requires_grad_()
    w = torch.randn(T, H, D, generator=g).to(torch.bfloat16)
    table, pos = pkg.rope_table(100, 48, device=dev), torch.arange(T, dtype=torch.int32, device=dev) * 3
    y = Rotate.apply(x.expand(T, H, D), table, pos)
    ref, _ = S.rope(x.detach().expand(T, H, D).contiguous(), table.cpu(), pos.cpu(), (24,))
    assert np.abs(S.f64(y) - ref).max() <= 2.0 ** -8 * 6.0
    y.backward(w.to(dev))
    dx, _ = S.rope(w, table.cpu(), pos.cpu(), (24,), inverse=True)
    # a turned pair is at most sqrt(2) of its larger value, here below 4.5, so that each of the H gradients is rounded
    # by at most 2^-9 * 8; their sum by bf16 again, H times H partial sums at most
    n = H if shared else 1
    want = dx.sum(1, keepdims=True) if shared else dx
    bound = n * 2.0 ** -6 + (n > 1) * n * 2.0 ** -8 * np.abs(dx).sum(1, keepdims=True)
    assert (np.abs(S.f64(x.grad) - want) <= bound).all()
