"""The rotated queries of an 8-bit append, written into part of a larger tensor."""
import numpy as np
import pytest
import torch

import varlen_gqa_attention_gb300 as pkg
from oracle import step_oracle as S
from test_rope_gpu import assert_rotated

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    torch.cuda.set_device(0)
    return torch.device("cuda:0")


def test_rotated_queries_into_part_of_a_larger_tensor(dev):
    # from rows that all heads share, every (row, head) its own place among others that stay as they are
    D, Hkv, Hq, T = 64, 3, 6, 21
    g = torch.Generator().manual_seed(4)
    base = torch.randn(T, 4, D, generator=g).to(torch.bfloat16)
    seq = np.array([[0, 20, 0, 25]], dtype=np.int32)
    table = pkg.rope_table(32, D)
    q = base[:, :1].expand(T, Hq, D)
    ref, _, wrote, _ = S.rope_append(q, base[:, 1:2].expand(T, Hkv, D), base[:, 2:3].expand(T, Hkv, D), 32, 1, seq, 0,
                                     table, (D // 2,))
    bd, seqd = base.to(dev), torch.from_numpy(seq).to(dev)
    for where in (np.s_[:, 1:7, :D], np.s_[:, 2:8, D:], np.s_[:, ::2, 16:16 + D]):
        out = torch.full((T, 9 if where[1] != np.s_[::2] else 12, 2 * D), 5.0, dtype=torch.bfloat16, device=dev)
        view = out[where]
        store = pkg.q8_store(32, 1, Hkv, D, device=dev)
        got = pkg.sdpa_rope_append_q8(bd[:, :1].expand(T, Hq, D), bd[:, 1:2].expand(T, Hkv, D),
                                      bd[:, 2:3].expand(T, Hkv, D), store, seqd, table.to(dev), q_out=view)
        assert got.data_ptr() == view.data_ptr() and len(wrote) == 20
        assert_rotated(view, ref, q, D, False)
        assert not bool(view[20].any())
        rest = torch.ones_like(out, dtype=torch.bool)
        rest[where] = False
        assert bool((out[rest] == 5).all())
