"""What the bound of the 8-bit attention's outputs (tests/q8_bounds.py) holds and what it rejects, on the CPU."""
import numpy as np
import pytest
import torch

import q8_bounds as B
from oracle import sdpa_varlen_oracle as O
from oracle import step_oracle as S
from test_q4_attention_gpu import queries
from test_q8_append_gpu import random_store

SEQ = [[0, 3, 0, 190], [3, 20, 1, 128], [23, 1, 0, 31]]


def cases(D):
    """Stores whose blocks have the smallest scale and the largest beside each other, in values and in keys."""
    v = random_store(192, 2, 2, D, 7, 10, 14)
    for col, every in ((0, (0, 6)), (1, (0, 6, 29))):
        for i, b in enumerate(every):
            v.v_scales[col, :, i::len(every)] = b
    k = random_store(192, 2, 2, D, 8, 12, 16)
    k.k_scales[0] = 29
    k.k_scales[1, :, ::2], k.k_scales[1, :, 1::2] = 29, 19
    return {"values": (v, D ** -0.5), "keys": (k, 2.0 ** -19)}


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("window", [0, 24])
def test_the_bound_holds_the_rounded_result_and_rejects_others(D, window):
    q = queries(24, 4, D, 8)
    for name, (store, scale) in cases(D).items():
        k, v = B.stores(store)
        ref, _, _ = O.sdpa_varlen(q, k, v, SEQ, True, window, scale, None, None)
        args = (q, store, SEQ, True, window, scale)
        good = S.to_bf16(ref)
        B.hold(good, *args)
        flipped, swapped = -good, good.roll(1, dims=1)
        one = good.clone()  # a single row and head of another
        one[5, 2] = good[6, 2]
        dim = good.clone()  # two neighbouring dims in each other's place
        dim[..., 0], dim[..., 1] = good[..., 1], good[..., 0]
        late, _, _ = O.sdpa_varlen(q, k, v, [[0, 3, 0, 189], [3, 20, 1, 127], [23, 1, 0, 30]], True, window, scale, None, None)
        near = S.to_bf16(ref * (1 + 2.0 ** -5))
        for bad in (torch.zeros_like(good), flipped, swapped, one, dim, S.to_bf16(late), near):
            with pytest.raises(AssertionError):
                B.hold(bad, *args)


def test_a_bound_that_holds_nothing_is_refused():
    store = random_store(32, 1, 1, 64, 1, 29, 30)  # scores in the hundred thousands
    with pytest.raises(AssertionError, match="hold nothing"):
        B.bound(queries(2, 1, 64, 1), store, [[0, 2, 0, 30]], True)


def test_rows_without_a_segment():
    store, q = random_store(32, 1, 1, 64, 1, 10, 12), queries(4, 1, 64, 1)
    ref, _, seg = B.bound(q, store, [[1, 2, 0, 2]], True)
    assert seg.tolist() == [-1, 0, 0, -1] and not ref[[0, 3]].any() and ref[1:3].any()
    assert np.abs(ref).max() < 1
