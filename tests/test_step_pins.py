"""Pins of the oracle's rotary positions and 4-bit store on facts of their own (CPU)."""
import math

import numpy as np
import pytest
import torch

from oracle import step_oracle as S


def _table(P, half, seed=0):
    a = np.random.default_rng(seed).uniform(-math.pi, math.pi, size=(P, half))
    return torch.from_numpy(np.stack([np.cos(a), np.sin(a)], -1)).float()


@pytest.mark.parametrize("interleaved", [False, True])
def test_rotation_keeps_lengths_and_its_inverse_undoes_it(interleaved):
    x = torch.randn(5, 3, 64, generator=torch.Generator().manual_seed(1)).to(torch.bfloat16)
    pos = np.array([[0, 3, 7, 2, 9], [1, 1, 8, 0, 4]])
    y, bad = S.rope(x, _table(10, 24), pos, (10, 14), interleaved)
    assert not bad.any()
    np.testing.assert_allclose(np.linalg.norm(y, axis=-1), np.linalg.norm(S.f64(x), axis=-1), rtol=1e-6)
    np.testing.assert_array_equal(y[..., 48:], S.f64(x)[..., 48:])
    back, _ = S.rope(y, _table(10, 24), pos, (10, 14), interleaved, inverse=True)
    np.testing.assert_allclose(back, S.f64(x), atol=1e-6)  # fp32 cos^2 + sin^2 is 1 to 2^-23


def test_rotated_products_depend_on_the_distance_alone():
    # with cos / sin of position * frequency, <R_p q, R_r k> is a function of p - r
    half = 16
    freq = 10000.0 ** (-np.arange(half) / half)
    a = np.arange(200)[:, None] * freq
    tab = np.stack([np.cos(a), np.sin(a)], -1)
    g = np.random.default_rng(2)
    q, k = g.normal(size=(1, 1, 64)), g.normal(size=(1, 1, 64))
    dots = []
    for shift in (0, 5, 90):
        qr, _ = S.rope(q, tab, [[37 + shift]], (half,))
        kr, _ = S.rope(k, tab, [[12 + shift]], (half,))
        dots.append(float((qr * kr).sum()))
    np.testing.assert_allclose(dots, dots[0], rtol=1e-10)


def test_rotation_by_complex_multiplication():
    x = np.random.default_rng(3).normal(size=(2, 1, 64))
    tab = _table(4, 32, 5).double().numpy()
    y, _ = S.rope(x, tab, [[3, 1]], (32,), interleaved=True)
    z = (x[..., 0::2] + 1j * x[..., 1::2]) * (tab[[3, 1], :, 0] + 1j * tab[[3, 1], :, 1])[:, None]
    np.testing.assert_allclose(y[..., 0::2], z.real, atol=1e-12)
    np.testing.assert_allclose(y[..., 1::2], z.imag, atol=1e-12)


def test_rows_outside_the_table_are_marked_and_zero_and_an_empty_axis_is_not_looked_at():
    x = np.ones((3, 1, 64))
    y, bad = S.rope(x, _table(4, 8), [[0, 4, -1], [99, 99, 99]], (8, 0))
    assert bad.tolist() == [False, True, True] and not y[1:].any() and y[0].any()


def test_every_byte_has_the_value_the_format_says():
    s = S.scale_of(np.arange(256))
    assert (np.diff(s) > 0).all() and s[0] == 2.0 ** -21 and s[255] == 1920.0
    codes = np.arange(256, dtype=np.uint8).reshape(8, 32)[:, :32]
    v = S.q4_unpack(codes, np.full((8, 2), 21 * 8, dtype=np.uint8))  # scale 1
    assert v[0, 0] == -8 and v[0, 1] == -8 and v[0, 2] == -7 and v[0, 3] == -8 and v[7, 63] == 7 and v[7, 62] == 7
    # exact in bf16 and in fp16
    every = (np.arange(16) - 8)[:, None] * s[None]
    t = torch.from_numpy(every)
    assert torch.equal(t.float().to(torch.bfloat16).double(), t)
    assert torch.equal(t.to(torch.float16).double(), t)


def test_packing_is_nearest_idempotent_and_within_half_a_step():
    g = torch.Generator().manual_seed(4)
    x = (torch.randn(200, 128, generator=g) * torch.exp(1.5 * torch.randn(200, 1, generator=g))).to(torch.bfloat16)
    c, b = S.q4_pack(x)
    v = S.q4_unpack(c, b)
    step = np.repeat(S.scale_of(b), 32, axis=-1)
    assert (np.abs(v - S.f64(x)) <= step / 2).all()
    assert (np.abs(v).max(-1) > 0).all()
    c2, b2 = S.q4_pack(S.to_bf16(v))  # what is stored stores as itself where a 7 is in the group
    again = S.q4_unpack(c2, b2)
    full = np.repeat((np.abs(v).reshape(200, 4, 32).max(-1) == 7 * S.scale_of(b)), 32, axis=-1)
    assert full.mean() > 0.5
    np.testing.assert_array_equal(again[full], v[full])


def test_packing_at_borders_and_extremes():
    x = torch.zeros(6, 32)
    x[0, 0] = 7.0                                  # scale 1: halves go to even
    x[0, 1:5] = torch.tensor([0.5, 1.5, -0.5, 2.5])
    x[2] = 1e9                                     # saturates
    x[3, 0], x[3, 1] = float("inf"), 2.0
    x[4, 0], x[4, 1] = float("nan"), 7.0
    x[5] = 1e-20                                   # below half the smallest step
    c, b = S.q4_pack(x.to(torch.bfloat16))
    v = S.q4_unpack(c, b)
    assert v[0, :5].tolist() == [7.0, 0.0, 2.0, 0.0, 2.0]
    assert not v[1].any() and b[1, 0] == 0
    assert (v[2] == 13440.0).all()
    assert v[3, 0] == 13440.0 and v[3, 1] == 0.0
    assert v[4, 0] == 0.0 and v[4, 1] == 7.0
    assert not v[5].any()


def test_a_tie_between_two_scales_goes_to_the_even_byte():
    x = torch.zeros(1, 32)
    x[0, 0] = 7 * (1 + 1 / 16)  # a seventh of it halfway between scale 1 (byte 168) and 9/8 (byte 169)
    _, b = S.q4_pack(x.to(torch.bfloat16))
    assert b[0, 0] == 168
    x[0, 0] = 7 * (1 + 3 / 16)  # between 9/8 (169) and 10/8 (170)
    _, b = S.q4_pack(x.to(torch.bfloat16))
    assert b[0, 0] == 170
    # 1/7 in 32 bits is 4.2e-8 too large, relatively: beyond half a step of 32 bits above a product of
    # about 1.43, which then lies above the border
    x[0, 0] = 7 * (1 + 9 / 16)  # between 12/8 (172) and 13/8 (173)
    _, b = S.q4_pack(x.to(torch.bfloat16))
    assert b[0, 0] == 173


def test_append_places_rows_as_the_plain_append_does():
    from oracle import sdpa_varlen_oracle as O

    g = torch.Generator().manual_seed(6)
    q, k, v = (torch.randn(9, h, 64, generator=g).to(torch.bfloat16) for h in (2, 1, 1))
    seq = np.array([[0, 3, 1, 20], [4, 2, 0, 1], [6, 2, 9, 5]])  # the second begins before position 0
    flat = torch.tensor([1.0, 0.0]).expand(64, 32, 2).contiguous()  # no turn at all
    qr, kb, wrote, st = S.rope_append(q, k, v, 16, 3, seq, 8, flat, (32,))
    store = torch.zeros(16, 3, 1, 64, dtype=torch.bfloat16)
    ks, _ = O.kv_append(store, store, k, v, seq, 8)
    mine = store.clone()
    for t, row, col in wrote:
        mine[row, col] = kb[t]
    assert torch.equal(mine, ks) and st == O.SEG_BAD_COL
    assert [w[0] for w in wrote] == [0, 1, 2, 5]
    assert not qr[[3, 4, 6, 7, 8]].any() and np.array_equal(qr[0], S.f64(q)[0])
