"""GPU parity of the rotary positions (sdpa_rope) against the 64-bit oracle.

A result is r = fma(a, cos, q), q = -(b sin), rounded to bf16.  q is off by 2^-24 of itself, r by 2^-24 of
itself, both at most |a| + |b| (cosines are at most 1), and the rounding to bf16 by 2^-8 of r: all in
all 2^-8 of the result and (1 + 2^-8) 2^-23, less than 2^-22, of the pair."""
import numpy as np
import pytest
import torch

import varlen_gqa_attention_gb300 as pkg
from oracle import step_oracle as S

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    torch.cuda.set_device(0)
    return torch.device("cuda:0")


def inputs(T, H, D, R, axes, P, seed):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(T, H, D, generator=g).to(torch.bfloat16)
    table = pkg.rope_table(P, R)
    pos = torch.randint(0, P, (axes, T), generator=g, dtype=torch.int32)
    half = R // 2
    cuts = sorted(torch.randint(0, half + 1, (axes - 1,), generator=g).tolist())
    return x, table, pos, tuple(b - a for a, b in zip([0] + cuts, cuts + [half]))


def assert_rotated(got, ref, x, R, interleaved, tag=""):
    pair = np.abs(S.f64(x)).copy()
    half = R // 2
    for j in range(half):
        u, w = S.pair_dims(j, half, interleaved)
        pair[..., u] = pair[..., w] = pair[..., u] + pair[..., w]
    err = np.abs(S.f64(got) - ref)
    bound = 2.0 ** -8 * np.abs(ref) + 2.0 ** -22 * pair
    assert (err <= bound).all(), f"{tag}: {np.argwhere(err > bound)[:3]}"
    assert np.array_equal(S.f64(got)[..., R:], ref[..., R:])  # the dims that are not turned


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("R,axes", [(16, 1), (48, 2), (64, 3), (64, 4)])
@pytest.mark.parametrize("T,H", [(1, 1), (3, 17), (130, 5)])
def test_rotation_matches_the_oracle(dev, D, interleaved, R, axes, T, H):
    R = D if R == 64 and axes == 3 else R
    x, table, pos, sections = inputs(T, H, D, R, axes, 1000, D + 7 * T + axes)
    ref, _ = S.rope(x, table, pos, sections, interleaved)
    got = pkg.sdpa_rope(x.to(dev), table.to(dev), pos.to(dev), sections=sections, interleaved=interleaved)
    assert_rotated(got, ref, x, R, interleaved)


@pytest.mark.parametrize("interleaved", [False, True])
def test_the_inverse_is_the_gradient(dev, interleaved):
    T, H, D, R = 33, 4, 128, 96
    x, table, pos, sections = inputs(T, H, D, R, 3, 5000, 3)
    w, _, _, _ = inputs(T, H, D, R, 3, 5000, 4)
    tab, p = table.to(dev), pos.to(dev)
    kw = dict(sections=sections, interleaved=interleaved)
    got = pkg.sdpa_rope(w.to(dev), tab, p, inverse=True, **kw)
    # the formula: the transpose of the rotation, applied to the output's gradient
    ref, _ = S.rope(w, table, pos, sections, interleaved, inverse=True)
    assert_rotated(got, ref, w, R, interleaved)
    # differences of f(x) = <w, rope(x)> along d: rope is linear, so they are exact but for the
    # rounding of the four tensors involved, each at most 2^-8 of its values
    d = torch.randn(T, H, D, generator=torch.Generator().manual_seed(5)).to(torch.bfloat16)
    up, down = (x.float() + d.float()).to(torch.bfloat16), (x.float() - d.float()).to(torch.bfloat16)
    f = [S.f64(pkg.sdpa_rope(v.to(dev), tab, p, **kw)) for v in (up, down)]
    step = S.f64(up) - S.f64(down)
    diff = (S.f64(w) * (f[0] - f[1])).sum()
    slope = (S.f64(got) * step).sum()
    bound = 2.0 ** -8 * ((np.abs(S.f64(w)) * (np.abs(f[0]) + np.abs(f[1]))).sum() + np.abs(S.f64(got) * step).sum())
    assert abs(diff - slope) <= bound


def test_in_place_and_strided_rows(dev):
    x, table, pos, sections = inputs(40, 6, 128, 128, 1, 300, 8)
    ref = S.rope(x, table, pos, sections)[0]
    y = x.to(dev)
    assert pkg.sdpa_rope(y, table.to(dev), pos[0].to(dev), out=y) is y
    assert_rotated(y, ref, x, 128, False)
    wide = torch.full((40, 10, 136), 7.0, dtype=torch.bfloat16, device=dev)
    part = wide[:, 2:8, 8:]
    part.copy_(x)
    out = torch.full((40, 20, 128), 5.0, dtype=torch.bfloat16, device=dev)
    pkg.sdpa_rope(part, table.to(dev), pos.to(dev), out=out[:, ::2][:, 1:7])
    assert torch.equal(out[:, 2:14:2], y)
    assert bool((out[:, 1::2] == 5).all()) and bool((out[:, 14:] == 5).all()) and bool((out[:, 0] == 5).all())
    assert bool((wide[:, :2] == 7).all()) and torch.equal(part.cpu(), x)


def test_positions_outside_the_table_are_reported_and_zero(dev):
    x, table, pos, sections = inputs(9, 5, 64, 32, 2, 50, 9)
    sections = (10, 6)
    pos[0, 2], pos[1, 5], pos[0, 7] = 50, -1, 2 ** 31 - 1
    status = torch.zeros(1, dtype=torch.int32, device=dev)
    got = pkg.sdpa_rope(x.to(dev), table.to(dev), pos.to(dev), sections=sections, status=status)
    ref, bad = S.rope(x, table, pos, sections)
    assert bad.nonzero()[0].tolist() == [2, 5, 7] and int(status) == pkg.ROPE_BAD_POS
    assert_rotated(got, ref, x, 32, False)
    assert not bool(got[[2, 5, 7]].any())
    status.zero_()  # an axis without pairs is not looked at
    pkg.sdpa_rope(x.to(dev), table.to(dev), pos[[0, 1]].clamp(0, 49).to(dev) * torch.tensor([[1], [1000]], device=dev,
                  dtype=torch.int32), sections=(16, 0), status=status)
    assert int(status) == 0


def test_infinities_and_nan_stay_in_their_pair(dev):
    x, table, pos, sections = inputs(2, 2, 64, 64, 1, 100, 10)
    x[0, 0, 3], x[1, 1, 40] = float("inf"), float("nan")
    got = S.f64(pkg.sdpa_rope(x.to(dev), table.to(dev), pos.to(dev)))
    assert np.isinf(got[0, 0, [3, 35]]).all() and np.isnan(got[1, 1, [8, 40]]).all()
    assert np.isfinite(got).sum() == got.size - 4


def test_no_rows_another_stream_and_a_captured_graph(dev):
    x, table, pos, sections = inputs(20, 3, 128, 64, 1, 64, 11)
    tab, p = table.to(dev), pos.to(dev)
    assert pkg.sdpa_rope(x[:0].to(dev), tab, p[:, :0]).shape == (0, 3, 128)
    ref = S.rope(x, table, pos, sections)[0]
    side = torch.cuda.Stream(dev)
    xd = x.to(dev)
    side.wait_stream(torch.cuda.current_stream())
    y = pkg.sdpa_rope(xd, tab, p, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert_rotated(y, ref, x, 64, False)
    out = torch.empty_like(xd)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        pkg.sdpa_rope(xd, tab, p, out=out)
    x2, _, pos2, _ = inputs(20, 3, 128, 64, 1, 64, 12)
    xd.copy_(x2)
    p.copy_(pos2)
    g.replay()
    torch.cuda.synchronize()
    assert_rotated(out, S.rope(x2, table, pos2, sections)[0], x2, 64, False)


def test_many_rows_on_few_warps(dev):
    # more rows than the launch has warps: each goes through several, the positions of some outside
    x, table, pos, _ = inputs(9000, 3, 64, 64, 2, 300, 14)
    sections = (20, 12)
    pos[0, ::1000], pos[1, 17::3000] = -5, 300
    status = torch.zeros(1, dtype=torch.int32, device=dev)
    got = pkg.sdpa_rope(x.to(dev), table.to(dev), pos.to(dev), sections=sections, status=status)
    ref, bad = S.rope(x, table, pos, sections)
    assert_rotated(got, ref, x, 64, False)
    assert int(status) == pkg.ROPE_BAD_POS and not bool(got[torch.from_numpy(bad).to(dev)].any())
