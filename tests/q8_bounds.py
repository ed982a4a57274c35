"""How far an 8-bit attention's output may be from the 64-bit one, row by row.

A score is a sum of D products in fp32: it is off by at most (D + 4) 2^-23 of sum_d |q_d k_d| scale (the 4: its scale,
rounded, and the exponent's sum), and exp2 with its argument's constant part by 2^-20.  A row's largest such sum over
the keys that it sees gives d; a probability over its row's sum is then off by 2 d of itself, by fp16's 2^-11, by 2^-23
for every key summed, and where it is below fp16's smallest step by 2^-32 of the sum.  The output is rounded to bf16 (2^-8).
d has to be small for the rest to follow, which is checked: a bound that any output meets checks nothing."""
import numpy as np

from oracle import sdpa_varlen_oracle as O
from oracle import step_oracle as S

MOST = 1 / 32  # of 2 d


def stores(store):
    return tuple(S.q8_column_store(np.asarray(c), np.asarray(b)).numpy()
                 for c, b in ((store.k_codes, store.k_scales), (store.v_codes, store.v_scales)))


def score_error(q, k, seq, causal, window, scale, modes=None):
    """d of each (row, head), the largest |v| of those that see v, and keys seen."""
    q = S.f64(q)
    T, Hq, D = q.shape
    rows, cols, Hkv, _ = k.shape
    seg, lo, hi, _ = O.visible_interval(seq, T, causal, window, rows, cols, modes)
    d = np.zeros((T, Hq))
    for t in range(T):
        if seg[t] < 0 or hi[t] <= lo[t]:
            continue
        seen = k[np.arange(lo[t], hi[t]) % rows, np.asarray(seq)[seg[t]][2]]  # [n, Hkv, D]
        per = np.einsum("hgd,nhd->hgn", np.abs(q[t]).reshape(Hkv, -1, D), np.abs(seen)).max(-1).reshape(Hq)
        d[t] = (D + 4) * 2.0 ** -23 * scale * per + 2.0 ** -20
    return d, np.maximum(hi - lo, 0), seg


def bound(q, store, seq, causal, window=0, scale=None, modes=None):
    """(64-bit outputs, how far off each may be, each row's segment)."""
    k, v = stores(store)
    scale = q.shape[2] ** -0.5 if scale is None else scale
    ref, _, _ = O.sdpa_varlen(q, k, v, seq, causal, window, scale, None, modes)
    mag, _, _ = O.sdpa_varlen(q, k, np.abs(v), seq, causal, window, scale, None, modes)
    d, n, seg = score_error(q, k, seq, causal, window, scale, modes)
    assert 2 * d.max() <= MOST, f"scores off by {d.max()}: the bound would hold nothing"
    rows = v.shape[0]
    _, lo, hi, _ = O.visible_interval(seq, q.shape[0], causal, window, rows, v.shape[1], modes)
    top = np.zeros(ref.shape)
    for t in np.flatnonzero((seg >= 0) & (hi > lo)):
        seen = np.abs(v[np.arange(lo[t], hi[t]) % rows, np.asarray(seq)[seg[t]][2]]).max(0)  # [Hkv, D]
        top[t] = np.repeat(seen, q.shape[1] // v.shape[2], axis=0)
    n = n[:, None, None]
    off = 2.0 ** -8 * np.abs(ref) + (2.0 ** -11 + 2 * d[..., None] + n * 2.0 ** -23) * mag + 2.0 ** -32 * n * top + 1e-30
    return ref, off, seg


def hold(got, *args, tag="", **kw):
    """Whether an output is within the bound; rows of no segment have to be 0."""
    ref, off, seg = bound(*args, **kw)
    g = S.f64(got)
    assert np.isfinite(g).all(), f"{tag}: not finite"
    wrong = np.abs(g - ref) > off
    assert not wrong[seg >= 0].any(), f"{tag}: {np.argwhere(wrong)[:3]}, {np.abs(g - ref)[wrong][:3]} of {off[wrong][:3]}"
    assert not g[seg == O.UNCOVERED].any(), tag
