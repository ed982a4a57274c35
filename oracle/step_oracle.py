"""Plain 64-bit statements of the rotary positions, the rotated append and the 4-bit column store.

Written from the definitions with NumPy (torch only carries bf16 tensors), element by element where
that is affordable; nothing here is shared with the library.
"""

from __future__ import annotations

import numpy as np
import torch

from . import sdpa_varlen_oracle as O

BAD_POS = 64
GROUP = 32


def f64(t) -> np.ndarray:
    return t.detach().cpu().double().numpy() if isinstance(t, torch.Tensor) else np.asarray(t, dtype=np.float64)


def to_bf16(x: np.ndarray) -> torch.Tensor:
    """Rounded to fp32, then to bf16 (halves to even both times)."""
    return torch.from_numpy(np.ascontiguousarray(x)).float().to(torch.bfloat16)


def pair_axis(sections) -> np.ndarray:
    """Axis of every pair."""
    return np.concatenate([np.full(n, a) for a, n in enumerate(sections)]).astype(np.int64)


def pair_dims(j: int, half: int, interleaved: bool):
    return (2 * j, 2 * j + 1) if interleaved else (j, j + half)


def rope(x, table, positions, sections, interleaved=False, inverse=False):
    """x [T, H, D], table [P, half, 2], positions [axes, T] -> ([T, H, D] in 64 bits, rows whose
    position is outside the table [T]).  Such rows are 0."""
    y = f64(x).copy()
    tab = f64(table)
    pos = np.asarray(positions, dtype=np.int64).reshape(len(sections), y.shape[0])
    P, half = tab.shape[0], tab.shape[1]
    axis = pair_axis(sections)
    used = sorted(set(axis.tolist()))
    bad = np.zeros(y.shape[0], dtype=bool)
    for a in used:
        bad |= (pos[a] < 0) | (pos[a] >= P)
    at = np.where(bad[None], 0, pos)
    for j in range(half):
        u, w = pair_dims(j, half, interleaved)
        c = tab[at[axis[j]], j, 0][:, None]
        s = tab[at[axis[j]], j, 1][:, None] * (-1.0 if inverse else 1.0)
        a, b = y[..., u].copy(), y[..., w].copy()
        y[..., u] = a * c - b * s
        y[..., w] = a * s + b * c
    y[bad] = 0.0
    return y, bad


def scale_of(b) -> np.ndarray:
    b = np.asarray(b, dtype=np.int64)
    return 2.0 ** ((b >> 3) - 21) * (1.0 + (b & 7) / 8.0)


def q4_unpack(codes, scales) -> np.ndarray:
    """[..., D / 2] and [..., D / 32] bytes -> [..., D] in 64 bits."""
    c = np.asarray(codes, dtype=np.int64)
    n = np.empty(c.shape[:-1] + (2 * c.shape[-1],), dtype=np.float64)
    n[..., 0::2] = (c & 15) - 8
    n[..., 1::2] = (c >> 4) - 8
    return n * np.repeat(scale_of(scales), GROUP, axis=-1)


def q4_pack(x):
    """bf16 [..., D] -> (codes [..., D / 2], scales [..., D / 32]) uint8.  The nearest of the 256
    scales to max|x| times 1/7, a product of 32 bits (the even byte where two are as near), then the nearest
    code in [-7, 7]."""
    v = f64(x)
    v = np.where(np.isnan(v), 0.0, v)
    g = v.reshape(v.shape[:-1] + (-1, GROUP))
    want = (np.abs(g).max(-1).astype(np.float32) * np.float32(1 / 7)).astype(np.float64)
    every = scale_of(np.arange(256))
    off = np.abs(every - np.minimum(want, 1e6)[..., None])
    near = off.min(-1, keepdims=True)
    even_first = np.argsort(np.arange(256) % 2, kind="stable")
    b = even_first[np.argmax((off <= near)[..., even_first], axis=-1)]
    s = scale_of(b)[..., None]
    n = np.clip(np.rint(g / s), -7, 7).reshape(v.shape).astype(np.int64) + 8
    return (n[..., 0::2] | (n[..., 1::2] << 4)).astype(np.uint8), b.astype(np.uint8)


def column_store(codes, scales) -> torch.Tensor:
    """A 4-bit store's values laid out as the bf16 column store [rows, cols, Hkv, D] (64 bits)."""
    return torch.from_numpy(np.ascontiguousarray(q4_unpack(codes, scales).transpose(2, 0, 1, 3)))


def step_rows(seq_info, T, rows, cols, window, seg_mode=None):
    """(segment of each packed row or -1, its position, its column, status bits)."""
    seg_id, _, _, status = O.visible_interval(seq_info, T, True, window, rows, cols,
                                              None if seg_mode is None else seg_mode)
    seq = np.asarray(seq_info, dtype=np.int64).reshape(-1, 4)
    live = np.where(seg_id >= 0, seg_id, -1)
    pos = np.full(T, -1, dtype=np.int64)
    col = np.zeros(T, dtype=np.int64)
    for t in range(T):
        if live[t] >= 0:
            qs, ql, c, kv = seq[live[t]]
            pos[t], col[t] = kv - ql + (t - qs), c
    return live, pos, col, status


def rope_append(q, k_new, v_new, rows, cols, seq_info, window, table, sections, positions=None, interleaved=False,
                seg_mode=None):
    """(q_out [T, Hq, D] in 64 bits, keys bf16 [T, Hkv, D], packed rows written [(t, row, col)], status)."""
    T = q.shape[0]
    live, pos, col, status = step_rows(seq_info, T, rows, cols, window, seg_mode)
    stays = (live >= 0) & (pos >= 0)
    at = np.where(stays, pos, 0)[None] if positions is None else np.asarray(positions).reshape(len(sections), T)
    at = np.where(stays[None], at, 0)  # a row that is not there is not looked up
    qr, bad = rope(q, table, at, sections, interleaved)
    kr, _ = rope(k_new, table, at, sections, interleaved)
    bad = bad & stays
    if bad.any():
        status |= BAD_POS
    keep = stays & ~bad
    qr[~keep] = 0.0
    return qr, to_bf16(kr), [(t, int(pos[t] % rows), int(col[t])) for t in range(T) if keep[t]], status
