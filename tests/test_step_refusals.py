"""Arguments that the rotary and 4-bit entries refuse, all of them before any CUDA call (the pointers of
the C calls are fake and never dereferenced)."""
import pytest
import torch

import varlen_gqa_attention_gb300 as pkg

FAKE = 0x10000
NULL, SHAPE, HEAD_DIM, GQA, STRIDE, ALIGN, WORKSPACE, ARG = 1, 2, 3, 4, 5, 6, 7, 8


def codes():
    """The error codes by name, as the header has them."""
    import os
    import re

    text = open(os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include",
                             "sdpa_varlen.h")).read()
    return {n: int(v) for n, v in re.findall(r"SDPA_ERR_([A-Z_]+) = (\d+)", text)}


def test_the_codes_are_the_headers():
    c = codes()
    assert [c[n] for n in ("NULL", "SHAPE", "HEAD_DIM", "GQA", "STRIDE", "ALIGN", "WORKSPACE", "ARG")] == \
        [NULL, SHAPE, HEAD_DIM, GQA, STRIDE, ALIGN, WORKSPACE, ARG]


def rotation(table=FAKE, table_rows=100, positions=FAKE, pos_stride=8, rot_dims=64, axes=1, sections=(32, 0, 0, 0),
             interleaved=0):
    return pkg._ROTATION.pack(table, table_rows, positions, pos_stride, rot_dims, axes, *sections, interleaved)


def store(**kw):
    a = dict(k_codes=FAKE, k_scales=FAKE, v_codes=FAKE, v_scales=FAKE)
    a.update(kw)
    return pkg._Q4_POINTERS.pack(*a.values())


BAD_ROTATIONS = [
    (rotation(table=0), NULL), (rotation(table=FAKE + 8), ALIGN), (rotation(table_rows=0), SHAPE),
    (rotation(table_rows=-1), SHAPE), (rotation(table_rows=1 << 31), SHAPE),
    (rotation(table_rows=(1 << 31) // 32), SHAPE),  # its pairs pass 31 bits
    (rotation(rot_dims=0, sections=(0,) * 4), ARG), (rotation(rot_dims=8, sections=(4, 0, 0, 0)), ARG),
    (rotation(rot_dims=80, sections=(40, 0, 0, 0)), ARG), (rotation(rot_dims=40, sections=(20, 0, 0, 0)), ARG),
    (rotation(axes=0), ARG), (rotation(axes=5), ARG), (rotation(sections=(31, 0, 0, 0)), ARG),
    (rotation(axes=3, sections=(30, 2, 1, 0)), ARG), (rotation(axes=3, sections=(40, -8, 0, 0)), ARG),
    (rotation(axes=2, sections=(2 ** 31 - 1, 2 ** 31 - 1, 0, 0)), ARG),
    (rotation(positions=FAKE + 2), ALIGN), (rotation(axes=2, sections=(16, 16, 0, 0), pos_stride=-1), STRIDE),
    (rotation(axes=2, sections=(16, 16, 0, 0), positions=0), NULL), (None, NULL),
]


def rope(**kw):
    a = dict(x=FAKE, T=8, H=4, D=64, x_rs=256, x_hs=64, rot=rotation(), inverse=0, out=FAKE, o_rs=256, o_hs=64,
             status=None, stream=None)
    a.update(kw)
    return pkg.library().sdpa_rope(*a.values())


@pytest.mark.parametrize("kw,code", [
    (dict(x=None), NULL), (dict(out=None), NULL), (dict(T=-1), SHAPE), (dict(T=1 << 31), SHAPE), (dict(H=0), SHAPE),
    (dict(H=(1 << 20) + 1), SHAPE), (dict(D=96), HEAD_DIM), (dict(D=0), HEAD_DIM), (dict(x=FAKE + 2), ALIGN),
    (dict(out=FAKE + 8), ALIGN), (dict(x_rs=250), STRIDE), (dict(x_hs=-64), STRIDE), (dict(o_rs=-8), STRIDE),
    (dict(o_hs=3), STRIDE), (dict(rot=rotation(positions=0)), NULL),
] + [(dict(rot=r), c) for r, c in BAD_ROTATIONS])
def test_rope(kw, code):
    assert rope(**kw) == code
    assert pkg.library().sdpa_last_error()


def append(fourbit, **kw):
    a = dict(q=FAKE, q_rs=256, q_hs=64, k=FAKE, k_rs=128, k_hs=64, v=FAKE, v_rs=128, v_hs=64, T=8, Hq=4, Hkv=2, D=64,
             rot=rotation())
    a.update(dict(store=store()) if fourbit else dict(k_store=FAKE, v_store=FAKE))
    a.update(rows=32, cols=2, seq=FAKE, mode=None, S=1, window=0, q_out=FAKE, o_rs=256, o_hs=64, status=None,
             stream=None)
    assert set(kw) <= set(a)
    a.update(kw)
    lib = pkg.library()
    return (lib.sdpa_rope_append_fourbit if fourbit else lib.sdpa_rope_append)(*a.values())


@pytest.mark.parametrize("fourbit", [False, True])
@pytest.mark.parametrize("kw,code", [
    (dict(q=None), NULL), (dict(k=None), NULL), (dict(v=None), NULL), (dict(q_out=None), NULL), (dict(seq=None), NULL),
    (dict(T=-1), SHAPE), (dict(T=1 << 31), SHAPE), (dict(S=-1), SHAPE), (dict(Hq=0), SHAPE), (dict(rows=0), SHAPE),
    (dict(cols=0), SHAPE), (dict(rows=1 << 31), SHAPE), (dict(Hq=1 << 20, Hkv=1 << 19), SHAPE),
    (dict(D=80), HEAD_DIM), (dict(Hq=3), GQA), (dict(Hq=258), GQA), (dict(window=-1), ARG),
    (dict(seq=FAKE + 4), ALIGN), (dict(mode=FAKE + 8), ALIGN), (dict(q=FAKE + 2), ALIGN), (dict(k=FAKE + 2), ALIGN),
    (dict(v=FAKE + 8), ALIGN), (dict(q_out=FAKE + 4), ALIGN), (dict(q_rs=-8), STRIDE), (dict(k_rs=4), STRIDE),
    (dict(k_hs=65), STRIDE), (dict(v_rs=-8), STRIDE), (dict(v_hs=1), STRIDE), (dict(o_hs=12), STRIDE),
] + [(dict(rot=r), c) for r, c in BAD_ROTATIONS])
def test_rope_append(fourbit, kw, code):
    assert append(fourbit, **kw) == code


@pytest.mark.parametrize("kw,code", [(dict(k_store=None), NULL), (dict(v_store=None), NULL),
                                     (dict(k_store=FAKE + 2), ALIGN), (dict(v_store=FAKE + 8), ALIGN)])
def test_bf16_stores(kw, code):
    assert append(False, **kw) == code


BAD_STORES = [(dict(store=None), NULL), (dict(rows=24), SHAPE), (dict(rows=8), SHAPE)] + \
    [(dict(store=store(**{n: p})), c) for n in ("k_codes", "k_scales", "v_codes", "v_scales")
     for p, c in ((0, NULL), (FAKE + 8, ALIGN))]


@pytest.mark.parametrize("kw,code", BAD_STORES)
def test_fourbit_stores(kw, code):
    assert append(True, **kw) == code
    assert unpack(**kw) == code
    assert attend(**kw) == code


def unpack(**kw):
    a = dict(store=store(), rows=32, cols=2, Hkv=2, D=64, seq=FAKE, mode=None, S=1, window=0, T=8, k_out=FAKE,
             v_out=FAKE, o_rs=128, o_hs=64, status=None, stream=None)
    assert set(kw) <= set(a)
    a.update(kw)
    return pkg.library().sdpa_fourbit_unpack(*a.values())


@pytest.mark.parametrize("kw,code", [
    (dict(k_out=None), NULL), (dict(v_out=None), NULL), (dict(seq=None), NULL), (dict(T=-1), SHAPE),
    (dict(Hkv=0), SHAPE), (dict(cols=-1), SHAPE), (dict(Hkv=1 << 20), SHAPE), (dict(D=32), HEAD_DIM),
    (dict(window=-2), ARG), (dict(seq=FAKE + 8), ALIGN), (dict(mode=FAKE + 4), ALIGN), (dict(k_out=FAKE + 2), ALIGN),
    (dict(v_out=FAKE + 2), ALIGN), (dict(o_rs=-8), STRIDE), (dict(o_hs=20), STRIDE),
])
def test_unpack(kw, code):
    assert unpack(**kw) == code


def attend(**kw):
    a = dict(q=FAKE, T=8, Hq=4, D=64, q_rs=256, q_hs=64, store=store(), rows=32, cols=2, Hkv=2, seq=FAKE, mode=None,
             S=1, causal=1, window=0, scale=0.125, out=FAKE, o_rs=256, o_hs=64, ws=FAKE, ws_bytes=1 << 30,
             status=None, stream=None)
    assert set(kw) <= set(a)
    a.update(kw)
    return pkg.library().sdpa_varlen_fourbit(*a.values())


@pytest.mark.parametrize("kw,code", [
    (dict(q=None), NULL), (dict(out=None), NULL), (dict(seq=None), NULL), (dict(ws=None), WORKSPACE),
    (dict(T=-1), SHAPE), (dict(rows=1 << 31), SHAPE), (dict(S=-1), SHAPE), (dict(D=112), HEAD_DIM), (dict(Hq=5), GQA),
    (dict(Hq=258), GQA), (dict(window=-1), ARG), (dict(scale=float("inf")), ARG), (dict(scale=float("nan")), ARG),
    (dict(scale=-0.125), ARG), (dict(q=FAKE + 2), ALIGN), (dict(out=FAKE + 8), ALIGN), (dict(seq=FAKE + 4), ALIGN),
    (dict(mode=FAKE + 8), ALIGN), (dict(ws=FAKE + 16), ALIGN), (dict(q_rs=-8), STRIDE), (dict(q_hs=60), STRIDE),
    (dict(o_rs=12), STRIDE), (dict(o_hs=-64), STRIDE),
])
def test_attend(kw, code):
    assert attend(**kw) == code


@pytest.mark.parametrize("D", [64, 128, 256])
def test_a_workspace_for_bounds_serves_every_smaller_call(D):
    need = pkg.library().sdpa_varlen_fourbit_workspace_bytes
    pkg.set_route_policy(pkg.ROUTE_SPLITK)  # without staged columns, of which a call takes what it is given
    try:
        for Hq, Hkv in ((8, 8), (32, 8), (16, 1), (256, 2)):
            for T in (1, 16, 64, 257, 2048):
                for S_ in (0, 1, 7, 64, 500):
                    bound = need(T, Hq, Hkv, D, S_, 4096, 64)
                    for t in (0, 1, 3, 40, 200, T):
                        for s in (0, 1, 6, 63, S_):
                            if t <= T and s <= S_:
                                assert need(t, Hq, Hkv, D, s, 4096, 64) <= bound, (Hq, Hkv, T, S_, t, s)
    finally:
        pkg.set_route_policy(pkg.ROUTE_AUTO)
    assert need(1, 3, 2, D, 1, 64, 1) == 0 and need(1, 2, 2, 96, 1, 64, 1) == 0 and need(1, 2, 2, D, 1, 1 << 31, 1) == 0


def test_staged_columns_follow_the_longest_segment():
    need = pkg.library().sdpa_varlen_fourbit_workspace_bytes
    col = 2 * 32768 * 8 * 128 * 2  # K and V of one column in bf16

    def staged(T, S_, D=128):
        pkg.set_route_policy(pkg.ROUTE_SPLITK)
        plain = need(T, 32, 8, D, S_, 32768, 64)
        pkg.set_route_policy(pkg.ROUTE_AUTO)
        return (need(T, 32, 8, D, S_, 32768, 64) - plain) / col

    assert staged(64, 64) == 0               # single tokens
    assert staged(94, 64) == 0               # a segment of 31 rows among them (124 packed)
    assert staged(95, 64) == 2               # of 32: the rows that fill a tile, twice over
    assert staged(64 + 300, 64) == 2         # more than 16 packed rows on average: 512 of a segment
    assert staged(15 + 127, 16) == 0 and staged(15 + 128, 16) == 1
    assert staged(256, 1) == 1 and staged(255, 1) == 0
    assert staged(8192, 4) == 4 and staged(1 << 16, 64) == 16  # of all, and of 2 GiB of them


# ------------------------------------------------------------------------------- the Python entries

bf, f32, i32, u8 = torch.bfloat16, torch.float32, torch.int32, torch.uint8


def z(*shape, dtype=bf):
    return torch.zeros(*shape, dtype=dtype)


def py_rope(**kw):
    a = dict(x=z(8, 4, 64), table=z(10, 32, 2, dtype=f32), positions=z(8, dtype=i32))
    a.update(kw)
    return pkg.sdpa_rope(a.pop("x"), a.pop("table"), a.pop("positions"), **a)


ROPE_BAD = [
    (dict(x=z(8, 4, 64, dtype=torch.float16)), "x must be bf16"), (dict(x=z(8, 256)), "x must be bf16"),
    (dict(x=z(8, 4, 128)[..., ::2]), "inner stride"), (dict(table=z(10, 32, dtype=f32)), "table"),
    (dict(table=z(10, 32, 2, dtype=torch.float64)), "table"), (dict(table=z(10, 64, 2, dtype=f32)[:, ::2]), "table"),
    (dict(positions=None), "positions"), (dict(positions=z(8, dtype=torch.int64)), "positions"),
    (dict(positions=z(7, dtype=i32)), "positions"), (dict(positions=z(16, dtype=i32)[::2]), "positions"),
    (dict(positions=z(2, 8, dtype=i32)), "positions"), (dict(sections=()), "axes"),
    (dict(sections=(8, 8, 8, 4, 4)), "axes"), (dict(sections=(16, 16)), "positions"),
    (dict(out=z(8, 4, 128)), "out must be"), (dict(out=z(8, 4, 64, dtype=f32)), "out must be"), (dict(), "CUDA device"),
]


@pytest.mark.parametrize("kw,needle", ROPE_BAD)
def test_python_rope(kw, needle):
    with pytest.raises(ValueError, match=needle):
        py_rope(**kw)


def q4(rows=32, cols=2, Hkv=2, D=64, **kw):
    return pkg.q4_store(rows, cols, Hkv, D)._replace(**kw)


def py_append(fourbit, **kw):
    a = dict(q=z(8, 4, 64), k=z(8, 2, 64), v=z(8, 2, 64), store=q4() if fourbit else (z(32, 2, 2, 64), z(32, 2, 2, 64)),
             seq=z(1, 4, dtype=i32), table=z(10, 32, 2, dtype=f32))
    a.update(kw)
    st = a.pop("store")
    args = [a.pop(n) for n in ("q", "k", "v")] + ([st] if fourbit else list(st)) + [a.pop("seq"), a.pop("table")]
    return (pkg.sdpa_rope_append_q4 if fourbit else pkg.sdpa_rope_append)(*args, **a)


@pytest.mark.parametrize("fourbit", [False, True])
@pytest.mark.parametrize("kw,needle", [
    (dict(q=z(8, 4, 64, dtype=f32)), "q must be bf16"), (dict(q=z(8, 4, 128)), "head dims"),
    (dict(k=z(8, 4, 64)), "k_new must be"), (dict(v=z(7, 2, 64)), "v_new must be"),
    (dict(k=z(8, 2, 128)[..., ::2]), "inner stride"), (dict(seq=z(1, 3, dtype=i32)), "seq_info"),
    (dict(seq=z(1, 4, dtype=torch.int64)), "seq_info"), (dict(seq=z(2, 4, dtype=i32)[::2].T), "seq_info"),
    (dict(seg_mode=z(1, 3, dtype=i32)), "seg_mode"), (dict(seg_mode=z(2, 2, dtype=i32)), "seg_mode"),
    (dict(q_out=z(8, 2, 64)), "q_out must be"), (dict(sections=(16, 16)), "need positions"),
    (dict(positions=z(9, dtype=i32)), "positions"), (dict(), "CUDA device"),
])
def test_python_append(fourbit, kw, needle):
    with pytest.raises(ValueError, match=needle):
        py_append(fourbit, **kw)


@pytest.mark.parametrize("store,needle", [
    ((z(32, 2, 2, 64), z(32, 2, 3, 64)), "stores"), ((z(32, 2, 128), z(32, 2, 128)), "stores"),
    ((z(32, 2, 2, 64, dtype=f32), z(32, 2, 2, 64)), "bf16"), ((z(32, 4, 2, 64)[:, ::2], z(32, 2, 2, 64)), "contiguous"),
])
def test_python_bf16_stores(store, needle):
    with pytest.raises(ValueError, match=needle):
        py_append(False, store=store)


BAD_PY_STORES = [
    (q4(k_codes=z(2, 2, 32, 16, dtype=u8)), "4-bit store"), (q4(v_scales=z(2, 2, 32, 4, dtype=u8)), "4-bit store"),
    (q4(v_codes=z(2, 2, 32, 32, dtype=torch.int8)), "uint8"), (q4(k_codes=z(2, 2, 64, 32, dtype=u8)[:, :, ::2]), "uint8"),
]


@pytest.mark.parametrize("store,needle", BAD_PY_STORES)
def test_python_fourbit_stores(store, needle):
    seq = z(1, 4, dtype=i32)
    for call in (lambda: py_append(True, store=store), lambda: pkg.sdpa_q4_unpack(store, seq, 3),
                 lambda: pkg.sdpa_varlen_q4(z(8, 4, 64), store, seq, causal=True)):
        with pytest.raises(ValueError, match=needle):
            call()


def test_python_store_maker():
    for kw in (dict(rows=24), dict(rows=0), dict(D=96), dict(cols=0), dict(Hkv=0)):
        with pytest.raises(ValueError):
            q4(**kw)


def test_python_unpack_and_attend():
    seq = z(1, 4, dtype=i32)
    for kw, needle in ((dict(k_out=z(3, 2, 128)), "k_out must be"), (dict(v_out=z(4, 2, 64)), "v_out must be"),
                       (dict(k_out=z(3, 2, 64), v_out=z(3, 4, 64)[:, ::2]), "share strides"), (dict(), "CUDA device")):
        with pytest.raises(ValueError, match=needle):
            pkg.sdpa_q4_unpack(q4(), seq, 3, **kw)
    for q, kw, needle in ((z(8, 4, 128), {}, "head dims"), (z(8, 4, 64, dtype=f32), {}, "q must be bf16"),
                          (z(8, 4, 64), dict(seg_mode=z(1, 2)), "seg_mode"), (z(8, 4, 64), dict(out=z(8, 4, 128)), "out must be"),
                          (z(8, 4, 64), {}, "CUDA device")):
        with pytest.raises(ValueError, match=needle):
            pkg.sdpa_varlen_q4(q, q4(), seq, causal=True, **kw)
