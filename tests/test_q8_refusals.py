"""Arguments that the 8-bit entries refuse, all of them before any CUDA call (the pointers of the C calls are fake
and never dereferenced)."""
import pytest
import torch

import varlen_gqa_attention_gb300 as pkg

from test_step_refusals import (ALIGN, ARG, BAD_ROTATIONS, FAKE, GQA, HEAD_DIM, NULL, SHAPE, STRIDE, WORKSPACE, f32, i32,
                                rotation,
                                u8, z)


def store(**kw):
    a = dict(k_codes=FAKE, k_scales=FAKE, v_codes=FAKE, v_scales=FAKE)
    a.update(kw)
    return pkg._Q8_POINTERS.pack(*a.values())


def append(**kw):
    a = dict(q=FAKE, q_rs=256, q_hs=64, k=FAKE, k_rs=128, k_hs=64, v=FAKE, v_rs=128, v_hs=64, T=8, Hq=4, Hkv=2, D=64,
             rot=rotation(), store=store(), rows=32, cols=2, seq=FAKE, mode=None, S=1, window=0, out=FAKE, o_rs=256,
             o_hs=64, status=None, stream=None)
    assert set(kw) <= set(a)
    a.update(kw)
    return pkg.library().sdpa_rope_append_eightbit(*a.values())


def unpack(**kw):
    a = dict(store=store(), rows=32, cols=2, Hkv=2, D=64, seq=FAKE, mode=None, S=1, window=0, T=8, k_out=FAKE,
             v_out=FAKE, o_rs=128, o_hs=64, status=None, stream=None)
    assert set(kw) <= set(a)
    a.update(kw)
    return pkg.library().sdpa_eightbit_unpack(*a.values())


BAD_STORES = [(dict(store=None), NULL), (dict(rows=24), SHAPE), (dict(rows=8), SHAPE)] + \
    [(dict(store=store(**{n: 0})), NULL) for n in ("k_codes", "k_scales", "v_codes", "v_scales")] + \
    [(dict(store=store(**{n: FAKE + 8})), ALIGN) for n in ("k_codes", "v_codes")]


@pytest.mark.parametrize("kw,code", BAD_STORES)
def test_stores(kw, code):
    assert append(**kw) == code
    assert unpack(**kw) == code


@pytest.mark.parametrize("rot,code", BAD_ROTATIONS)
def test_append_rotations(rot, code):
    assert append(rot=rot) == code


@pytest.mark.parametrize("kw,code", [
    (dict(q=None), NULL), (dict(k=None), NULL), (dict(v=None), NULL), (dict(out=None), NULL), (dict(seq=None), NULL),
    (dict(T=-1), SHAPE), (dict(S=-1), SHAPE), (dict(cols=0), SHAPE), (dict(rows=1 << 31), SHAPE), (dict(D=96), HEAD_DIM),
    (dict(Hq=5), GQA), (dict(Hq=258), GQA), (dict(window=-1), ARG), (dict(q=FAKE + 2), ALIGN), (dict(k=FAKE + 8), ALIGN),
    (dict(v=FAKE + 8), ALIGN), (dict(out=FAKE + 8), ALIGN), (dict(seq=FAKE + 4), ALIGN), (dict(mode=FAKE + 4), ALIGN),
    (dict(k_rs=12), STRIDE), (dict(v_hs=-64), STRIDE), (dict(q_hs=60), STRIDE), (dict(o_rs=-256), STRIDE),
    (dict(Hq=1 << 20, Hkv=1 << 20), SHAPE),
])
def test_append(kw, code):
    assert append(**kw) == code


@pytest.mark.parametrize("kw,code", [
    (dict(k_out=None), NULL), (dict(v_out=None), NULL), (dict(seq=None), NULL), (dict(T=-1), SHAPE),
    (dict(Hkv=0), SHAPE), (dict(cols=-1), SHAPE), (dict(Hkv=1 << 20), SHAPE), (dict(D=32), HEAD_DIM),
    (dict(window=-2), ARG), (dict(seq=FAKE + 8), ALIGN), (dict(mode=FAKE + 4), ALIGN), (dict(k_out=FAKE + 2), ALIGN),
    (dict(v_out=FAKE + 2), ALIGN), (dict(o_rs=-8), STRIDE), (dict(o_hs=20), STRIDE),
])
def test_unpack(kw, code):
    assert unpack(**kw) == code


def test_no_rows_do_nothing():
    assert append(T=0, q=None, k=None, v=None, out=None) == 0
    assert unpack(T=0, k_out=None, v_out=None) == 0


# ------------------------------------------------------------------------------- the Python entries

def q8(rows=32, cols=2, Hkv=2, D=64, **kw):
    return pkg.q8_store(rows, cols, Hkv, D)._replace(**kw)


def py_append(**kw):
    a = dict(q=z(8, 4, 64), k=z(8, 2, 64), v=z(8, 2, 64), store=q8(), seq=z(1, 4, dtype=i32),
             table=z(10, 32, 2, dtype=f32))
    a.update(kw)
    return pkg.sdpa_rope_append_q8(*[a.pop(n) for n in ("q", "k", "v", "store", "seq", "table")], **a)


@pytest.mark.parametrize("kw,needle", [
    (dict(q=z(8, 4, 64, dtype=f32)), "q must be bf16"), (dict(q=z(8, 4, 128)), "head dims"),
    (dict(k=z(8, 4, 64)), "k_new must be"), (dict(v=z(7, 2, 64)), "v_new must be"),
    (dict(k=z(8, 2, 128)[..., ::2]), "inner stride"), (dict(seq=z(1, 3, dtype=i32)), "seq_info"),
    (dict(seg_mode=z(2, 2, dtype=i32)), "seg_mode"), (dict(q_out=z(8, 2, 64)), "q_out must be"),
    (dict(sections=(16, 16)), "need positions"), (dict(positions=z(9, dtype=i32)), "positions"),
    (dict(window=2 ** 31), "window|CUDA device"), (dict(), "CUDA device"),
])
def test_python_append(kw, needle):
    with pytest.raises(ValueError, match=needle):
        py_append(**kw)


@pytest.mark.parametrize("bad,needle", [
    (q8(k_codes=z(2, 2, 32, 32, dtype=u8)), "8-bit store"), (q8(v_scales=z(2, 2, 4, dtype=u8)), "8-bit store"),
    (q8(v_codes=z(2, 2, 32, 64, dtype=torch.int8)), "uint8"), (q8(k_codes=z(2, 2, 64, 64, dtype=u8)[:, :, ::2]), "uint8"),
    (pkg.Q8Store(*[z(2, 2, 24, 64, dtype=u8), z(2, 2, 1, dtype=u8)] * 2), "8-bit store"),
    (pkg.q4_store(32, 2, 2, 64), "8-bit store"),
])
def test_python_stores(bad, needle):
    seq = z(1, 4, dtype=i32)
    for call in (lambda: py_append(store=bad), lambda: pkg.sdpa_q8_unpack(bad, seq, 3)):
        with pytest.raises(ValueError, match=needle):
            call()


def test_python_store_maker():
    for kw in (dict(rows=24), dict(rows=0), dict(D=96), dict(cols=0), dict(Hkv=0)):
        with pytest.raises(ValueError):
            q8(**kw)


def test_python_unpack():
    seq = z(1, 4, dtype=i32)
    for kw, needle in ((dict(k_out=z(3, 2, 128)), "k_out must be"), (dict(v_out=z(4, 2, 64)), "v_out must be"),
                       (dict(k_out=z(3, 2, 64), v_out=z(3, 4, 64)[:, ::2]), "share strides"), (dict(), "CUDA device")):
        with pytest.raises(ValueError, match=needle):
            pkg.sdpa_q8_unpack(q8(), seq, 3, **kw)


def attend(**kw):
    a = dict(q=FAKE, T=8, Hq=4, D=64, q_rs=256, q_hs=64, store=store(), rows=32, cols=2, Hkv=2, seq=FAKE, mode=None,
             S=1, causal=1, window=0, scale=0.125, out=FAKE, o_rs=256, o_hs=64, ws=FAKE, ws_bytes=1 << 30,
             status=None, stream=None)
    assert set(kw) <= set(a)
    a.update(kw)
    return pkg.library().sdpa_varlen_eightbit(*a.values())


@pytest.mark.parametrize("kw,code", BAD_STORES + [
    (dict(q=None), NULL), (dict(out=None), NULL), (dict(seq=None), NULL), (dict(ws=None), WORKSPACE),
    (dict(T=-1), SHAPE), (dict(rows=1 << 31), SHAPE), (dict(S=-1), SHAPE), (dict(D=112), HEAD_DIM), (dict(Hq=5), GQA),
    (dict(Hq=258), GQA), (dict(window=-1), ARG), (dict(scale=float("inf")), ARG), (dict(scale=float("nan")), ARG),
    (dict(scale=-0.125), ARG), (dict(q=FAKE + 2), ALIGN), (dict(out=FAKE + 8), ALIGN), (dict(seq=FAKE + 4), ALIGN),
    (dict(mode=FAKE + 8), ALIGN), (dict(ws=FAKE + 16), ALIGN), (dict(q_rs=-8), STRIDE), (dict(q_hs=60), STRIDE),
    (dict(o_rs=12), STRIDE), (dict(o_hs=-64), STRIDE), (dict(cols=1 << 30, Hkv=2), SHAPE),
])
def test_attend(kw, code):
    assert attend(**kw) == code


@pytest.mark.parametrize("D", [64, 128, 256])
def test_a_workspace_for_bounds_serves_every_smaller_call(D):
    need = pkg.library().sdpa_varlen_eightbit_workspace_bytes
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


def test_python_attend():
    seq = z(1, 4, dtype=i32)
    for q, kw, needle in ((z(8, 4, 128), {}, "head dims"), (z(8, 4, 64, dtype=f32), {}, "q must be bf16"),
                          (z(8, 4, 64), dict(seg_mode=z(1, 2)), "seg_mode"), (z(8, 4, 64), dict(out=z(8, 4, 128)), "out must be"),
                          (z(8, 4, 64), {}, "CUDA device")):
        with pytest.raises(ValueError, match=needle):
            pkg.sdpa_varlen_q8(q, q8(), seq, causal=True, **kw)
    with pytest.raises(ValueError, match="8-bit store"):
        pkg.sdpa_varlen_q8(z(8, 4, 64), pkg.q4_store(32, 2, 2, 64), seq, causal=True)
