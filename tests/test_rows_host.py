"""Rotation, append and attention without a GPU: the 64-bit forms pinned by
identities, the scaled frequencies against them, and every refusal of the
entry points (fake device addresses; nothing is launched)."""
import ctypes
import os

import numpy as np
import pytest

import kv_cache_eviction_tria_gb300 as tria
from oracle import attend_oracle as A
from synth import counter_rng as C


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(tria.LIB_PATH):
        from kv_cache_eviction_tria_gb300 import _build
        _build.build()
    return tria.load_library()


# ----------------------------------------------------------------------------- the 64-bit forms

@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_rotated_products_depend_on_the_distance_alone(layout):
    rng = np.random.default_rng(0)
    q, k = rng.standard_normal((2, 1, 1, 64))
    w, _ = A.frequencies(64, 1e4, 16)
    dot = [float((A.turn(q, [a], w, 1.0, 16, layout) * A.turn(k, [b], w, 1.0, 16, layout)).sum()) for a, b in ((9, 4), (105, 100), (5, 0))]
    assert max(dot) - min(dot) < 1e-11
    np.testing.assert_allclose(A.turn(q, [0], w, 1.0, 16, layout), q)


def test_interleaved_to_half_is_a_permutation_of_interleaved():
    rng = np.random.default_rng(1)
    x = rng.standard_normal((3, 2, 32))
    w, _ = A.frequencies(32, 1e4)
    a, b = A.turn(x, [1, 2, 3], w, 1.0, 0, "interleaved"), A.turn(x, [1, 2, 3], w, 1.0, 0, "interleaved_to_half")
    np.testing.assert_array_equal(np.concatenate([a[..., 0::2], a[..., 1::2]], -1), b)
    half = np.concatenate([x[..., 0::2], x[..., 1::2]], -1)
    np.testing.assert_allclose(A.turn(half, [1, 2, 3], w), b)


def test_scaled_frequencies_at_their_ends():
    w0, _ = A.frequencies(128, 1e6)
    y, m = A.frequencies(128, 1e6, 0, "yarn", 4.0, 32768)
    b, _ = A.frequencies(128, 1e6, 0, "bands", 4.0, 32768)
    for s in (y, b):
        assert s[0] == w0[0] and np.isclose(s[-1], w0[-1] / 4) and np.all(s <= w0) and np.all(s >= w0 / 4 * (1 - 1e-12))
    assert np.isclose(m, 1 + 0.1 * np.log(4))
    n, _ = A.frequencies(128, 1e6, 0, "ntk", 4.0)
    assert n[0] == 1.0 and np.isclose(n[-1], w0[-1] / 4)


def test_q8_0_is_the_generators():
    x = np.random.default_rng(2).standard_normal((5, 96)).astype(np.float32)
    for a, b in zip(A.quantize_q8_0(x), C.quantize_q8_0(x)):
        np.testing.assert_array_equal(a, b)


def test_q4_0_codes():
    x = np.zeros((1, 32), np.float32)
    x[0, 5], x[0, 20], x[0, 31] = 8.0, -8.0, 3.4
    data, scale = A.quantize_q4_0(x)
    assert scale[0, 0] == -1.0                           # the first value of largest modulus gives code 0
    codes = A.codes_q4_0(data)[0]
    assert codes[5] == 0 and codes[20] == 15 and codes[31] == 5 and codes[0] == 8
    assert data[0, 4] == (codes[4] | codes[20] << 4)
    np.testing.assert_array_equal(A.values(data, scale, "q4_0")[0, [5, 20, 31, 0]], [8, -7, 3, 0])
    z, s = A.quantize_q4_0(np.zeros((1, 32), np.float32))
    assert np.all(z == 0x88) and s[0, 0] == 0 and not np.signbit(s[0, 0])


def test_attention_special_cases():
    rng = np.random.default_rng(3)
    k, v = rng.standard_normal((2, 9, 32))
    q = rng.standard_normal((2, 32))
    pos = np.arange(9) * 2
    out, lse, w, _ = A.attend_rows(q, 100, k, v, pos)
    np.testing.assert_allclose(w.sum(-1), 1)
    np.testing.assert_allclose(out, w @ v)
    out, lse, _, _ = A.attend_rows(q, 4, k, v, pos, window=1)
    np.testing.assert_allclose(out, np.repeat(v[2:3], 2, 0))
    out, lse, w, _ = A.attend_rows(q, 16, k, v, pos, window=3, sink=2)
    assert set(np.flatnonzero(w[0])) == {0, 1, 7, 8}
    out, lse, _, _ = A.attend_rows(q, -1, k, v, pos)
    assert not out.any() and np.all(lse == -np.inf)


# ----------------------------------------------------------------------------- frequencies of the library

@pytest.mark.parametrize("scaling,kw", [("none", {}), ("linear", dict(factor=4.0)), ("ntk", dict(factor=3.0)),
                                        ("yarn", dict(factor=4.0, orig_ctx=32768)),
                                        ("yarn", dict(factor=16.0, orig_ctx=4096, low=2.0, high=20.0)),
                                        ("bands", dict(factor=8.0, orig_ctx=8192)),
                                        ("bands", dict(factor=2.0, orig_ctx=100, low=0.5, high=9.0))])
@pytest.mark.parametrize("hd,nonrot", [(128, 0), (64, 32), (96, 80)])
def test_frequencies(lib, scaling, kw, hd, nonrot):
    w, m = tria.rope_frequencies(head_dim=hd, nonrot_dim=nonrot, theta=5e5, scaling=scaling, **kw)
    a, am = A.frequencies(hd, 5e5, nonrot, scaling, **kw)
    np.testing.assert_allclose(w, a, rtol=1e-13)
    assert abs(m - am) < 1e-13
    assert tria.rope_frequencies(head_dim=hd, nonrot_dim=nonrot, theta=5e5, scaling=scaling, mscale=2.5, **kw)[1] == 2.5


@pytest.mark.parametrize("bad,code", [
    (dict(head_dim=48), 2), (dict(head_dim=288), 2), (dict(head_dim=0), 2), (dict(nonrot_dim=8), 2), (dict(nonrot_dim=64), 1),
    (dict(nonrot_dim=-16), 1), (dict(theta=1.0), 1), (dict(theta=float("nan")), 1), (dict(scaling="linear", factor=0.5), 1),
    (dict(scaling="yarn", factor=4.0, orig_ctx=0), 1), (dict(scaling="bands", factor=4.0, orig_ctx=100, low=5.0), 1),
    (dict(scaling="yarn", factor=float("inf"), orig_ctx=10), 1), (dict(mscale=-1.0), 1), (dict(mscale=float("nan")), 1),
    (dict(omega=[float("inf")] * 32), 1), (dict(omega=[0.5] * 32, scaling="linear", factor=2.0), 1)])
def test_bad_rotations_are_refused(lib, bad, code):
    kw = {**dict(head_dim=64, theta=1e4), **bad}
    with pytest.raises((tria.TriaError, ValueError)) as e:
        tria.rope_frequencies(**kw)
    if isinstance(e.value, tria.TriaError):
        assert e.value.status == code
    with pytest.raises((tria.TriaError, ValueError)) as e:
        tria.Rope(**kw)
    if isinstance(e.value, tria.TriaError):
        assert e.value.status == code


# ----------------------------------------------------------------------------- refusals

def cache(**kw):
    a = dict(k=0x10000, v=0x20000, pos=0x30000, n_live=0x40000, seq_row0=[0, 200], capacity=[100, 90], head_dim=64,
             n_kv_heads=2, k_type="f16", v_type="f16", k_scale=None, v_scale=None)
    a.update(kw)
    return tria.LayerCache(**a)


def attention(lib, c, code, ws=0x100000, ws_bytes=1 << 30, tok0=(0, 1, 2), **kw):
    a = tria._Attention(1, 4, 0x1000, 0x2000, 0x3000, 256, 256, 0x4000, None, 0.0, 0, 0)
    t = np.asarray(tok0, np.int32)
    a.tok0 = t.ctypes.data
    for k, v in kw.items():
        setattr(a, k, v)
    s = c.c_struct()
    assert lib.tria_attend(ctypes.byref(s), ctypes.byref(a), ws, ws_bytes, None) == code, kw


def test_attend_refusals(lib):
    c = cache()
    I, S, W = tria.ERR_INVALID_ARG, tria.ERR_UNSUPPORTED, tria.ERR_WORKSPACE
    for kw in (dict(q=0), dict(out=0), dict(pos=0), dict(q=0x1008), dict(out=0x2004), dict(pos=0x4002), dict(lse=0x3001),
               dict(q_stride=252), dict(out_stride=128), dict(q_stride=257), dict(window=-1), dict(sink=-1), dict(scale=-0.5),
               dict(scale=float("nan")), dict(scale=float("inf")), dict(tok0=(1, 1, 2)), dict(tok0=(0, 2, 1)), dict(n_q_heads=0)):
        attention(lib, c, I, **kw)
    for kw in (dict(n_q_heads=5), dict(n_q_heads=18), dict(type=2), dict(type=3), dict(type=9)):
        attention(lib, c, S, **kw)
    attention(lib, c, W, ws=0)
    attention(lib, c, W, ws=0x100010)
    need = tria.attend_workspace_size(c, 4, 1)
    attention(lib, c, W, ws_bytes=need - 1)
    attention(lib, c, tria.OK, tok0=(0, 0, 0), q=0, out=0, pos=0)      # no tokens: nothing to do
    attention(lib, cache(k_type="q4_0"), I)                            # scales are missing
    attention(lib, cache(k_scale=0x50000), I)                          # scales of a type without
    attention(lib, cache(head_dim=288), S)
    s = c.c_struct()
    assert lib.tria_attend(ctypes.byref(s), None, 0x100000, 1 << 30, None) == I
    assert lib.tria_attend_workspace_size(ctypes.byref(s), 3, np.zeros(3, np.int32).ctypes.data) == 0
    assert lib.tria_attend_workspace_size(ctypes.byref(s), 4, None) == 0


def test_rotate_and_append_refusals(lib):
    I, S, W = tria.ERR_INVALID_ARG, tria.ERR_UNSUPPORTED, tria.ERR_WORKSPACE

    class Handle(ctypes.Structure):       # a handle's host part, read by the checks only
        _fields_ = [("head_dim", ctypes.c_int32), ("nonrot_dim", ctypes.c_int32), ("layout", ctypes.c_int32),
                    ("pad", ctypes.c_int32), ("mscale", ctypes.c_double), ("turns", ctypes.c_void_p)]
    rope = Handle(64, 0, 0, 0, 1.0, None)
    h = (tria._Heads * 2)()

    def rotate(code, type=1, n_parts=1, n=3, pos=0x4000, eps=1e-6, rope_p=ctypes.byref(rope), **kw):
        for x in h:
            x.x, x.out, x.norm, x.n_heads, x.x_stride, x.out_stride = 0x1000, 0x2000, None, 2, 128, 128
        for k, v in kw.items():
            setattr(h[n_parts - 1 if 0 < n_parts < 3 else 0], k, v)
        assert lib.tria_rotate(rope_p, type, h, n_parts, n, pos, eps, None) == code, kw

    for kw in (dict(rope_p=None), dict(n_parts=0), dict(n_parts=3), dict(n=-1), dict(pos=0), dict(pos=0x4002), dict(eps=-1.0),
               dict(eps=float("nan")), dict(x=0), dict(out=0), dict(x=0x1008), dict(norm=0x1004), dict(n_heads=0),
               dict(x_stride=120), dict(out_stride=132), dict(n_parts=2, x=0)):
        rotate(I, **kw)
    rotate(S, type=2)
    rotate(tria.OK, n=0, pos=0)

    def append(code, c=None, ws=0x100000, ws_bytes=1 << 20, tok0=(0, 1, 2), rope_p=ctypes.byref(rope), **kw):
        a = tria._Qkv()
        a.type, a.n_q_heads, a.q, a.k, a.v, a.q_out = 1, 4, 0x1000, 0x2000, 0x3000, 0x4000
        a.q_stride, a.k_stride, a.v_stride, a.q_out_stride, a.eps, a.pos = 256, 128, 128, 256, 1e-6, 0x5000
        t = np.asarray(tok0, np.int32)
        a.tok0 = t.ctypes.data
        for k, v in kw.items():
            setattr(a, k, v)
        s = (c or cache()).c_struct()
        assert lib.tria_append_qkv(rope_p, ctypes.byref(s), ctypes.byref(a), ws, ws_bytes, None) == code, kw

    for kw in (dict(rope_p=None), dict(n_q_heads=-1), dict(q=0), dict(k=0), dict(v=0), dict(q_out=0), dict(k=0x2004),
               dict(k_stride=64), dict(v_stride=130), dict(q_norm=0x6004), dict(k_norm=0x6008), dict(k_held=0x6008),
               dict(v_held=0x6001), dict(pos=0), dict(pos=0x5001), dict(n_before=0x7001), dict(eps=-1e-9), dict(tok0=(0, 2, 1)),
               dict(tok0=(3, 3, 3)), dict(c=cache(head_dim=32)), dict(c=cache(v_type="q8_0"))):
        append(I, **kw)
    append(S, type=3)
    append(W, ws=0)
    append(W, ws=0x100008)
    append(W, ws_bytes=16)
    append(tria.OK, tok0=(0, 0, 0), q=0, k=0, v=0, pos=0)


def test_refusals_of_sizes_and_of_uneven_strides_in_place(lib):
    """Counts that pass 31 bits, logit factors outside float's range, rows past a tile's 31-bit coordinate; an output
    in the place of its input with another stride, whose heads would be overwritten before they are read."""
    I, S = tria.ERR_INVALID_ARG, tria.ERR_UNSUPPORTED
    c = cache()
    t = np.asarray([0, 1 << 29, 1 << 29], np.int32)
    s = c.c_struct()
    assert lib.tria_attend_workspace_size(ctypes.byref(s), 4, t.ctypes.data) == 0
    attention(lib, c, S, tok0=t)
    attention(lib, c, I, scale=1e39)
    attention(lib, cache(seq_row0=[0, (1 << 31) - 100]), S, tok0=(0, 9, 9))

    class Handle(ctypes.Structure):
        _fields_ = [("head_dim", ctypes.c_int32), ("nonrot_dim", ctypes.c_int32), ("layout", ctypes.c_int32),
                    ("pad", ctypes.c_int32), ("mscale", ctypes.c_double), ("turns", ctypes.c_void_p)]
    rope = Handle(64, 0, 0, 0, 1.0, None)
    h = tria._Heads()
    h.x, h.out, h.norm, h.n_heads, h.x_stride, h.out_stride = 0x1000, 0x1000, None, 2, 128, 256
    assert lib.tria_rotate(ctypes.byref(rope), 1, ctypes.byref(h), 1, 3, 0x4000, 1e-6, None) == I
    a = tria._Qkv()
    a.type, a.n_q_heads, a.q, a.k, a.v, a.q_out = 1, 4, 0x1000, 0x2000, 0x3000, 0x1000
    a.q_stride, a.k_stride, a.v_stride, a.q_out_stride, a.eps, a.pos = 512, 128, 128, 256, 1e-6, 0x5000
    two = np.asarray([0, 1, 2], np.int32)
    a.tok0 = two.ctypes.data
    assert lib.tria_append_qkv(ctypes.byref(rope), ctypes.byref(s), ctypes.byref(a), 0x100000, 1 << 20, None) == I


def test_q4_0_cache_in_the_other_entry_points(lib):
    """The pass's host checks take q4_0 planes, and bf16 is no type of a cache."""
    c = cache(k_type="q4_0", v_type="q4_0", k_scale=0x50000, v_scale=0x60000)
    assert tria.workspace_size(c, 4) > 0
    bad = cache()
    bad.k_type = tria.BF16
    with pytest.raises(tria.TriaError):
        tria.workspace_size(bad, 4)
