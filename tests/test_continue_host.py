"""Shared prefixes, beam selection and reordering without a GPU: the 64-bit
forms pinned by hand, and every refusal of the entry points (fake device
addresses; nothing is launched)."""
import ctypes
import os

import numpy as np
import pytest

import kv_cache_eviction_tria_gb300 as tria
from oracle import beam_oracle as B

I, S, W = tria.ERR_INVALID_ARG, tria.ERR_UNSUPPORTED, tria.ERR_WORKSPACE
_KEPT = []          # the caches whose host arrays the structs below point to


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(tria.LIB_PATH):
        from kv_cache_eviction_tria_gb300 import _build
        _build.build()
    return tria.load_library()


def cache(n_seqs=2, base=0x10000, cap=100, **kw):
    kv = kw.get("n_kv_heads", 2)
    a = dict(k=base, v=base + 0x1000, pos=base + 0x2000, n_live=base + 0x3000, seq_row0=[kv * cap * s for s in range(n_seqs)],
             capacity=[cap] * n_seqs, head_dim=64, n_kv_heads=kv)
    a.update(kw)
    c = tria.LayerCache(**a)
    _KEPT.append(c)
    return c.c_struct()


# ----------------------------------------------------------------------------- the 64-bit forms

def test_values_are_log_probabilities():
    v = B.values(np.log([[1.0, 3.0, 4.0], [5.0, 4.0, 1.0]]), [0.0, np.log(0.5)])
    np.testing.assert_allclose(np.exp(v), [[1 / 8, 3 / 8, 1 / 2], [0.25, 0.2, 0.05]])
    over = B.values(np.zeros((2, 3)), [-1.0, -2.0], ended=[0, 1], end_token=2)
    np.testing.assert_allclose(over[0], -1 - np.log(3))
    assert over[1].tolist() == [-np.inf, -np.inf, -2.0]
    for junk in (np.nan, np.inf):
        assert (B.values([[0.0, junk, 1.0]], [0.0]) == -np.inf).all()
    assert (B.values([[-np.inf] * 3], [0.0]) == -np.inf).all() and (B.values([[0.0] * 3], [-np.inf]) == -np.inf).all()


def test_choice_and_places():
    v = np.array([[0.0, 5.0, 4.0], [4.0, 1.0, 1.0], [-1.0, -2.0, -np.inf]])
    assert [(b, t) for b, t, _ in B.choose(v, 10, 5)] == [(10, 1), (10, 2), (11, 0), (11, 1), (11, 2)]
    assert [(b, t) for b, t, _ in B.choose(v, 0, 3, in_place=True)] == [(0, 1), (1, 0), (0, 2)]


# ----------------------------------------------------------------------------- refusals

def test_attend_prefix_refusals(lib):
    def attend(code, prefix=None, own=None, seq0=(0, 2), ws=0x100000, ws_bytes=1 << 40, tok0=(0, 1, 2), **kw):
        p, c = prefix or cache(1, 0x40000), own or cache()
        a = tria._Attention()
        a.type, a.n_q_heads, a.q, a.out, a.pos, a.q_stride, a.out_stride = 1, 4, 0x1000, 0x2000, 0x3000, 256, 256
        t, s0 = np.asarray(tok0, np.int32), np.asarray(seq0, np.int32)
        a.tok0 = t.ctypes.data
        for k, v in kw.items():
            setattr(a, k, v)
        assert lib.tria_attend_prefix(ctypes.byref(p), ctypes.byref(c), s0.ctypes.data if len(s0) else None, ctypes.byref(a), ws,
                                      ws_bytes, None) == code, kw

    for kw in (dict(seq0=()), dict(seq0=(1, 2)), dict(seq0=(0, 1)), dict(seq0=(0, 3)), dict(prefix=cache(2, 0x40000), seq0=(0, 3, 2)),
               dict(prefix=cache(1, 0x40000, n_kv_heads=4)), dict(prefix=cache(1, 0x40000, head_dim=128)), dict(q=0), dict(out=0),
               dict(pos=0), dict(q=0x1008), dict(out=0x2004), dict(lse=0x2002), dict(q_stride=128), dict(out_stride=260), dict(window=-1),
               dict(sink=-1), dict(scale=-1.0), dict(scale=float("nan")), dict(scale=1e39), dict(round_keys=2), dict(tok0=(0, 2, 1)),
               dict(tok0=(1, 2, 3)), dict(n_q_heads=0), dict(prefix=cache(1, 0x40000, k_type="q8_0"))):
        attend(I, **kw)
    for kw in (dict(type=2), dict(n_q_heads=5), dict(n_q_heads=18), dict(prefix=cache(1, 0x40000, head_dim=288), own=cache(head_dim=288))):
        attend(S, **kw)
    attend(S, own=cache(seq_row0=[0, (1 << 31) - 100]), tok0=(0, 9, 18))
    attend(S, prefix=cache(1, 0x40000, seq_row0=[(1 << 31) - 100]), tok0=(0, 5, 9))
    attend(W, ws=0)
    attend(W, ws=0x100010)
    p, c = cache(1, 0x40000), cache()
    one, two = np.asarray([0, 2], np.int32), np.asarray([0, 1, 2], np.int32)
    need = lib.tria_attend_prefix_workspace_size(ctypes.byref(p), ctypes.byref(c), one.ctypes.data, 4, two.ctypes.data)
    assert need >= lib.tria_attend_workspace_size(ctypes.byref(c), 4, two.ctypes.data) > 0
    attend(W, ws_bytes=need - 1)
    attend(tria.OK, tok0=(0, 0, 0), q=0, out=0, pos=0)
    assert lib.tria_attend_prefix(ctypes.byref(p), ctypes.byref(c), one.ctypes.data, None, 0x100000, 1 << 34, None) == I
    assert lib.tria_attend_prefix_workspace_size(ctypes.byref(p), ctypes.byref(c), one.ctypes.data, 3, two.ctypes.data) == 0
    assert lib.tria_attend_prefix_workspace_size(ctypes.byref(p), None, one.ctypes.data, 4, two.ctypes.data) == 0
    assert lib.tria_attend_prefix_workspace_size(ctypes.byref(p), ctypes.byref(c), one.ctypes.data, 4, None) == 0


def tria_max_vocab():
    header = open(os.path.join(os.path.dirname(tria.LIB_PATH), os.pardir, "include", "tria.h")).read()
    return int(header.split("TRIA_MAX_VOCAB ")[1].split()[0])


def test_beam_select_refusals(lib):
    def select(code, seq0=(0, 3, 6), ws=0x100000, ws_bytes=1 << 30, **kw):
        b = tria._Beams()
        s0 = np.asarray(seq0, np.int32)
        b.type, b.n_groups, b.seq0, b.vocab, b.n_out, b.logits, b.stride = 1, len(s0) - 1, s0.ctypes.data, 100, 3, 0x1000, 100
        b.total, b.end_token, b.total_out, b.parent_out, b.token_out = 0x2000, -1, 0x3000, 0x4000, 0x5000
        for k, v in kw.items():
            setattr(b, k, v)
        assert lib.tria_beam_select(ctypes.byref(b), ws, ws_bytes, None) == code, kw

    for kw in (dict(logits=0), dict(total=0), dict(total_out=0), dict(parent_out=0), dict(token_out=0), dict(logits=0x1001),
               dict(type=0, logits=0x1002), dict(total=0x2002), dict(total_out=0x3001), dict(parent_out=0x4002), dict(token_out=0x5002),
               dict(ended_out=0x6001), dict(ended=0x7002, end_token=1), dict(stride=99), dict(vocab=0), dict(n_out=0), dict(n_groups=0),
               dict(end_token=100), dict(end_token=-2), dict(ended=0x7000), dict(in_place=2), dict(in_place=1, n_out=2),
               dict(n_out=4, total_out=0x2000), dict(n_out=2, ended=0x7000, ended_out=0x7000, end_token=0), dict(vocab=1, n_out=4),
               dict(seq0=(1, 3, 6)), dict(seq0=(0, 0, 6)), dict(seq0=(0, 4, 3)), dict(seq0=(0, 2, 6), in_place=1)):
        select(I, **kw)
    for kw in (dict(type=2), dict(type=3), dict(vocab=tria_max_vocab() + 1, stride=1 << 30), dict(n_out=65), dict(seq0=(0, 33)),
               dict(seq0=range(0, 390, 3))):
        select(S, **kw)
    select(W, ws=0)
    select(W, ws=0x100080)
    s0 = np.asarray([0, 3, 6], np.int32)
    need = lib.tria_beam_select_workspace_size(s0.ctypes.data, 2, 100, 3)
    select(W, ws_bytes=need - 1)
    assert lib.tria_beam_select(None, 0x100000, 1 << 30, None) == I
    assert lib.tria_beam_select_workspace_size(None, 2, 100, 3) == 0 and lib.tria_beam_select_workspace_size(s0.ctypes.data, 2, 0, 3) == 0
    assert lib.tria_beam_select_workspace_size(s0.ctypes.data, 2, 100, 65) == 0


def test_reorder_refusals(lib):
    def reorder(code, caches=None, n_layers=None, seq0=(0, 4), parent=0x9000, ws=0x100000, ws_bytes=256, n_groups=None):
        caches = [cache(4, 0x10000 + 0x8000 * i) for i in range(3)] if caches is None else caches
        arr = (tria._LayerCache * max(len(caches), 1))(*caches)
        s0 = np.asarray(seq0, np.int32)
        assert lib.tria_reorder(arr if caches else None, len(caches) if n_layers is None else n_layers, s0.ctypes.data if len(s0) else None,
                                len(s0) - 1 if n_groups is None else n_groups, parent, ws, ws_bytes, None) == code

    a, b = cache(4, 0x10000), cache(4, 0x18000)
    shared = []
    for name in ("k", "v", "pos", "n_live"):
        x = cache(4, 0x18000)
        setattr(x, name, getattr(a, name))
        shared.append([a, x])
    for kw in ([dict(caches=c) for c in shared] +
               [dict(caches=[a, cache(4, 0x18000, head_dim=128)]), dict(caches=[a, cache(3, 0x18000)]), dict(caches=[a, cache(4, 0x18000, n_kv_heads=1)]),
                dict(caches=[a, cache(4, 0x18000, k_type="f32")]), dict(caches=[a, cache(4, 0x18000, v_type="f32")]),
                dict(caches=[a, cache(4, 0x18000, cap=101)]), dict(caches=[]), dict(n_layers=0), dict(seq0=()), dict(seq0=(0, 3)),
                dict(seq0=(1, 4)), dict(seq0=(0, 3, 2, 4)), dict(n_groups=0), dict(parent=0), dict(parent=0x9002),
                dict(caches=[cache(4, 0x10000, seq_row0=[0, 100, 400, 600])])]):
        reorder(I, **kw)
    reorder(S, caches=[cache(4, 0x10000 + 0x8000 * i) for i in range(129)])
    reorder(S, caches=[cache(33, 0x10000)], seq0=(0, 33))
    reorder(W, ws=0)
    reorder(W, ws=0x100080)
    reorder(W, ws_bytes=255)
    s0 = np.asarray([0, 4], np.int32)
    arr = (tria._LayerCache * 2)(a, b)
    assert lib.tria_reorder_workspace_size(arr, 2, s0.ctypes.data, 1) == 256
    assert lib.tria_reorder_workspace_size(arr, 2, None, 1) == 0 and lib.tria_reorder_workspace_size(None, 2, s0.ctypes.data, 1) == 0
    twice = (tria._LayerCache * 2)(a, a)
    assert lib.tria_reorder_workspace_size(twice, 2, s0.ctypes.data, 1) == 0


def test_rows_past_a_tiles_coordinate_take_no_tiles(lib):
    """A prefix whose last row's index needs more than 31 bits: up to 16 columns read it without tiles, which shows in the
    workspace."""
    t, s0 = np.asarray([0, 1, 2], np.int32), np.asarray([0, 2], np.int32)
    size = [lib.tria_attend_prefix_workspace_size(ctypes.byref(cache(1, 0x40000, seq_row0=[r])), ctypes.byref(cache()), s0.ctypes.data, 4,
                                                  t.ctypes.data) for r in (0, (1 << 31) - 201, (1 << 31) - 200)]
    assert size[0] == size[1] > size[2] > 0
