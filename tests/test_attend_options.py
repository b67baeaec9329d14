"""Options of tria_attend that are checked on the host (fake device addresses; nothing is launched)."""
import ctypes
import os

import numpy as np
import pytest

import kv_cache_eviction_tria_gb300 as tria


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(tria.LIB_PATH):
        from kv_cache_eviction_tria_gb300 import _build
        _build.build()
    return tria.load_library()


@pytest.mark.parametrize("value,code", [(0, tria.OK), (1, tria.OK), (2, tria.ERR_INVALID_ARG), (-1, tria.ERR_INVALID_ARG)])
def test_round_keys_is_yes_or_no(lib, value, code):
    c = tria.LayerCache(k=0x10000, v=0x20000, pos=0x30000, n_live=0x40000, seq_row0=[0], capacity=[100], head_dim=64, n_kv_heads=2)
    tok0 = np.zeros(2, np.int32)                             # no tokens: checked, and nothing to do
    a = tria._Attention(1, 4, 0x1000, 0x2000, 0x3000, 256, 256, 0x4000, tok0.ctypes.data, 0.0, 0, 0, value)
    assert lib.tria_attend(c.c_ref(), ctypes.byref(a), 0x100000, 1 << 30, None) == code
