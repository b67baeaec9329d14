"""What tria_reorder refuses of layers that share a plane (fake device addresses;
nothing is launched)."""
import ctypes
import os

import numpy as np
import pytest

import kv_cache_eviction_tria_gb300 as tria
from test_continue_host import cache, lib  # noqa: F401 (a fixture)

PLANES = ("k", "v", "k_scale", "v_scale", "pos", "n_live")


def layer(i, **kw):
    base = 0x10000 + 0x8000 * i
    return cache(4, base, k_type="q8_0", v_type="q4_0", k_scale=base + 0x4000, v_scale=base + 0x5000, **kw)


def reorder(lib, caches):  # noqa: F811
    arr, s0 = (tria._LayerCache * len(caches))(*caches), np.asarray([0, 4], np.int32)
    size = lib.tria_reorder_workspace_size(arr, len(caches), s0.ctypes.data, 1)
    # (a workspace of no bytes: what passes the checks of the caches is not launched)
    return size, lib.tria_reorder(arr, len(caches), s0.ctypes.data, 1, 0x9000, 0x100000, 0, None)


def test_layers_of_their_own_are_taken(lib):  # noqa: F811
    assert reorder(lib, [layer(0), layer(1), layer(2)]) == (256, tria.ERR_WORKSPACE)


@pytest.mark.parametrize("of", PLANES)
@pytest.mark.parametrize("to", PLANES)
@pytest.mark.parametrize("layers", [(0, 1), (0, 2), (2, 0), (1, 1)])
def test_a_plane_of_two_is_refused(lib, of, to, layers):  # noqa: F811
    """Any plane in the place of any other one, of another layer or of the same one."""
    if layers[0] == layers[1] and of == to:
        return
    c = [layer(i) for i in range(3)]
    setattr(c[layers[1]], to, getattr(c[layers[0]], of))
    assert reorder(lib, c) == (0, tria.ERR_INVALID_ARG)


def test_scales_start_on_any_value(lib):  # noqa: F811
    """Layers side by side in one array, whose rows' scales take no multiple of 16 bytes."""
    for off in (2, 4, 8, 14):
        c = [layer(0), layer(1)]
        c[1].k_scale += off
        c[0].v_scale += off
        assert reorder(lib, c) == (256, tria.ERR_WORKSPACE)
    for name, off in (("k_scale", 1), ("v_scale", 3), ("k", 8), ("v", 8), ("pos", 2), ("n_live", 2)):
        c = [layer(0), layer(1)]
        setattr(c[1], name, getattr(c[1], name) + off)
        assert reorder(lib, c) == (0, tria.ERR_INVALID_ARG)
