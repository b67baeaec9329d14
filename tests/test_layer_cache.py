"""The binding's LayerCache keeps a C struct between calls: what that must not
change. No GPU: planes are addresses, or stand-ins for tensors."""
import copy
import pickle

import numpy as np
import pytest

import kv_cache_eviction_tria_gb300 as tria


class Plane:
    """What the binding asks of a tensor."""
    is_cuda = True

    def __init__(self, at, contiguous=True):
        self.at, self.contiguous = at, contiguous

    def data_ptr(self):
        return self.at

    def is_contiguous(self):
        return self.contiguous


def cache(make=lambda at: at):
    return tria.LayerCache(k=make(0x10000), v=make(0x20000), pos=make(0x30000), n_live=make(0x40000), seq_row0=[0, 200],
                           capacity=[100, 90], head_dim=64, n_kv_heads=2, k_type="q8_0", v_type="q4_0",
                           k_scale=make(0x50000), v_scale=make(0x60000))


def fields(ref):
    c = ref._obj
    out = {n: getattr(c, n) for n, _ in c._fields_}
    out["seq_row0"], out["capacity"] = list(c.seq_row0[:c.n_seqs]), list(c.capacity[:c.n_seqs])
    return out


@pytest.mark.parametrize("again", [copy.copy, copy.deepcopy, lambda c: pickle.loads(pickle.dumps(c))])
@pytest.mark.parametrize("used", [False, True])
def test_a_cache_is_copied_after_its_use(again, used):
    c = cache()
    want = fields(c.c_ref()) if used else fields(cache().c_ref())
    d = again(c)
    assert fields(d.c_ref()) == want
    d.head_dim = 32                                          # the copy's struct is its own
    assert fields(d.c_ref())["head_dim"] == 32 and fields(c.c_ref()) == want


def test_the_struct_follows_fields_and_planes():
    c = cache(Plane)
    a = fields(c.c_ref())
    c.k.at = 0x70000                                         # a plane that was given other storage
    assert fields(c.c_ref()) == {**a, "k": 0x70000}
    c.k = Plane(0x80000)
    c.capacity = np.asarray([50, 40], np.int32)
    assert fields(c.c_ref()) == {**a, "k": 0x80000, "capacity": [50, 40]}
    c.capacity[0] = 7                                        # in place
    assert fields(c.c_ref())["capacity"] == [7, 40]


@pytest.mark.parametrize("name", ["k", "v", "pos", "n_live", "k_scale", "v_scale"])
def test_a_plane_restrided_in_place_is_refused(name):
    """At the address that it had, as torch's transpose_ or as_strided_ leave it."""
    c = cache(Plane)
    c.c_ref()
    getattr(c, name).contiguous = False
    with pytest.raises(ValueError):
        c.c_ref()
    getattr(c, name).contiguous = True
    c.c_ref()
