"""tria_reorder over layers that lie side by side in one array per plane, so that
a layer's scales start anywhere; and over large groups of them."""
import numpy as np
import pytest

import _rows as R
from oracle import beam_oracle as B

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")


@pytest.mark.parametrize("hd,k,v", [(32, "q8_0", "q4_0"), (64, "q4_0", "q8_0"), (96, "q8_0", "q8_0"), (128, "q8_0", "f16"), (160, "f16", "q4_0"),
                                    (256, "q4_0", "q4_0")])
@pytest.mark.parametrize("beams,n_kv,cap", [(3, 1, 31), (5, 3, 63), (9, 1, 129)])
def test_layers_side_by_side(lib, hd, k, v, beams, n_kv, cap):
    rng = np.random.default_rng(hd + beams)
    n_layers, rows = 4, [int(x) for x in rng.integers(1, cap + 1, beams)]
    made = [R.Cache(lib, rng, rows=rows, cap=[cap] * beams, n_kv=n_kv, hd=hd, k_type=k, v_type=v, guard=0) for _ in range(n_layers)]
    c0 = made[0]
    total = beams * n_kv * cap
    host = {name: np.stack([c.h[name][:total] if name != "n_live" else c.h[name] for c in made]) for name, a in c0.h.items() if a is not None}
    dev = {name: torch.from_numpy(a.copy()).cuda() for name, a in host.items()}
    view = lambda name, l: dev[name][l] if name in dev else None
    caches = [lib.LayerCache(k=view("k", l), v=view("v", l), k_scale=view("k_scale", l), v_scale=view("v_scale", l), pos=view("pos", l),
                             n_live=view("n_live", l), seq_row0=c0.row0, capacity=c0.cap, head_dim=hd, n_kv_heads=n_kv, k_type=k, v_type=v)
              for l in range(n_layers)]
    ws = c0.ws(lib.reorder_workspace_size(caches))
    for parent in (np.roll(np.arange(beams), 1), np.maximum(np.arange(beams) - 1, 0), rng.integers(0, beams, beams), rng.permutation(beams)):
        lib.reorder(caches, torch.from_numpy(parent.astype(np.int32)).cuda(), ws=ws)
        assert lib.device_status(ws) == lib.OK
        for l in range(n_layers):
            planes = {name: a[l].view(np.uint8 if name != "pos" else np.int32) for name, a in host.items() if name != "n_live"}
            want, n = B.reorder(planes, host["n_live"][l], parent, c0.row0, c0.cap, n_kv)
            assert np.array_equal(dev["n_live"][l].cpu().numpy(), n)
            for name, a in want.items():
                got = dev[name][l].cpu().numpy()
                assert np.array_equal(got.view(a.dtype), a), name
                host[name][l] = got
            host["n_live"][l] = n
