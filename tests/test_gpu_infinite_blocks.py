"""Infinities that tria_append_qkv quantises: what the cache reads as, and what is given out as held."""
import numpy as np
import pytest

import _rows as R
from oracle import attend_oracle as A

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")


@pytest.mark.parametrize("kind", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("kt", ["q8_0", "q4_0"])
@pytest.mark.parametrize("where", [{0: np.inf}, {15: -np.inf}, {16: np.inf, 31: -np.inf}, {3: -np.inf, 20: np.inf, 21: -np.inf},
                                   {1: np.inf, 2: np.inf}])
def test_a_block_with_infinities(lib, kt, kind, where):
    """Its values read as NaN, the other blocks as they are without it; the held values are those that the cache's codes
    and scales stand for."""
    x = np.random.default_rng(5).standard_normal((3, 2, 64)).astype(np.float32)
    held = []
    for bad in (False, True):
        y = x.copy()
        if bad:
            for at, value in where.items():
                y[1, 1, 32 + at] = value
        c = R.Cache(lib, np.random.default_rng(0), rows=[2], cap=[8], n_kv=2, hd=64, k_type=kt, v_type=kt)
        new = R.act(y, kind)
        kh, vh = (torch.empty_like(new) for _ in range(2))
        pos = torch.tensor([50, 51, 52], device="cuda", dtype=torch.int32)
        ws = c.ws(lib.workspace_size(c.cache, 0))
        still = lib.Rope(head_dim=64, nonrot_dim=32, omega=[0.0] * 16)   # (a rotated infinity would reach its pair)
        lib.append_qkv(still, c.cache, None, new, new, pos, ws=ws, k_held=kh, v_held=vh)
        assert lib.device_status(ws) == lib.OK
        cached = []
        for name in ("k", "v"):
            rows = np.stack([np.arange(3) + c.row0[0] + g * 8 + 2 for g in range(2)], 1)
            with np.errstate(invalid="ignore"):
                cached.append(A.values(c.d[name].cpu().numpy()[rows], c.d[name + "_scale"].cpu().numpy()[rows], kt))
        held.append([R.host(kh), R.host(vh)] + cached)
    hurt = np.zeros(x.shape, bool)
    hurt[1, 1, 32:] = True
    for clean, got in zip(*held):
        assert np.isnan(got[hurt]).all() and np.array_equal(got[~hurt], clean[~hurt])
    for h, cc in zip(held[1][:2], held[1][2:]):              # (held values of 16 bits are rounded once)
        np.testing.assert_allclose(h, cc, rtol=R.HALF_STEP[kind], atol=2.0 ** -25)
