"""tria_reorder: bit for bit what moving the rows one by one gives, for maps of
every kind, ragged rows, every type, several layers, and the calls that leave
a group as it was."""
import numpy as np
import pytest

import _rows as R
from oracle import beam_oracle as B

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")
PLANES = ("k", "k_scale", "v", "v_scale", "pos")


def layers(lib, rng, n, rows, cap, n_kv, hd, k, v):
    return [R.Cache(lib, rng, rows=rows, cap=cap, n_kv=n_kv, hd=hd, k_type=k, v_type=v) for _ in range(n)]


def state(c):
    return {k: c.d[k].view(torch.uint8 if k != "pos" else torch.int32).cpu().numpy() for k in PLANES if c.d[k] is not None}, \
        c.d["n_live"].cpu().numpy()


def move(lib, cs, parent, seq0, ws=None, code=0, kept=()):
    """reorder(), checked; kept: groups that must stay as they are."""
    before = [state(c) for c in cs]
    if ws is None:
        ws = cs[0].ws(lib.reorder_workspace_size([c.cache for c in cs], seq0))
    lib.reorder([c.cache for c in cs], torch.tensor(np.asarray(parent), device="cuda", dtype=torch.int32), seq0=seq0, ws=ws)
    assert lib.device_status(ws) == code
    p = np.array(parent)
    for g in kept:
        p[seq0[g]:seq0[g + 1]] = np.arange(seq0[g], seq0[g + 1])
    for c, (planes, live) in zip(cs, before):
        use = np.where(live < 0, 0, live)
        want, n = B.reorder(planes, np.minimum(use, c.cap), p, c.row0, c.cap, c.n_kv)
        for g in kept:
            n[seq0[g]:seq0[g + 1]] = live[seq0[g]:seq0[g + 1]]
        got, got_n = state(c)
        assert np.array_equal(n, got_n)
        for k in planes:
            assert np.array_equal(got[k], want[k]), k


def maps(rng, n):
    yield np.arange(n)                                        # nobody moves
    yield np.zeros(n, int)                                    # one parent for all
    yield np.roll(np.arange(n), 1)                            # one ring
    yield np.arange(n)[::-1].copy()                                # pairs change places
    yield np.maximum(np.arange(n) - 1, 0)                     # a chain
    yield rng.permutation(n)
    for _ in range(3):
        yield rng.integers(0, n, n)


@pytest.mark.parametrize("k,v", [("f16", "f16"), ("q8_0", "q8_0"), ("q4_0", "q8_0"), ("f32", "q4_0")])
@pytest.mark.parametrize("hd", [32, 64, 96, 128, 160, 256])
def test_types_and_head_dims(lib, k, v, hd):
    rng = np.random.default_rng(hd)
    for parent in ([0, 0, 0, 1], [3, 2, 1, 0], [1, 2, 3, 0]):
        move(lib, layers(lib, rng, 2, [37, 70, 5, 64], [70] * 4, 3, hd, k, v), parent, [0, 4])


@pytest.mark.parametrize("beams", [1, 2, 3, 4, 5, 8, 9, 17, 32])
def test_maps(lib, beams):
    rng = np.random.default_rng(beams)
    rows = [int(x) for x in rng.integers(0, 90, beams)]
    for parent in maps(rng, beams):
        move(lib, layers(lib, rng, 1, rows, [90 + s % 3 for s in range(beams)], 2, 64, "f16", "q8_0"), parent, [0, beams])


@pytest.mark.parametrize("n_layers", [1, 5, 40])
def test_several_groups_and_layers(lib, n_layers):
    """Ragged groups, one of them without sequences; layers of different lengths."""
    rng = np.random.default_rng(n_layers)
    seq0 = [0, 4, 4, 5, 17, 24]
    cs = layers(lib, rng, n_layers, [1] * 24, [130] * 24, 2, 64, "q8_0", "f16")
    for i, c in enumerate(cs):
        c.d["n_live"].copy_(torch.from_numpy(np.random.default_rng(i).integers(0, 131, 24).astype(np.int32)))
    ws = cs[0].ws(256)
    for _ in range(3):                                        # one workspace, one call after another
        parent = np.concatenate([a + rng.integers(0, b - a, b - a) for a, b in zip(seq0, seq0[1:]) if b > a])
        move(lib, cs, parent, seq0, ws=ws)


def test_many_groups_take_several_launches(lib):
    """128 groups of a sequence and more layers than one launch's table holds; of 64 pairs, every other one changes places."""
    rng = np.random.default_rng(1)
    cs = layers(lib, rng, 18, [3] * 128, [4] * 128, 1, 32, "f16", "f16")
    move(lib, cs, np.arange(128), np.arange(129))
    parent = np.arange(128).reshape(64, 2)
    parent[::2] = parent[::2, ::-1].copy()
    cs = layers(lib, rng, 40, [3] * 128, [4] * 128, 1, 32, "f16", "f16")
    move(lib, cs, parent.reshape(-1), np.arange(65) * 2)


def test_long_rows(lib):
    rng = np.random.default_rng(2)
    move(lib, layers(lib, rng, 1, [9000, 5, 8191, 0, 4097, 1], [9000] * 6, 2, 128, "q4_0", "q8_0"), [0, 0, 4, 2, 4, 2], [0, 6])


def test_refused_groups_stay(lib):
    rng = np.random.default_rng(3)
    D, C = lib.ERR_DEVICE_ARG, lib.ERR_CAPACITY
    seq0 = [0, 3, 6]
    for parent in ([1, 3, 0, 3, 3, 4], [1, -1, 0, 3, 3, 4], [1, 1 << 30, 0, 3, 3, 4], [1, -(1 << 31), 0, 3, 3, 4]):
        move(lib, layers(lib, rng, 2, [7] * 6, [9] * 6, 2, 64, "f16", "f16"), parent, seq0, code=D, kept=[0])
    for bad in (-1, 10):
        cs = layers(lib, rng, 2, [7] * 6, [9] * 6, 2, 64, "f16", "f16")
        for c in cs:
            c.d["n_live"][4] = bad
        move(lib, cs, [1, 2, 0, 3, 3, 5], seq0, code=D, kept=[1])
    cs = layers(lib, rng, 2, [7, 3, 2, 7, 3, 3], [9, 9, 9, 9, 9, 5], 2, 64, "f16", "f16")
    move(lib, cs, [1, 2, 0, 4, 5, 3], seq0, code=C, kept=[1])
    ws = cs[0].ws(256)
    move(lib, cs, [1, 2, 0, 3, 5, 4], seq0, ws=ws)            # the longer one stays: it fits


def test_captured_and_replayed(lib):
    rng = np.random.default_rng(4)
    cs = layers(lib, rng, 3, [20] * 8, [40] * 8, 2, 64, "f16", "f16")
    ws, parent = cs[0].ws(256), torch.arange(8, device="cuda", dtype=torch.int32)
    lib.reorder([c.cache for c in cs], parent, ws=ws)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        lib.reorder([c.cache for c in cs], parent, ws=ws)
    for _ in range(4):
        for c in cs:
            c.d["n_live"].copy_(torch.from_numpy(rng.integers(0, 41, 8).astype(np.int32)))
        p = rng.integers(0, 8, 8)
        parent.copy_(torch.from_numpy(p.astype(np.int32)))
        before = [state(c) for c in cs]
        g.replay()
        for c, (planes, live) in zip(cs, before):
            want, n = B.reorder(planes, live, p, c.row0, c.cap, c.n_kv)
            got, got_n = state(c)
            assert np.array_equal(n, got_n) and all(np.array_equal(got[k], want[k]) for k in planes)
