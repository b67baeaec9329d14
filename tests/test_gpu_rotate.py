"""tria_rotate and tria_append_qkv against 64 bits: layouts, scaled
frequencies, partial heads, strides, far positions; the rows that land in the
cache, their types, what stays untouched, and the errors a device finds."""
import numpy as np
import pytest

import _rows as R
from oracle import attend_oracle as A

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

SCALINGS = [dict(), dict(scaling="linear", factor=4.0), dict(scaling="ntk", factor=2.5),
            dict(scaling="yarn", factor=4.0, orig_ctx=32768), dict(scaling="bands", factor=8.0, orig_ctx=8192)]


def turn_tolerance(x, norm, mscale, kind, want):
    """fp32 steps: the sum of squares of 16 values a lane and 4 shuffles (20 roundings, halved by the root), root, two
    products (17 in all with the division); the phase is off by half a turn x 2^-24 (pi 2^-24) and the sine by two
    more, mscale one, the rotation three: 27 x 2^-24 of the pair's length, sqrt(2) for its two members; 40 covers it.
    The result is rounded once."""
    x = np.abs(np.asarray(x, np.float64))
    if norm is not None:
        x = x / np.sqrt((x * x).mean(-1, keepdims=True) + 1e-6) * np.abs(norm)
    size = x.max(-1, keepdims=True) * mscale
    return 40 * R.U24 * 1.5 * size + R.HALF_STEP[kind] * np.abs(want) * 1.001 + 2.0 ** -25


@pytest.mark.parametrize("layout", ["half", "interleaved", "interleaved_to_half"])
@pytest.mark.parametrize("hd,nonrot", [(128, 0), (64, 32), (96, 0), (256, 64), (32, 16), (224, 0)])
@pytest.mark.parametrize("kind", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("norm", [True, False])
def test_rotate(lib, layout, hd, nonrot, kind, norm):
    rng = np.random.default_rng(hd)
    for i, sc in enumerate(SCALINGS):
        n, hq, hk = (1, 7, 33, 2, 5)[i], (8, 5, 32, 1, 3)[i], (2, 1, 8, 1, 3)[i]
        rope = lib.Rope(head_dim=hd, nonrot_dim=nonrot, theta=1e6, layout=layout, **sc)
        w, m = A.frequencies(hd, 1e6, nonrot, **{**dict(scaling="none"), **sc})
        joint = R.act(rng.standard_normal((n, hq + 2 * hk, hd)) * 2, kind)      # a joint projection's slices
        pos = rng.integers(0, 200000, n).astype(np.int32)
        wt = [(1 + 0.3 * rng.standard_normal(hd)).astype(np.float32) if norm else None for _ in range(2)]
        parts, outs = [], []
        for x, g in ((joint[:, :hq], wt[0]), (joint[:, hq:hq + hk], wt[1])):
            o = torch.full((n, x.shape[1] + 1, hd), 9.0, device="cuda", dtype=x.dtype)
            outs.append(o)
            parts.append((x, o[:, :x.shape[1]], None if g is None else torch.from_numpy(g).cuda()))
        before = joint.clone()
        lib.rotate(rope, parts, torch.from_numpy(pos).cuda())
        assert torch.equal(joint, before)
        for (x, o, _), g, whole in zip(parts, wt, outs):
            want = A.turn(R.host(x), pos, w, m, nonrot, layout, g)
            assert np.all(np.abs(R.host(o) - want) <= turn_tolerance(R.host(x), g, m, kind, want))
            assert (whole[:, -1] == 9).all()
        # in place
        for x, _, g in parts:
            want = torch.empty_like(x.contiguous())
            lib.rotate(rope, [(x, want, g)], torch.from_numpy(pos).cuda())
            y = x.contiguous().clone()
            lib.rotate(rope, [(y, y, g)], torch.from_numpy(pos).cuda())
            assert torch.equal(y, want)
        rope.close()


def test_rotate_far_positions_and_given_frequencies(lib):
    """Positions up to 2^31 - 1 keep their phase (exact integer phase arithmetic), and negative ones turn back."""
    w = np.array([1.0, 0.37, 1e-3, 2.5e-7] * 8)
    rope = lib.Rope(head_dim=64, omega=w, mscale=0.5)
    pos = np.array([0, 1, 2 ** 20 + 3, 2 ** 31 - 1, -5, -(2 ** 30)], np.int32)
    x = np.zeros((6, 1, 64), np.float32)
    x[..., :32] = 1.0
    t = R.act(x, "f32")
    out = torch.empty_like(t)
    lib.rotate(rope, [(t, out, None)], torch.from_numpy(pos).cuda())
    # the phase in exact integers: w / 2 pi to 64 bits of a turn, as the frequencies are held
    turns = [int((v / (2 * np.pi)) % 1.0 * 2.0 ** 64) for v in w]
    ang = np.array([[(tt * int(p)) % 2 ** 64 / 2.0 ** 64 * 2 * np.pi for tt in turns] for p in pos])
    want = 0.5 * np.concatenate([np.cos(ang), np.sin(ang)], -1)[:, None]
    assert np.all(np.abs(R.host(out) - want) <= 40 * R.U24)


def test_scaled_rotation_is_the_scorers(lib):
    """tria_rope_frequencies gives the omega that tria_load_stats takes, and rotates by it."""
    for sc in SCALINGS:
        w, m = lib.rope_frequencies(head_dim=128, theta=1e6, **sc)
        a, am = A.frequencies(128, 1e6, 0, **{**dict(scaling="none"), **sc})
        np.testing.assert_allclose(w, a, rtol=1e-13)
        assert abs(m - am) < 1e-13
        x = R.act(np.random.default_rng(1).standard_normal((3, 2, 128)), "f32")
        pos = torch.tensor([5, 100, 100000], device="cuda", dtype=torch.int32)
        o = [torch.empty_like(x) for _ in range(2)]
        lib.rotate(lib.Rope(head_dim=128, theta=1e6, **sc), [(x, o[0], None)], pos)
        lib.rotate(lib.Rope(head_dim=128, omega=w, mscale=m), [(x, o[1], None)], pos)
        assert torch.equal(*o)


CASES = [dict(hd=128, n_kv=8, nq=32, k="q8_0", v="q8_0", kind="f16", tokens=[1], rows=[100]),
         dict(hd=128, n_kv=2, nq=8, k="q4_0", v="q4_0", kind="bf16", tokens=[1, 1, 1], rows=[0, 5, 63]),
         dict(hd=64, n_kv=3, nq=3, k="f16", v="q4_0", kind="f32", tokens=[0, 40, 3], rows=[7, 0, 31]),
         dict(hd=96, n_kv=1, nq=8, k="q4_0", v="f16", kind="f16", tokens=[5, 0], rows=[2, 2], nonrot=48),
         dict(hd=256, n_kv=4, nq=0, k="q8_0", v="f32", kind="bf16", tokens=[3, 2], rows=[1, 17], layout="interleaved_to_half"),
         dict(hd=32, n_kv=2, nq=4, k="f32", v="q8_0", kind="f32", tokens=[300], rows=[11], nonrot=16),
         dict(hd=160, n_kv=1, nq=1, k="f16", v="f16", kind="bf16", tokens=[2, 9, 1], rows=[3, 3, 3])]


@pytest.mark.parametrize("case", CASES)
@pytest.mark.parametrize("norm,given", [(True, False), (False, True)])
def test_append_qkv(lib, case, norm, given):
    hd, n_kv, nq, kind = case["hd"], case["n_kv"], case["nq"], case["kind"]
    nonrot, layout = case.get("nonrot", 0), case.get("layout", "half")
    rng = np.random.default_rng(hd)
    tokens, rows = case["tokens"], case["rows"]
    c = R.Cache(lib, rng, rows=rows, cap=[r + t + 2 for r, t in zip(rows, tokens)], n_kv=n_kv, hd=hd, k_type=case["k"],
                v_type=case["v"])
    n = sum(tokens)
    tok0 = np.concatenate([[0], np.cumsum(tokens)]).astype(np.int32)
    joint = R.act(rng.standard_normal((n, nq + 2 * n_kv, hd)), kind)
    if n:
        joint[0, nq + n_kv, :32] = 0                       # a block of zeros
        joint[-1, nq + n_kv, 3], joint[-1, nq + n_kv, 19] = 6.0, -6.0    # two values of the largest modulus
    q, k, v = joint[:, :nq], joint[:, nq:nq + n_kv], joint[:, nq + n_kv:]
    wq, wk = [(1 + 0.3 * rng.standard_normal(hd)).astype(np.float32) if norm else None for _ in range(2)]
    pos = np.concatenate([c.last(s) + 1 + np.arange(t) for s, t in enumerate(tokens)] + [[]]).astype(np.int32)
    rope = lib.Rope(head_dim=hd, nonrot_dim=nonrot, theta=1e4, layout=layout)
    w, m = A.frequencies(hd, 1e4, nonrot)
    q_out = torch.zeros(n, nq, hd, device="cuda", dtype=joint.dtype) if nq else None
    k_held, v_held = (torch.zeros(n, n_kv, hd, device="cuda", dtype=joint.dtype) for _ in range(2))
    ws = c.ws(lib.workspace_size(c.cache, 0))
    kw = {}
    if given:                                              # the rows before the call are the caller's
        kw["n_before"] = torch.tensor(rows, device="cuda", dtype=torch.int32)
        c.d["n_live"].fill_(1)
    dev = lambda a: None if a is None else torch.from_numpy(a).cuda()  # noqa: E731
    for _ in range(2 if given else 1):                     # a step taken again writes the same rows
        lib.append_qkv(rope, c.cache, q if nq else None, k, v, torch.from_numpy(pos).cuda(), q_out=q_out, tok0=tok0,
                       q_norm=dev(wq), k_norm=dev(wk), k_held=k_held, v_held=v_held, ws=ws, **kw)
    assert lib.device_status(ws) == lib.OK
    assert c.d["n_live"].tolist() == [r + t for r, t in zip(rows, tokens)]
    if nq:
        want = A.turn(R.host(q), pos, w, m, nonrot, layout, wq)
        assert np.all(np.abs(R.host(q_out) - want) <= turn_tolerance(R.host(q), wq, m, kind, want))
    got = {name: None if t is None else t.cpu().numpy() for name, t in c.d.items()}
    want_k = A.turn(R.host(k), pos, w, m, nonrot, layout, wk)
    off_k = turn_tolerance(R.host(k), wk, m, "f32", want_k)
    touched = np.zeros(len(got["pos"]), bool)
    for s, t in enumerate(tokens):
        for g in range(n_kv):
            r0 = c.row0[s] + g * c.cap[s] + rows[s]
            sl, tk = slice(r0, r0 + t), slice(tok0[s], tok0[s + 1])
            touched[sl] = True
            np.testing.assert_array_equal(got["pos"][sl], pos[tk])
            # values come as they are: the same fp32 steps give the same codes and scales
            data, scale = A.hold(R.host(v)[tk, g].astype(np.float32), case["v"])
            np.testing.assert_array_equal(got["v"][sl], data)
            if scale is not None:
                np.testing.assert_array_equal(got["v_scale"][sl], scale)
            held = A.values(got["v"][sl], None if scale is None else got["v_scale"][sl], case["v"])
            assert np.all(np.abs(R.host(v_held)[tk, g] - held) <= R.HALF_STEP[kind] * np.abs(held) + 2.0 ** -25)
            kk, kd = want_k[tk, g], off_k[tk, g]
            held = A.values(got["k"][sl], None if c.k_type[0] == "f" else got["k_scale"][sl], case["k"])
            assert np.all(np.abs(R.host(k_held)[tk, g] - held) <= R.HALF_STEP[kind] * np.abs(held) + 2.0 ** -25)
            if case["k"][0] == "f":
                step = R.HALF_STEP[case["k"]]
                assert np.all(np.abs(held - kk) <= kd + step * (np.abs(kk) + kd) * 1.001 + 2.0 ** -25)
                continue
            # the block's scale within its own rounding, the value within half a code of it (q4_0's top code is cut
            # half a code early: code 16 does not exist)
            b = np.abs(kk).reshape(t, hd // 32, 32).max(-1)
            lv = 127 if case["k"] == "q8_0" else 8
            e = kd.max(initial=0)
            sc = np.abs(got["k_scale"][sl].astype(np.float64))
            assert np.all(np.abs(sc - b / lv) <= (b / lv + e) * R.U16 * 1.001 + e / lv + 2.0 ** -25)
            step = np.repeat(b / lv + e, 32, -1)
            room = step * (0.5 if lv == 127 else 1.0) + e + step * lv * R.U16 * 1.01 + 2.0 ** -20
            assert np.all(np.abs(held - kk) <= room)
            if lv == 8:                                    # all but the cut ones within half a code
                codes = A.codes_q4_0(got["k"][sl])
                assert np.all((np.abs(held - kk) <= step * 0.5 + e + step * lv * R.U16 * 1.01 + 2.0 ** -20) | (codes == 15))
    for name in ("k", "v", "k_scale", "v_scale", "pos"):   # every other row as it was
        if got[name] is not None:
            assert got[name][~touched].tobytes() == c.h[name][~touched].tobytes(), name


def test_append_that_does_not_fit(lib):
    """A sequence without room and one with a bad count are left alone and reported; the others are appended."""
    rng = np.random.default_rng(3)
    for rows, code in (([6, 9], "ERR_CAPACITY"), ([6, 11], "ERR_DEVICE_ARG")):
        c = R.Cache(lib, rng, rows=[6, 9], cap=[10, 10], n_kv=2, hd=64, k_type="q8_0", v_type="f16")
        c.d["n_live"].copy_(torch.tensor(rows, dtype=torch.int32))
        x = R.act(rng.standard_normal((4, 2, 64)), "f16")
        pos = torch.tensor([100, 101, 100, 101], device="cuda", dtype=torch.int32)
        ws = c.ws(lib.workspace_size(c.cache, 0))
        lib.append_qkv(lib.Rope(head_dim=64, theta=1e4), c.cache, None, x, x, pos, ws=ws)
        assert lib.device_status(ws) == getattr(lib, code)
        assert c.d["n_live"].tolist() == [8, rows[1]]
        r = c.row0[1]
        for name in ("k", "v", "k_scale", "pos"):
            assert c.d[name][r:].cpu().numpy().tobytes() == c.h[name][r:].tobytes()
        assert (c.d["pos"][c.row0[0] + 6:c.row0[0] + 8].cpu() == torch.tensor([100, 101])).all()


def test_append_qkv_equals_append_of_ready_rows(lib):
    """The rows that tria_append_qkv makes are those that tria_append copies when it is given the same values."""
    rng = np.random.default_rng(4)
    for kt, vt in (("q8_0", "q4_0"), ("q4_0", "f16"), ("f16", "q8_0")):
        c = R.Cache(lib, rng, rows=[3, 0], cap=[12, 8], n_kv=2, hd=64, k_type=kt, v_type=vt)
        d = R.Cache(lib, np.random.default_rng(0), rows=[3, 0], cap=[12, 8], n_kv=2, hd=64, k_type=kt, v_type=vt)
        for name, t in c.d.items():
            if t is not None:
                d.d[name].copy_(t)
        k, v = (R.act(rng.standard_normal((10, 2, 64)), "f32") for _ in range(2))
        pos = torch.tensor(list(range(20, 25)) * 2, device="cuda", dtype=torch.int32)
        ws = c.ws(lib.workspace_size(c.cache, 0))
        rope = lib.Rope(head_dim=64, theta=1e4)
        lib.append_qkv(rope, c.cache, None, k, v, pos, ws=ws)
        turned = torch.empty_like(k)
        lib.rotate(rope, [(k, turned, None)], pos)
        new = {}
        for name, x, kind in (("k", turned, kt), ("v", v, vt)):
            data, scale = A.hold(x.cpu().numpy().reshape(2, 5, 2, 64).transpose(0, 2, 1, 3), kind)
            new[name] = torch.from_numpy(np.ascontiguousarray(data)).cuda()
            new[name + "_scale"] = None if scale is None else torch.from_numpy(np.ascontiguousarray(scale)).cuda()
        lib.append(d.cache, new["k"], new["v"], pos.reshape(2, 5), ws=ws, k_scale_new=new["k_scale"], v_scale_new=new["v_scale"])
        for name, t in c.d.items():
            if t is not None:
                assert t.cpu().numpy().tobytes() == d.d[name].cpu().numpy().tobytes(), (kt, vt, name)


@pytest.mark.parametrize("kt", ["q8_0", "q4_0"])
@pytest.mark.parametrize("at", [0, 15, 16, 31])
def test_a_nan_reaches_its_block(lib, kt, at):
    """A quantised block with a NaN reads as NaN in all of its values, in the cache and in what is held; the other
    blocks are what they are without it."""
    rng = np.random.default_rng(5)
    x = rng.standard_normal((3, 2, 64)).astype(np.float32)
    held = []
    for bad in (False, True):
        y = x.copy()
        if bad:
            y[1, 1, 32 + at] = np.nan
        c = R.Cache(lib, np.random.default_rng(0), rows=[2], cap=[8], n_kv=2, hd=64, k_type=kt, v_type=kt)
        kh, vh = (torch.empty(3, 2, 64, device="cuda") for _ in range(2))
        pos = torch.tensor([50, 51, 52], device="cuda", dtype=torch.int32)
        ws = c.ws(lib.workspace_size(c.cache, 0))
        still = lib.Rope(head_dim=64, nonrot_dim=32, omega=[0.0] * 16)   # (a rotated NaN would reach its pair)
        lib.append_qkv(still, c.cache, None, R.act(y, "f32"), R.act(y, "f32"), pos, ws=ws, k_held=kh, v_held=vh)
        assert lib.device_status(ws) == lib.OK
        cached = []
        for name in ("k", "v"):
            rows = np.stack([np.arange(3) + c.row0[0] + g * 8 + 2 for g in range(2)], 1)
            cached.append(A.values(c.d[name].cpu().numpy()[rows], c.d[name + "_scale"].cpu().numpy()[rows], kt))
        held.append([R.host(kh), R.host(vh)] + cached)
    hurt = np.zeros(x.shape, bool)
    hurt[1, 1, 32:] = True
    for clean, got in zip(*held):
        assert np.isnan(got[hurt]).all() and np.array_equal(got[~hurt], clean[~hurt])
    assert np.array_equal(held[1][0], held[1][2], equal_nan=True) and np.array_equal(held[1][1], held[1][3], equal_nan=True)
