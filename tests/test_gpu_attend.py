"""tria_attend against attention in 64 bits: types, head layouts, lengths from
none to long, windows with first rows that stay visible, masks that leave a
token nothing, junk in rows that no token sees, split and joined units."""
import numpy as np
import pytest

import _rows as R

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")


def run(lib, c, nq, kind, tokens, *, window=0, sink=0, scale=None, seed=0, heat=1.0, back=0, junk=None, ws=None, stride=0):
    """tokens[s] new tokens of sequence s, the newest ones (`back` positions earlier), checked against 64 bits."""
    rng = np.random.default_rng(seed + 1)
    tok0 = np.concatenate([[0], np.cumsum(tokens)]).astype(np.int32)
    n = int(tok0[-1])
    pos = np.concatenate([c.last(s) - back - np.arange(t)[::-1] for s, t in enumerate(tokens)] + [[]]).astype(np.int32)
    wide = R.act(rng.standard_normal((n, nq + stride, c.hd)) * heat, kind)
    q = wide[:, :nq]
    out = torch.full((n + 1, nq, c.hd), 7.0, device="cuda", dtype=q.dtype)
    lse = torch.full((n + 1, nq), 7.0, device="cuda")
    if ws is None:
        ws = c.ws(lib.attend_workspace_size(c.cache, nq, tok0))
    lib.attend(c.cache, q, out[:n], torch.from_numpy(pos).cuda(), tok0=tok0, lse=lse[:n], window=window, sink=sink,
               scale=scale or 0.0, ws=ws)
    assert lib.device_status(ws) == lib.OK
    assert (out[n] == 7).all() and (lse[n] == 7).all()
    if n == 0:
        return out, lse
    want = R.attend_expected(c, R.host(q), pos, tok0, nq, window, sink, scale)
    tensor = kind != "f32" and "f32" not in (c.k_type, c.v_type)
    R.check_attend(R.host(out[:n]), R.host(lse[:n]), want, kind, tensor, max(c.rows), c.hd,
                   q_exact=kind == "f16", k_exact=c.k_type == "f16")
    return out, lse


TYPES = [("f16", "f16", "f16"), ("bf16", "f16", "f16"), ("f16", "q8_0", "q8_0"), ("bf16", "q4_0", "q4_0"),
         ("f16", "q8_0", "q4_0"), ("f16", "q4_0", "f16"), ("f16", "f16", "q8_0"), ("f32", "f32", "f32"),
         ("f32", "q4_0", "q8_0"), ("f16", "f32", "f16"), ("bf16", "f16", "f32")]


@pytest.mark.parametrize("kind,k,v", TYPES)
@pytest.mark.parametrize("hd,n_kv,group", [(64, 2, 4), (128, 2, 4), (256, 1, 2)])
def test_single_tokens(lib, kind, k, v, hd, n_kv, group):
    rng = np.random.default_rng(hd + group)
    c = R.Cache(lib, rng, rows=[1, 33, 700, 17, 128], cap=[5, 33, 701, 40, 130], n_kv=n_kv, hd=hd, k_type=k, v_type=v)
    run(lib, c, n_kv * group, kind, [1] * 5)


@pytest.mark.parametrize("hd,n_kv,group", [(32, 3, 1), (96, 1, 8), (160, 2, 3), (192, 1, 5), (224, 1, 6), (128, 2, 7), (64, 1, 1),
                                           (256, 2, 8)])
@pytest.mark.parametrize("kind,k,v", [("f16", "f16", "f16"), ("bf16", "q4_0", "q8_0")])
def test_head_shapes(lib, kind, k, v, hd, n_kv, group):
    rng = np.random.default_rng(hd)
    c = R.Cache(lib, rng, rows=[260, 3], cap=[261, 9], n_kv=n_kv, hd=hd, k_type=k, v_type=v)
    run(lib, c, n_kv * group, kind, [1, 1])
    run(lib, c, n_kv * group, kind, [5, 3], stride=3)


@pytest.mark.parametrize("tokens", [[0, 1, 4], [2, 2, 2], [3, 0, 0], [0, 0, 0], [1, 9, 40], [17, 1, 65]])
@pytest.mark.parametrize("kind,k,v", [("f16", "f16", "f16"), ("f16", "q8_0", "q4_0"), ("f32", "f32", "f32")])
def test_several_tokens_causal(lib, kind, k, v, tokens):
    rng = np.random.default_rng(5)
    c = R.Cache(lib, rng, rows=[40, 300, 90], cap=[41, 300, 95], n_kv=2, hd=64, k_type=k, v_type=v)
    run(lib, c, 8, kind, tokens)


@pytest.mark.parametrize("window,sink", [(1, 0), (16, 4), (100, 1), (100, 200), (4096, 3), (37, 50)])
@pytest.mark.parametrize("tokens", [1, 2, 21])
@pytest.mark.parametrize("kind,k,v,hd", [("f16", "f16", "f16", 128), ("bf16", "q8_0", "q4_0", 64), ("f32", "f32", "f32", 64)])
def test_window_and_first_rows(lib, kind, k, v, hd, tokens, window, sink):
    rng = np.random.default_rng(window)
    c = R.Cache(lib, rng, rows=[513, 60, 22], cap=[520, 61, 22], n_kv=2, hd=hd, k_type=k, v_type=v)
    run(lib, c, 8, kind, [tokens] * 3, window=window, sink=sink)


@pytest.mark.parametrize("kind,k,v", [("f16", "f16", "f16"), ("f32", "f32", "f32"), ("f16", "q8_0", "q8_0")])
@pytest.mark.parametrize("tokens", [1, 3, 20])
def test_tokens_that_see_nothing(lib, kind, k, v, tokens):
    """Queries before every row, queries in the middle of the rows, a sequence without rows."""
    rng = np.random.default_rng(9)
    c = R.Cache(lib, rng, rows=[50, 0, 200], cap=[50, 8, 201], n_kv=2, hd=64, k_type=k, v_type=v)
    out, lse = run(lib, c, 4, kind, [tokens] * 3, back=10000)
    assert (out[:3 * tokens] == 0).all() and torch.isinf(lse[:3 * tokens]).all()
    run(lib, c, 4, kind, [tokens] * 3, back=100, window=30, sink=2)
    run(lib, c, 4, kind, [tokens] * 3, back=333)


@pytest.mark.parametrize("kind,k,v", [("f16", "f16", "f16"), ("f32", "f32", "f32"), ("bf16", "q8_0", "q4_0")])
@pytest.mark.parametrize("tokens", [1, 4, 40])
@pytest.mark.parametrize("bad", [np.nan, np.inf, -np.inf])
@pytest.mark.parametrize("edge", [0, 1])
def test_junk_in_hidden_rows(lib, kind, k, v, tokens, bad, edge):
    """Rows outside the window and a row newer than every token hold NaN or infinities; with edge = 0 so does the
    oldest row of the first token's window, which that token alone sees."""
    rng = np.random.default_rng(11)
    c = R.Cache(lib, rng, rows=[300], cap=[300], n_kv=1, hd=64, k_type=k, v_type=v, gaps=False)
    hidden = list(range(7, 300 - tokens - 63 - edge)) + [299]
    for r in hidden:
        for name in ("k", "v"):
            a = c.h[name] if c.h[name].dtype.kind == "f" else c.h[name + "_scale"]
            a[c.row0[0] + r] = bad
    c.d = {n: torch.from_numpy(a.copy()).cuda() if a is not None else None for n, a in c.h.items()}
    c.cache.k, c.cache.v, c.cache.k_scale, c.cache.v_scale = c.d["k"], c.d["v"], c.d["k_scale"], c.d["v_scale"]
    rng2 = np.random.default_rng(3)
    q = R.act(rng2.standard_normal((tokens, 4, 64)), kind)
    out, lse = torch.zeros_like(q), torch.zeros(tokens, 4, device="cuda")
    pos = np.arange(300 - tokens, 300, dtype=np.int32) - 1   # the last token stands before the newest row
    ws = c.ws(lib.attend_workspace_size(c.cache, 4, tokens))
    lib.attend(c.cache, q, out, torch.from_numpy(pos).cuda(), lse=lse, window=64, sink=7, ws=ws)
    c.rows = [299]                                           # no token sees the newest row
    want = R.attend_expected(c, R.host(q), pos, [0, tokens], 4, 64, 7)
    tensor = kind != "f32"
    R.check_attend(R.host(out), R.host(lse), want, kind, tensor, 300, 64, q_exact=kind == "f16", k_exact=k == "f16")


@pytest.mark.parametrize("tokens", [4, 40])
@pytest.mark.parametrize("kind,k,v", [("f16", "f16", "f16"), ("bf16", "q8_0", "q4_0"), ("f32", "f32", "f32")])
def test_junk_that_later_tokens_see(lib, kind, k, v, tokens):
    """A value row of infinities that the last token sees and the earlier ones do not."""
    rng = np.random.default_rng(12)
    c = R.Cache(lib, rng, rows=[200], cap=[200], n_kv=1, hd=64, k_type=k, v_type=v, gaps=False)
    a = c.h["v"] if c.h["v"].dtype.kind == "f" else c.h["v_scale"]
    a[c.row0[0] + 199] = np.inf
    c.d["v"].copy_(torch.from_numpy(c.h["v"]))
    if c.d["v_scale"] is not None:
        c.d["v_scale"].copy_(torch.from_numpy(c.h["v_scale"]))
    q = R.act(np.random.default_rng(4).standard_normal((tokens, 4, 64)), kind)
    out = torch.zeros_like(q)
    pos = torch.arange(200 - tokens, 200, device="cuda", dtype=torch.int32)
    ws = c.ws(lib.attend_workspace_size(c.cache, 4, tokens))
    lib.attend(c.cache, q, out, pos, ws=ws)
    assert not torch.isfinite(out[-1]).any()
    c.rows = [199]
    want = R.attend_expected(c, R.host(q)[:-1], pos.cpu().numpy()[:-1], [0, tokens - 1], 4)
    R.check_attend(R.host(out[:-1]), None, want, kind, kind != "f32", 200, 64, q_exact=kind == "f16", k_exact=k == "f16")


@pytest.mark.parametrize("kind,k,v,hd,group", [("f16", "f16", "f16", 128, 4), ("bf16", "q4_0", "q4_0", 128, 4),
                                               ("f16", "q8_0", "q8_0", 256, 2), ("f32", "f32", "f32", 64, 4)])
@pytest.mark.parametrize("tokens", [1, 3])
def test_long_rows_are_split_and_joined(lib, kind, k, v, hd, group, tokens):
    """One long sequence beside short ones; a second call on the same workspace gives the same bits."""
    rng = np.random.default_rng(21)
    c = R.Cache(lib, rng, rows=[20011, 7, 1500], cap=[20100, 64, 1600], n_kv=1, hd=hd, k_type=k, v_type=v)
    ws = c.ws(lib.attend_workspace_size(c.cache, group, tokens))
    a = run(lib, c, group, kind, [tokens] * 3, ws=ws)
    b = run(lib, c, group, kind, [tokens] * 3, ws=ws)
    assert all(torch.equal(x, y) for x, y in zip(a, b))


@pytest.mark.parametrize("kind,k,v", [("f16", "f16", "f16"), ("bf16", "q8_0", "q4_0"), ("f16", "q4_0", "q8_0")])
@pytest.mark.parametrize("hd,group,tokens,rows,window", [(128, 4, 300, 300, 0), (128, 4, 130, 1000, 0), (64, 8, 77, 500, 200),
                                                         (256, 2, 150, 400, 0), (128, 7, 65, 333, 50), (128, 1, 257, 600, 0)])
def test_prompts(lib, kind, k, v, hd, group, tokens, rows, window):
    rng = np.random.default_rng(rows)
    c = R.Cache(lib, rng, rows=[rows, tokens // 2 + 3], cap=[rows + 1, tokens], n_kv=2, hd=hd, k_type=k, v_type=v,
                gaps=rows != tokens)
    run(lib, c, 2 * group, kind, [tokens, tokens // 2], window=window, sink=3 if window else 0)


def test_peaked_and_far_logits(lib):
    """Logits of several hundred: one row takes all the weight, and no exponential overflows."""
    rng = np.random.default_rng(31)
    for kind, k, v in (("f16", "f16", "f16"), ("bf16", "q8_0", "q8_0"), ("f32", "f32", "f32")):
        c = R.Cache(lib, rng, rows=[400], cap=[400], n_kv=1, hd=128, k_type=k, v_type=v)
        run(lib, c, 4, kind, [1], heat=60.0)
        run(lib, c, 4, kind, [40], heat=60.0)
        run(lib, c, 4, kind, [1], scale=3.0)


@pytest.mark.parametrize("size", [1e-4, 300.0])
def test_small_and_large_values(lib, size):
    """Values (and their block scales) near both ends of fp16."""
    rng = np.random.default_rng(41)
    for k, v in (("f16", "f16"), ("q8_0", "q8_0"), ("q4_0", "q4_0")):
        c = R.Cache(lib, rng, rows=[500], cap=[500], n_kv=1, hd=128, k_type=k, v_type=v)
        a = c.h["v"] if v == "f16" else c.h["v_scale"]
        a[...] = (a.astype(np.float32) * size).astype(np.float16)
        c.d["v" if v == "f16" else "v_scale"].copy_(torch.from_numpy(a))
        for tokens in (1, 40):
            q = R.act(rng.standard_normal((tokens, 4, 128)), "bf16")
            out = torch.zeros_like(q)
            pos = np.arange(tokens, dtype=np.int32) + c.last(0) - tokens + 1
            lib.attend(c.cache, q, out, torch.from_numpy(pos).cuda(), ws=c.ws(lib.attend_workspace_size(c.cache, 4, tokens)))
            want = R.attend_expected(c, R.host(q), pos, [0, tokens], 4)
            R.check_attend(R.host(out), None, want, "bf16", True, 500, 128, q_exact=False, k_exact=k == "f16")


def test_bad_n_live_is_reported_and_skipped(lib):
    rng = np.random.default_rng(51)
    c = R.Cache(lib, rng, rows=[40, 60], cap=[40, 60], n_kv=1, hd=64, k_type="f16", v_type="f16")
    for tokens in (1, 40):
        c.d["n_live"].copy_(torch.tensor([41, 60], dtype=torch.int32))
        q = R.act(rng.standard_normal((2 * tokens, 4, 64)), "f16")
        out = torch.full_like(q, 7.0)
        pos = torch.full((2 * tokens,), 10 ** 6, device="cuda", dtype=torch.int32)
        ws = c.ws(lib.attend_workspace_size(c.cache, 4, tokens))
        lib.attend(c.cache, q, out, pos, ws=ws)
        assert lib.device_status(ws) == lib.ERR_DEVICE_ARG
        assert (out[:tokens] == 7).all() and (out[tokens:] != 7).any()
        c.d["n_live"].copy_(torch.tensor([40, 60], dtype=torch.int32))
        lib.attend(c.cache, q, out, pos, ws=ws)              # the workspace stays usable
        assert lib.device_status(ws) == lib.OK and (out[:tokens] != 7).any()


@pytest.mark.parametrize("tokens", [1, 33])
def test_captured_and_replayed(lib, tokens):
    """A captured call follows n_live, rows and queries from replay to replay; two graphs have a workspace each."""
    rng = np.random.default_rng(61)
    c = R.Cache(lib, rng, rows=[900], cap=[1000], n_kv=2, hd=128, k_type="f16", v_type="f16", gaps=False)
    q = R.act(rng.standard_normal((tokens, 8, 128)), "f16")
    pos = torch.arange(900 - tokens, 900, device="cuda", dtype=torch.int32)
    out = torch.zeros_like(q)
    ws = c.ws(lib.attend_workspace_size(c.cache, 8, tokens))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        lib.attend(c.cache, q, out, pos, ws=ws)
    torch.cuda.current_stream().wait_stream(side)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        lib.attend(c.cache, q, out, pos, ws=ws)
    for rows in (900, 450, 64):
        c.d["n_live"].fill_(rows)
        pos.copy_(torch.arange(rows - tokens, rows, device="cuda", dtype=torch.int32))
        q.copy_(R.act(np.random.default_rng(rows).standard_normal((tokens, 8, 128)), "f16"))
        g.replay()
        once = torch.zeros_like(q)
        lib.attend(c.cache, q, once, pos, ws=c.ws(lib.attend_workspace_size(c.cache, 8, tokens)))
        assert torch.equal(once, out)
        c.rows = [rows]
        want = R.attend_expected(c, R.host(q), pos.cpu().numpy(), [0, tokens], 8)
        R.check_attend(R.host(out), None, want, "f16", True, 900, 128)


def test_two_streams_with_their_own_workspaces(lib):
    rng = np.random.default_rng(71)
    c = R.Cache(lib, rng, rows=[5000, 200], cap=[5000, 256], n_kv=2, hd=128, k_type="q8_0", v_type="q8_0")
    q = [R.act(rng.standard_normal((2, 8, 128)), "f16") for _ in range(2)]
    pos = torch.tensor([c.last(0), c.last(1)], device="cuda", dtype=torch.int32)
    alone, both = [], [torch.zeros_like(x) for x in q]
    for x in q:
        o = torch.zeros_like(x)
        lib.attend(c.cache, x, o, pos, ws=c.ws(lib.attend_workspace_size(c.cache, 8, 1)))
        alone.append(o)
    ws = [c.ws(lib.attend_workspace_size(c.cache, 8, 1)) for _ in q]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in q]
    for _ in range(5):
        for s, x, o, w in zip(streams, q, both, ws):
            lib.attend(c.cache, x, o, pos, ws=w, stream=s)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(alone, both))


def test_one_workspace_for_calls_of_different_shapes(lib):
    """Calls whose units and parts differ leave a shared workspace fit for the next one."""
    rng = np.random.default_rng(31)
    c = R.Cache(lib, rng, rows=[900], cap=[1024], n_kv=8, hd=64, k_type="f16", v_type="f16")
    ws = c.ws(max(lib.attend_workspace_size(c.cache, 32, t) for t in (1, 2, 50, 400)))
    for i, (kind, t, window) in enumerate([("f32", 2, 0), ("f32", 50, 0), ("f16", 1, 0), ("f32", 50, 0), ("f16", 1, 300),
                                           ("f16", 400, 0), ("f16", 2, 0), ("f16", 400, 0), ("f32", 50, 100)]):
        run(lib, c, 32, kind, [t], window=window, seed=i, ws=ws)


@pytest.mark.parametrize("kind,k", [("f16", "f16"), ("bf16", "q4_0"), ("f32", "f32")])
@pytest.mark.parametrize("tokens", [1, 40])
def test_planes_without_rows(lib, kind, k, tokens):
    c = R.Cache(lib, np.random.default_rng(2), rows=[0, 0], cap=[0, 0], n_kv=2, hd=64, k_type=k, v_type=k)
    out, lse = run(lib, c, 8, kind, [tokens, 0])
    assert (out[:tokens] == 0).all() and (lse[:tokens] == -np.inf).all()


@pytest.mark.parametrize("kind,tokens", [("f16", 1), ("bf16", 1), ("f16", 40), ("bf16", 40), ("f32", 3)])
@pytest.mark.parametrize("scale", [1e-44, 1e-60])
def test_logits_near_zero(lib, kind, tokens, scale):
    """A factor that vanishes in fp32 leaves equal weights; hidden rows stay hidden."""
    c = R.Cache(lib, np.random.default_rng(3), rows=[70, 300], cap=[80, 300], n_kv=2, hd=128, k_type="f16", v_type="f16")
    run(lib, c, 8, kind, [tokens, tokens], scale=scale, back=30)


@pytest.mark.parametrize("hd", [96, 160, 192, 224])
@pytest.mark.parametrize("kind,k,v", [("f16", "f16", "f16"), ("bf16", "q8_0", "q4_0"), ("f16", "q4_0", "q8_0")])
@pytest.mark.parametrize("tokens,rows,window", [([50, 3], [120, 700], 0), ([130, 1], [2100, 40], 0), ([40, 2], [300, 90], 65)])
def test_head_dims_between_the_kernels(lib, kind, k, v, hd, tokens, rows, window):
    """Prompts whose heads are padded to the next tile, next to decode steps of the same call."""
    c = R.Cache(lib, np.random.default_rng(17), rows=rows, cap=[r + 9 for r in rows], n_kv=2, hd=hd, k_type=k, v_type=v)
    run(lib, c, 8, kind, tokens, window=window, sink=3 if window else 0, seed=hd, back=2)


@pytest.mark.parametrize("k,v", [("q8_0", "q8_0"), ("q4_0", "q4_0"), ("f16", "q4_0"), ("q4_0", "f16")])
@pytest.mark.parametrize("tokens", [1, 4])
def test_scales_of_three_blocks(lib, k, v, tokens):
    """head_dim 96: a pair of value scales may belong to two rows, of which a token sees one; hidden scales are huge."""
    rng = np.random.default_rng(23)
    c = R.Cache(lib, rng, rows=[77, 16, 1], cap=[80, 16, 4], n_kv=2, hd=96, k_type=k, v_type=v)
    if c.h["v_scale"] is not None:
        for s in range(3):                                      # rows that no token sees (back = 5 positions)
            for g in range(2):
                r0, n = c.row0[s] + g * c.cap[s], c.rows[s]
                late = np.flatnonzero(c.h["pos"][r0:r0 + n] > c.last(s) - 5)
                c.h["v_scale"][r0 + late] = 60000.0
        c.d["v_scale"].copy_(torch.from_numpy(c.h["v_scale"]))
    run(lib, c, 8, "f16", [tokens] * 3, back=5)


@pytest.mark.parametrize("k,v", [("q8_0", "q4_0"), ("q4_0", "f16")])
@pytest.mark.parametrize("hd", [64, 128, 192])
def test_prompts_over_codes_with_and_without_lse(lib, k, v, hd):
    """With a log-sum-exp asked for, logits over quantised keys are those of exact keys; without one the keys are rounded
    to fp16 once. Both outputs are within check_attend's bounds of the rounded keys."""
    c = R.Cache(lib, np.random.default_rng(41), rows=[400, 61], cap=[410, 64], n_kv=2, hd=hd, k_type=k, v_type=v)
    rng = np.random.default_rng(42)
    tok0 = np.array([0, 70, 131], np.int32)
    pos = np.concatenate([c.last(s) - np.arange(t)[::-1] for s, t in enumerate((70, 61))]).astype(np.int32)
    q = R.act(rng.standard_normal((131, 8, hd)), "f16")
    ws = c.ws(lib.attend_workspace_size(c.cache, 8, tok0))
    want = R.attend_expected(c, R.host(q), pos, tok0, 8)
    for lse in (torch.empty(131, 8, device="cuda"), None):
        out = torch.empty_like(q)
        lib.attend(c.cache, q, out, torch.from_numpy(pos).cuda(), tok0=tok0, lse=lse, ws=ws)
        assert lib.device_status(ws) == lib.OK
        R.check_attend(R.host(out), None, want, "f16", True, 400, hd, k_exact=False)
        if lse is not None:                      # (hd + 2) 2^-24 of the moduli and the sum's roundings, none of the keys'
            tl = (hd + 2) * R.U24 * want[3] + (400 / 32 + 64) * R.U24 + R.U24 * 4 * np.abs(want[1])
            assert np.all(np.abs(R.host(lse) - want[1]) <= tl)
