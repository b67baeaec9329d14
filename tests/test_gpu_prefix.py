"""tria_attend_prefix against one joint softmax in 64 bits: types, head layouts,
one sequence to many, prefixes and own rows from none to long, windows that
end in either part, masks that leave a token nothing, junk that no token sees."""
import numpy as np
import pytest

import _prefix as P
import _rows as R
from oracle import attend_oracle as A

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")


def run(lib, p, c, seq0, nq, kind, tokens, *, window=0, sink=0, scale=None, seed=0, heat=1.0, back=0, ws=None, stride=0, newest=None,
        want_lse=True):
    """tokens[s] new tokens of sequence s, the newest ones (`back` positions earlier), checked against 64 bits."""
    rng = np.random.default_rng(seed + 1)
    newest = P.follow(p, c, seq0) if newest is None else newest
    tok0 = np.concatenate([[0], np.cumsum(tokens)]).astype(np.int32)
    n = int(tok0[-1])
    pos = np.concatenate([newest[s] - back - np.arange(t)[::-1] for s, t in enumerate(tokens)] + [[]]).astype(np.int32)
    wide = R.act(rng.standard_normal((n, nq + stride, c.hd)) * heat, kind)
    q = wide[:, :nq]
    out = torch.full((n + 1, nq, c.hd), 7.0, device="cuda", dtype=q.dtype)
    lse = torch.full((n + 1, nq), 7.0, device="cuda")
    if ws is None:
        ws = c.ws(lib.attend_prefix_workspace_size(p.cache, c.cache, nq, tok0, seq0))
    lib.attend_prefix(p.cache, c.cache, q, out[:n], torch.from_numpy(pos).cuda(), seq0=seq0, tok0=tok0, lse=lse[:n] if want_lse else None,
                      window=window, sink=sink, scale=scale or 0.0, ws=ws)
    assert lib.device_status(ws) == lib.OK
    assert (out[n] == 7).all() and (lse[n] == 7).all()
    if n == 0:
        return out, lse
    want = P.expected(p, c, seq0, R.host(q), pos, tok0, nq, window, sink, scale)
    f32 = kind == "f32" or ("f32" in (p.k_type, p.v_type) and "f32" in (c.k_type, c.v_type))
    exact = p.k_type == c.k_type == "f16"
    P.check(R.host(out[:n]), R.host(lse[:n]) if want_lse else None, want, kind, not f32, max(p.rows) + max(c.rows), c.hd,
            q_exact=kind == "f16", k_exact=exact)
    return out, lse


TYPES = [("f16", "f16", "f16"), ("bf16", "f16", "f16"), ("f16", "q8_0", "q8_0"), ("bf16", "q4_0", "q4_0"), ("f16", "q8_0", "q4_0"),
         ("f16", "q4_0", "f16"), ("f16", "f16", "q8_0"), ("f32", "f32", "f32"), ("f32", "q4_0", "q8_0")]


@pytest.mark.parametrize("kind,k,v", TYPES)
@pytest.mark.parametrize("hd,n_kv,group", [(64, 2, 4), (128, 2, 4), (256, 1, 2)])
@pytest.mark.parametrize("seqs", [3, 9, 40])
def test_single_tokens(lib, kind, k, v, hd, n_kv, group, seqs):
    rng = np.random.default_rng(hd + seqs)
    p, c = P.pair(lib, rng, shared=[700], rows=[1 + 7 * s % 40 for s in range(seqs)], n_kv=n_kv, hd=hd, types=(k, v))
    run(lib, p, c, [0, seqs], n_kv * group, kind, [1] * seqs)


@pytest.mark.parametrize("kind,k,v", TYPES)
@pytest.mark.parametrize("shared", [[1, 300, 129], [128, 64, 1000], [0, 31, 2]])
def test_several_prefixes(lib, kind, k, v, shared):
    """Groups of none, few and many sequences; prefixes that end inside a tile, at its end, or hold nothing."""
    rng = np.random.default_rng(shared[1])
    p, c = P.pair(lib, rng, shared=shared, rows=[3, 50, 0, 17, 1, 130, 64, 5, 9, 11, 20], n_kv=2, hd=128, types=(k, v))
    run(lib, p, c, [0, 2, 11, 11], 8, kind, [1] * 11, stride=2)
    p, c = P.pair(lib, rng, shared=shared, rows=[3, 50, 2, 17, 1, 130, 64, 5, 9, 11, 20], n_kv=2, hd=128, types=(k, v))
    run(lib, p, c, [0, 1, 4, 11], 8, kind, [1, 0, 3, 1, 0, 2, 1, 1, 5, 1, 9])


@pytest.mark.parametrize("hd,n_kv,group", [(32, 3, 1), (96, 1, 8), (160, 2, 3), (192, 1, 5), (224, 1, 6), (128, 2, 7), (64, 1, 1), (256, 2, 8)])
@pytest.mark.parametrize("kind,k,v", [("f16", "f16", "f16"), ("bf16", "q4_0", "q8_0"), ("f16", "q8_0", "f16")])
def test_head_shapes(lib, kind, k, v, hd, n_kv, group):
    rng = np.random.default_rng(hd)
    p, c = P.pair(lib, rng, shared=[260, 515], rows=[3, 20, 1, 9, 33, 7, 8], n_kv=n_kv, hd=hd, types=(k, v))
    run(lib, p, c, [0, 5, 7], n_kv * group, kind, [1] * 7)
    p, c = P.pair(lib, rng, shared=[260, 515], rows=[30, 20, 41, 39, 33, 7, 18], n_kv=n_kv, hd=hd, types=(k, v))
    run(lib, p, c, [0, 3, 7], n_kv * group, kind, [5, 20, 1, 33, 2, 7, 0])


@pytest.mark.parametrize("own", [("q8_0", "q8_0"), ("f16", "q4_0"), ("f32", "f32")])
@pytest.mark.parametrize("kind", ["f16", "bf16"])
def test_caches_of_different_types(lib, kind, own):
    rng = np.random.default_rng(3)
    p, c = P.pair(lib, rng, shared=[400], rows=[60] * 6, n_kv=2, hd=128, types=("q4_0", "q4_0"), own_types=own)
    newest = P.follow(p, c, [0, 6])
    for t in (1, 4):
        run(lib, p, c, [0, 6], 8, kind, [t] * 6, newest=newest)


@pytest.mark.parametrize("window,sink", [(1, 0), (16, 4), (100, 1), (100, 200), (4096, 3), (600, 50)])
@pytest.mark.parametrize("tokens", [1, 3, 30])
@pytest.mark.parametrize("kind,k,v,hd", [("f16", "f16", "f16", 128), ("bf16", "q8_0", "q4_0", 64), ("f32", "f32", "f32", 64)])
def test_window_and_first_rows(lib, kind, k, v, hd, tokens, window, sink):
    rng = np.random.default_rng(window)
    p, c = P.pair(lib, rng, shared=[513, 40], rows=[60, 35, 200, 31, 90, 33], n_kv=2, hd=hd, types=(k, v))
    run(lib, p, c, [0, 4, 6], 8, kind, [tokens] * 6, window=window, sink=sink)


@pytest.mark.parametrize("kind,k,v", [("f16", "f16", "f16"), ("f32", "f32", "f32"), ("f16", "q8_0", "q8_0")])
@pytest.mark.parametrize("seqs,tokens", [(2, 1), (9, 1), (3, 20)])
def test_tokens_that_see_nothing(lib, kind, k, v, seqs, tokens):
    """Queries before every row, in the middle of the prefix, between the prefix and the own rows."""
    rng = np.random.default_rng(9)
    p, c = P.pair(lib, rng, shared=[150, 0], rows=[50] * seqs + [0], n_kv=2, hd=64, types=(k, v))
    seq0 = [0, seqs, seqs + 1]
    newest = P.follow(p, c, seq0)
    n = seqs * tokens
    out, lse = run(lib, p, c, seq0, 4, kind, [tokens] * (seqs + 1), back=10000, newest=newest)
    assert (out[:n + tokens] == 0).all() and (lse[:n + tokens] == -np.inf).all()
    for back in (100, 260, 400):
        run(lib, p, c, seq0, 4, kind, [tokens] * (seqs + 1), back=back, newest=newest)
        run(lib, p, c, seq0, 4, kind, [tokens] * (seqs + 1), back=back, newest=newest, window=30, sink=2)


@pytest.mark.parametrize("kind,k,v", [("f16", "f16", "f16"), ("f32", "f32", "f32"), ("bf16", "q8_0", "q4_0")])
@pytest.mark.parametrize("seqs", [2, 12])
@pytest.mark.parametrize("bad", [np.nan, np.inf, -np.inf])
def test_junk_in_hidden_rows(lib, kind, k, v, seqs, bad):
    """Rows of the prefix outside the window, and own rows newer than every token, hold NaN or infinities."""
    rng = np.random.default_rng(11)
    p, c = P.pair(lib, rng, shared=[300], rows=[20] * seqs, n_kv=1, hd=64, types=(k, v), gaps=False)
    newest = P.follow(p, c, [0, seqs])

    def plane(x, name):
        return x.h[name] if x.h[name].dtype.kind == "f" else x.h[name + "_scale"]

    for name in ("k", "v"):
        plane(p, name)[p.row0[0] + 5:p.row0[0] + 254] = bad  # positions 5 .. 253; the tokens stand at 317 and see 254 on
        for s in range(seqs):
            plane(c, name)[c.row0[s] + 18:c.row0[s] + 20] = bad
    for x in (p, c):
        for n, a in x.h.items():
            if a is not None:
                x.d[n].copy_(torch.from_numpy(a))
        for name in ("k", "v"):                             # the 64-bit form reads zeros there
            a = plane(x, name)
            a[~np.isfinite(a)] = 0
    out, _ = run(lib, p, c, [0, seqs], 4, kind, [1] * seqs, window=64, sink=5, back=2, newest=newest)
    assert torch.isfinite(out).all()


def test_a_token_that_sees_junk_alone_is_not_finite(lib):
    rng = np.random.default_rng(12)
    for seqs in (2, 12):
        p, c = P.pair(lib, rng, shared=[300], rows=[20] * seqs, n_kv=1, hd=64, types=("f16", "f16"), gaps=False)
        newest = P.follow(p, c, [0, seqs])
        p.d["v"][p.row0[0] + 290] = float("inf")
        pos = torch.tensor(newest, device="cuda", dtype=torch.int32)
        pos[1:] = 285
        q = R.act(rng.standard_normal((seqs, 4, 64)), "f16")
        out = torch.zeros_like(q)
        lib.attend_prefix(p.cache, c.cache, q, out, pos, ws=c.ws(lib.attend_prefix_workspace_size(p.cache, c.cache, 4, 1)))
        assert not torch.isfinite(out[0]).any() and torch.isfinite(out[1:]).all()


@pytest.mark.parametrize("kind,k,v", [("f16", "f16", "f16"), ("bf16", "q8_0", "q4_0"), ("f16", "q4_0", "q8_0")])
@pytest.mark.parametrize("hd,group,tokens,shared,window", [(128, 4, 100, 300, 0), (64, 8, 77, 500, 200), (256, 2, 150, 400, 0),
                                                           (128, 1, 257, 600, 0)])
def test_chunks_of_prompts(lib, kind, k, v, hd, group, tokens, shared, window):
    rng = np.random.default_rng(shared)
    p, c = P.pair(lib, rng, shared=[shared], rows=[tokens + 3, tokens // 2, tokens], n_kv=2, hd=hd, types=(k, v))
    run(lib, p, c, [0, 3], 2 * group, kind, [tokens, tokens // 2, 1], window=window, sink=3 if window else 0)


def test_peaked_and_far_logits(lib):
    rng = np.random.default_rng(31)
    for kind, k, v in (("f16", "f16", "f16"), ("bf16", "q8_0", "q8_0"), ("f32", "f32", "f32")):
        for seqs in (1, 12):
            p, c = P.pair(lib, rng, shared=[400], rows=[30] * seqs, n_kv=1, hd=128, types=(k, v))
            newest = P.follow(p, c, [0, seqs])
            run(lib, p, c, [0, seqs], 4, kind, [1] * seqs, heat=60.0, newest=newest)
            run(lib, p, c, [0, seqs], 4, kind, [1] * seqs, scale=3.0, newest=newest)
            run(lib, p, c, [0, seqs], 4, kind, [1] * seqs, scale=1e-44, newest=newest)


@pytest.mark.parametrize("size", [1e-4, 300.0])
def test_small_and_large_values(lib, size):
    """Values (and their block scales) near both ends of fp16."""
    rng = np.random.default_rng(41)
    for k, v in (("f16", "f16"), ("q8_0", "q8_0"), ("q4_0", "q4_0")):
        p, c = P.pair(lib, rng, shared=[500], rows=[40] * 9, n_kv=1, hd=128, types=(k, v))
        for x in (p, c):
            a = x.h["v"] if v == "f16" else x.h["v_scale"]
            a[...] = (a.astype(np.float32) * size).astype(np.float16)
            x.d["v" if v == "f16" else "v_scale"].copy_(torch.from_numpy(a))
        run(lib, p, c, [0, 9], 4, "bf16", [1] * 9)


def test_without_lse_and_with_rounded_keys(lib):
    """out has the same bits with and without lse; rounded keys stay within their rounding."""
    rng = np.random.default_rng(43)
    for k, v in (("q8_0", "q4_0"), ("f16", "f16")):
        p, c = P.pair(lib, rng, shared=[900], rows=[70] * 10, n_kv=2, hd=128, types=(k, v))
        newest = P.follow(p, c, [0, 10])
        a, _ = run(lib, p, c, [0, 10], 8, "f16", [2] * 10, newest=newest)
        b, _ = run(lib, p, c, [0, 10], 8, "f16", [2] * 10, newest=newest, want_lse=False)
        assert torch.equal(a, b)
        q = R.act(np.random.default_rng(1).standard_normal((20, 8, 128)), "f16")
        out = torch.empty_like(q)
        pos = torch.tensor(np.repeat(newest, 2) - np.tile([1, 0], 10), device="cuda", dtype=torch.int32)
        lib.attend_prefix(p.cache, c.cache, q, out, pos, round_keys=True, ws=c.ws(lib.attend_prefix_workspace_size(p.cache, c.cache, 8, 2)))
        want = P.expected(p, c, [0, 10], R.host(q), pos.cpu().numpy(), np.arange(11) * 2, 8)
        P.check(R.host(out), None, want, "f16", True, 970, 128, k_exact=False)


def test_bad_n_live_is_reported_and_skipped(lib):
    rng = np.random.default_rng(51)
    for seqs, tokens in ((4, 1), (20, 1), (4, 30)):
        p, c = P.pair(lib, rng, shared=[60, 60], rows=[40] * seqs, n_kv=1, hd=64, types=("f16", "f16"), spare=0)
        P.follow(p, c, [0, seqs // 2, seqs])
        q = R.act(rng.standard_normal((seqs * tokens, 4, 64)), "f16")
        pos = torch.full((seqs * tokens,), 10 ** 6, device="cuda", dtype=torch.int32)
        ws = c.ws(lib.attend_prefix_workspace_size(p.cache, c.cache, 4, tokens))
        half = seqs * tokens // 2
        for x, at, bad in ((p, 0, 61), (p, 0, -1), (c, 0, 41), (c, 1, -5)):
            keep = x.d["n_live"].clone()
            x.d["n_live"][at] = bad
            out = torch.full_like(q, 7.0)
            lib.attend_prefix(p.cache, c.cache, q, out, pos, ws=ws)
            assert lib.device_status(ws) == lib.ERR_DEVICE_ARG
            lost = slice(0, half) if x is p else slice(at * tokens, (at + 1) * tokens)
            assert (out[lost] == 7).all() and torch.isfinite(out).all() and (out[half:] != 7).any()
            x.d["n_live"].copy_(keep)
            lib.attend_prefix(p.cache, c.cache, q, out, pos, ws=ws)      # the workspace stays usable
            assert lib.device_status(ws) == lib.OK and (out[lost] != 7).any()


@pytest.mark.parametrize("seqs,tokens,k", [(3, 1, "f16"), (17, 1, "f16"), (17, 1, "q8_0"), (3, 33, "f16")])
def test_captured_and_replayed(lib, seqs, tokens, k):
    """A captured call follows both n_live, rows and queries from replay to replay."""
    rng = np.random.default_rng(61)
    p, c = P.pair(lib, rng, shared=[900], rows=[300] * seqs, n_kv=2, hd=128, types=(k, k), gaps=False)
    P.follow(p, c, [0, seqs])
    q = R.act(rng.standard_normal((seqs * tokens, 8, 128)), "f16")
    pos = torch.zeros(seqs * tokens, device="cuda", dtype=torch.int32)
    out = torch.zeros_like(q)
    size = lib.attend_prefix_workspace_size(p.cache, c.cache, 8, tokens)
    ws = c.ws(size)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        lib.attend_prefix(p.cache, c.cache, q, out, pos, ws=ws)
    torch.cuda.current_stream().wait_stream(side)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        lib.attend_prefix(p.cache, c.cache, q, out, pos, ws=ws)
    for shared, rows in ((900, 300), (450, 299), (64, 40)):
        p.d["n_live"].fill_(shared)
        c.d["n_live"].fill_(rows)
        pos.copy_(torch.tensor(np.tile(np.arange(900 + rows - tokens, 900 + rows), seqs), dtype=torch.int32))
        q.copy_(R.act(np.random.default_rng(rows).standard_normal((seqs * tokens, 8, 128)), "f16"))
        g.replay()
        once = torch.zeros_like(q)
        lib.attend_prefix(p.cache, c.cache, q, once, pos, ws=c.ws(size))
        assert torch.equal(once, out)
        p.rows, c.rows = [shared], [rows] * seqs
        want = P.expected(p, c, [0, seqs], R.host(q), pos.cpu().numpy(), np.arange(seqs + 1) * tokens, 8)
        P.check(R.host(out), None, want, "f16", True, 1200, 128, k_exact=k == "f16")


def test_two_streams_with_their_own_workspaces(lib):
    rng = np.random.default_rng(71)
    p, c = P.pair(lib, rng, shared=[5000], rows=[200] * 12, n_kv=2, hd=128, types=("q8_0", "q8_0"))
    newest = P.follow(p, c, [0, 12])
    q = [R.act(rng.standard_normal((12, 8, 128)), "f16") for _ in range(2)]
    pos = torch.tensor(newest, device="cuda", dtype=torch.int32)
    size = lib.attend_prefix_workspace_size(p.cache, c.cache, 8, 1)
    alone, both = [], [torch.zeros_like(x) for x in q]
    for x in q:
        o = torch.zeros_like(x)
        lib.attend_prefix(p.cache, c.cache, x, o, pos, ws=c.ws(size))
        alone.append(o)
    ws = [c.ws(size) for _ in q]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in q]
    for _ in range(5):
        for s, x, o, w in zip(streams, q, both, ws):
            lib.attend_prefix(p.cache, c.cache, x, o, pos, ws=w, stream=s)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(alone, both))


def test_one_workspace_for_calls_of_both_kinds(lib):
    """Calls whose units and parts differ leave a shared workspace fit for the next one, attention without a prefix too."""
    rng = np.random.default_rng(31)
    shapes = [("f32", "f32", 2, 3), ("f16", "f16", 20, 1), ("f16", "q8_0", 20, 1), ("f16", "f16", 2, 1), ("f16", "q4_0", 3, 40), ("f16", "f16", 30, 2),
              ("f32", "f32", 5, 9), ("f16", "q8_0", 3, 1)]
    made = []
    for kind, k, seqs, tokens in shapes:
        p, c = P.pair(lib, rng, shared=[1500], rows=[50] * seqs, n_kv=4, hd=64, types=(k, k))
        made.append((p, c, P.follow(p, c, [0, seqs])))
    size = max(lib.attend_prefix_workspace_size(p.cache, c.cache, 16, t) for (p, c, _), (_, _, _, t) in zip(made, shapes))
    ws = made[0][0].ws(size)
    for i, ((p, c, newest), (kind, k, seqs, tokens)) in enumerate(zip(made, shapes)):
        run(lib, p, c, [0, seqs], 16, kind, [tokens] * seqs, seed=i, ws=ws, newest=newest, window=0 if i % 2 else 400)
        q = R.act(rng.standard_normal((2, 16, 64)), kind)
        once, out = torch.zeros_like(q), torch.zeros_like(q)
        at = torch.full((2,), p.last(0), device="cuda", dtype=torch.int32)
        lib.attend(p.cache, q, out, at, ws=ws)
        lib.attend(p.cache, q, once, at, ws=p.ws(lib.attend_workspace_size(p.cache, 16, 2)))
        assert torch.equal(once, out)


@pytest.mark.parametrize("kind,k,v", [("f16", "f16", "f16"), ("bf16", "q8_0", "q4_0"), ("f16", "q4_0", "q8_0"), ("f16", "f16", "q8_0")])
@pytest.mark.parametrize("seqs,tokens,window,sink", [(1, 1, 0, 0), (4, 1, 0, 0), (4, 1, 100, 3), (2, 2, 40, 0), (3, 80, 0, 0), (3, 80, 120, 5),
                                                     (2, 150, 0, 0)])
@pytest.mark.parametrize("n_kv,hd", [(2, 64), (1, 256)])
def test_prefixes_of_large_capacity(lib, kind, k, v, seqs, tokens, window, sink, n_kv, hd):
    """How a prefix is read depends on its capacity too: few live rows in a place for very many give the same results."""
    rng = np.random.default_rng(81)
    for shared, spare in (([400, 0], 90000 // n_kv), ([400, 0], 3)):
        p, c = P.pair(lib, rng, shared=shared, rows=[tokens + 9] * (seqs + 1), n_kv=n_kv, hd=hd, types=(k, v), spare=spare, own_spare=5, gaps=False)
        newest = P.follow(p, c, [0, seqs, seqs + 1])
        run(lib, p, c, [0, seqs, seqs + 1], 4 * n_kv, kind, [tokens] * seqs + [1], newest=newest, window=window, sink=sink)


def test_bad_n_live_in_prefixes_of_large_capacity(lib):
    rng = np.random.default_rng(51)
    for seqs, tokens in ((4, 1), (2, 150)):
        p, c = P.pair(lib, rng, shared=[60, 60], rows=[tokens + 40] * seqs, n_kv=1, hd=64, types=("q8_0", "q8_0"), spare=90000, own_spare=0)
        P.follow(p, c, [0, seqs // 2, seqs])
        q = R.act(rng.standard_normal((seqs * tokens, 4, 64)), "f16")
        pos = torch.full((seqs * tokens,), 10 ** 6, device="cuda", dtype=torch.int32)
        ws = c.ws(lib.attend_prefix_workspace_size(p.cache, c.cache, 4, tokens))
        half = seqs * tokens // 2
        for bad in (-1, 90061):
            keep = p.d["n_live"].clone()
            p.d["n_live"][0] = bad
            out = torch.full_like(q, 7.0)
            lib.attend_prefix(p.cache, c.cache, q, out, pos, ws=ws)
            assert lib.device_status(ws) == lib.ERR_DEVICE_ARG
            assert (out[:half] == 7).all() and torch.isfinite(out).all() and (out[half:] != 7).any()
            p.d["n_live"].copy_(keep)
            lib.attend_prefix(p.cache, c.cache, q, out, pos, ws=ws)
            assert lib.device_status(ws) == lib.OK and (out[:half] != 7).any()


@pytest.mark.parametrize("kind,k,v,hd", [("f16", "f16", "f16", 128), ("f16", "f16", "f16", 256), ("f16", "f16", "q8_0", 64), ("f16", "q8_0", "q4_0", 128),
                                         ("f16", "q4_0", "f16", 64)])
@pytest.mark.parametrize("seqs", [4, 20])
def test_logits_that_rise_again_and_again(lib, kind, k, v, hd, seqs):
    """Logits rise by 9.5 powers of two every 64 rows, so that the reference of the softmax moves at every tile, and fall back
    to their start after 2000 rows; the same call gives the same bits ten times, whatever the workspace held."""
    n_kv, rows = 8, 24000
    rng = np.random.default_rng(hd)
    p, c = P.pair(lib, rng, shared=[rows], rows=[5] * seqs, n_kv=n_kv, hd=hd, types=(k, v), gaps=False, spare=0)
    sign = rng.choice([-1.0, 1.0], hd)
    rise = (np.arange(rows) % 2000) * (9.5 / 64 * np.log(2))
    for g in range(n_kv):
        r0 = p.row0[0] + g * p.cap[0]
        data, scale = A.hold((rise[:, None] * sign / np.sqrt(hd) + 0.3 * rng.standard_normal((rows, hd))).astype(np.float32), k)
        for name, x in (("k", data), ("k_scale", scale)):
            if x is not None:
                p.h[name][r0:r0 + rows] = x
    for name in ("k", "k_scale"):
        if p.h[name] is not None:
            p.d[name].copy_(torch.from_numpy(p.h[name]))
    newest = P.follow(p, c, [0, seqs])
    q = R.act(sign * (1 + 0.1 * rng.standard_normal((seqs, 4 * n_kv, hd))), kind)
    pos = torch.tensor(newest, device="cuda", dtype=torch.int32)
    first = None
    for i in range(10):
        out, lse = torch.zeros_like(q), torch.zeros(seqs, 4 * n_kv, device="cuda")
        ws = torch.full((lib.attend_prefix_workspace_size(p.cache, c.cache, 4 * n_kv, 1),), 255, dtype=torch.uint8, device="cuda")
        lib.workspace_init(ws)
        lib.attend_prefix(p.cache, c.cache, q, out, pos, lse=lse, ws=ws)
        assert lib.device_status(ws) == lib.OK
        if first is None:
            first = out, lse
            want = P.expected(p, c, [0, seqs], R.host(q), pos.cpu().numpy(), np.arange(seqs + 1), 4 * n_kv)
            P.check(R.host(out), R.host(lse), want, kind, True, rows + 5, hd, k_exact=k == "f16")
        assert torch.equal(out, first[0]) and torch.equal(lse, first[1])
