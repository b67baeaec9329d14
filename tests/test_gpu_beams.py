"""tria_beam_select against the whole sorted list of continuations in 64 bits:
types, widths, odd vocabularies, ties, masked and broken rows, beams that are
over, places, aliases, replays."""
import numpy as np
import pytest

import _rows as R
from oracle import beam_oracle as B

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

# total_out is v rounded to fp32 (2^-24 |v|) and carries the sum's error: exponentials 2 units and their arguments
# (|x - top| e^(x - top) <= 1/e roundings), a thread's 32 terms and 13 levels above in fp32: under 64 x 2^-24 of the sum,
# so as much of its logarithm; comparisons hold beyond twice that.
LOG_TOL = 64 * R.U24


def make(rng, beams, vocab, kind, spread=3.0):
    return R.act(rng.standard_normal((beams, vocab)) * spread, kind)


def run(lib, logits, total, seq0, n_out, *, ended=None, end_token=-1, in_place=False, ws=None, stream=None):
    n_groups = len(seq0) - 1
    out = dict(total_out=torch.full((n_groups + 1, n_out), 7.0, device="cuda"),
               **{k: torch.full((n_groups + 1, n_out), -7, device="cuda", dtype=torch.int32) for k in ("parent", "token", "ended_out")})
    if ws is None:
        ws = torch.empty(lib.beam_select_workspace_size(seq0, logits.shape[1], n_out), dtype=torch.uint8, device="cuda")
        lib.workspace_init(ws)
    t = torch.tensor(np.asarray(total, np.float32)).cuda()
    e = None if ended is None else torch.tensor(np.asarray(ended, np.int32)).cuda()
    lib.beam_select(logits, t, out["total_out"][:-1], out["parent"][:-1], out["token"][:-1], seq0=seq0, ended=e,
                    ended_out=out["ended_out"][:-1], end_token=end_token, in_place=in_place, ws=ws, stream=stream)
    assert lib.device_status(ws) == lib.OK
    assert (out["total_out"][-1] == 7).all() and all((out[k][-1] == -7).all() for k in ("parent", "token", "ended_out"))
    return {k: v[:-1].cpu().numpy() for k, v in out.items()}


def check(got, logits, total, seq0, n_out, ended=None, end_token=-1, in_place=False):
    """Every choice equal to the sorted list's, but where the totals of different beams are nearer than the tolerance:
    there the values alone are compared."""
    v = B.values(logits.float().cpu().numpy(), np.asarray(total, np.float32), ended, end_token)
    for g in range(len(seq0) - 1):
        a, b = seq0[g], seq0[g + 1]
        want = B.choose(v[a:b], a, n_out, in_place)
        flat = np.sort(v[a:b].reshape(-1))[::-1]
        gap = np.abs(np.diff(flat[:n_out + 1], append=-np.inf)) if flat.size <= n_out else np.abs(np.diff(flat[:n_out + 1]))
        with np.errstate(invalid="ignore"):
            near = bool(((gap <= 2 * LOG_TOL) & (gap > 0)).any())
        for i, (parent, token, val) in enumerate(want):
            if not near:
                assert (got["parent"][g, i], got["token"][g, i]) == (parent, token)
            if not near or not in_place:
                x = got["total_out"][g, i]
                assert x == val if not np.isfinite(val) else abs(x - val) <= R.U24 * abs(val) + LOG_TOL
            val = v[got["parent"][g, i], got["token"][g, i]]
            x = got["total_out"][g, i]
            assert x == val if not np.isfinite(val) else abs(x - val) <= R.U24 * abs(val) + LOG_TOL
            over = got["token"][g, i] == end_token or (ended is not None and ended[got["parent"][g, i]])
            assert got["ended_out"][g, i] == int(bool(over))


@pytest.mark.parametrize("kind", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("vocab", [1, 7, 31, 256, 1000, 2049, 8192, 8193, 33333, 100001])
@pytest.mark.parametrize("widths,n_out", [([4], 4), ([1], 1), ([3, 1, 8], 5), ([32], 64), ([2] * 20, 2)])
def test_widths_and_vocabularies(lib, kind, vocab, widths, n_out):
    rng = np.random.default_rng(vocab + n_out)
    seq0 = np.concatenate([[0], np.cumsum(widths)])
    n_out = min(n_out, min(widths) * vocab)
    n = int(seq0[-1])
    logits, total = make(rng, n, vocab, kind), -5 * rng.random(n)
    check(run(lib, logits, total, seq0, n_out), logits, total, seq0, n_out)


@pytest.mark.parametrize("kind", ["f16", "f32"])
@pytest.mark.parametrize("offset,stride", [(0, 1003), (1, 1003), (3, 1001), (8, 1008), (0, 2000)])
def test_unaligned_rows_and_strides(lib, kind, offset, stride):
    """Rows that start anywhere; the same row has the same sum wherever it lies, so that equal rows tie by beam."""
    rng = np.random.default_rng(stride)
    row = make(rng, 1, 1000, kind)
    flat = torch.zeros(offset + 6 * stride + 8, device="cuda", dtype=row.dtype)
    logits = flat[offset:].as_strided((6, 1000), (stride, 1))
    logits.copy_(row.expand(6, 1000))
    got = run(lib, logits, [-1.0] * 6, [0, 6], 12)
    best = np.argsort(-row[0].float().cpu().numpy(), kind="stable")[:2]
    if row[0, best[0]] != row[0, best[1]]:
        assert got["parent"][0].tolist() == [0, 1, 2, 3, 4, 5] * 2
        assert got["token"][0].tolist() == [best[0]] * 6 + [best[1]] * 6
    check(got, logits, [-1.0] * 6, [0, 6], 12)


@pytest.mark.parametrize("n_out", [1, 5, 17, 64])
def test_ties(lib, n_out):
    """All logits equal; many equal largest ones at one end; zeros of both signs."""
    for vocab in (100, 5000, 20000):
        logits = torch.zeros(3, vocab, device="cuda", dtype=torch.float16)
        got = run(lib, logits, [-1.0, -1.0, -1.0], [0, 3], n_out)
        assert got["parent"].max() == 0 and got["token"][0].tolist() == list(range(n_out))
        logits[:, 1::2] = -0.0
        logits[1, vocab - 70:] = 2.0
        check(run(lib, logits, [-1.0, -1.0, -3.0], [0, 3], n_out), logits, [-1.0, -1.0, -3.0], [0, 3], n_out)


@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("vocab", [40, 9000, 30000])
def test_masked_vocabularies(lib, kind, vocab):
    """All but a few tokens are -inf; fewer finite continuations than asked for: -inf ones by their index."""
    rng = np.random.default_rng(5)
    logits = torch.full((4, vocab), -np.inf, device="cuda", dtype=R.act(np.zeros(1), kind).dtype)
    for b, k in enumerate((1, 3, 12, 0)):
        logits[b, torch.from_numpy(rng.choice(vocab, k, replace=False)).cuda()] = make(rng, 1, max(k, 1), kind)[0, :k]
    total = [-1.0, -2.0, -0.5, 0.0]
    for n_out in (4, 16, 40):
        check(run(lib, logits, total, [0, 4], n_out), logits, total, [0, 4], n_out)


def test_broken_rows_and_totals(lib):
    rng = np.random.default_rng(6)
    logits = make(rng, 8, 3000, "f32")
    logits[1, 1234] = float("nan")
    logits[2, 5] = float("inf")
    logits[3] = -float("inf")
    total = [-1.0, 0.0, 0.0, 0.0, -np.inf, np.inf, np.nan, -1.5]
    check(run(lib, logits, total, [0, 8], 20), logits, total, [0, 8], 20)
    check(run(lib, logits[1:7], total[1:7], [0, 6], 9), logits[1:7], total[1:7], [0, 6], 9)      # nothing but -inf


def test_lowest_and_largest_logits(lib):
    for kind in ("f16", "bf16", "f32"):
        low = torch.finfo(R.act(np.zeros(1), kind).dtype)
        logits = make(np.random.default_rng(8), 3, 5000, kind)
        logits[0, 100:] = low.min                            # masks of the type's lowest value
        logits[1] = low.min
        logits[2, 7] = low.max
        total = [-1.0, -2.0, -3.0]
        check(run(lib, logits, total, [0, 3], 8), logits, total, [0, 3], 8)


@pytest.mark.parametrize("total", [[0.0, -1.0], [-50.0, 0.0]])
def test_many_large_values_on_few_threads(lib, total):
    """Logits arranged so that the candidates overflow the list: the best are taken one after the other."""
    vocab = 16384
    logits = make(np.random.default_rng(9), 2, vocab, "f32", spread=1.0)
    # of every 1024 tokens, threads 0 .. 63 of a CTA hold the first 256: the largest lie there
    at = (np.arange(8)[:, None, None] * 1024 + np.arange(64)[None, :, None] * 4 + np.arange(4)).reshape(-1)
    logits[0, torch.from_numpy(at).cuda()] = 30 + torch.rand(len(at), device="cuda")
    check(run(lib, logits, total, [0, 2], 64), logits, total, [0, 2], 64)


@pytest.mark.parametrize("kind", ["f16", "f32"])
@pytest.mark.parametrize("in_place", [False, True])
def test_beams_that_are_over(lib, kind, in_place):
    rng = np.random.default_rng(10)
    logits = make(rng, 12, 4001, kind)
    total, ended = -3 * rng.random(12), (rng.random(12) < 0.5).astype(np.int32)
    ended[:6] = 1                                             # a group all of whose beams are over
    logits[torch.from_numpy(ended != 0).cuda()] = float("nan")   # their logits are not looked at
    clean = logits.clone()
    clean[torch.from_numpy(ended != 0).cuda()] = 0
    for end in (0, 2500, 4000):
        got = run(lib, logits, total, [0, 6, 12], 6, ended=ended, end_token=end, in_place=in_place)
        check(got, clean, total, [0, 6, 12], 6, ended, end, in_place)


@pytest.mark.parametrize("beams", [1, 2, 5, 8, 32])
def test_places(lib, beams):
    """Survivors stay where they are; parents that reorder() reads are never written."""
    rng = np.random.default_rng(beams)
    for _ in range(5):
        logits, total = make(rng, 3 * beams, 700, "f16", 4.0), -2 * rng.random(3 * beams)
        seq0 = np.arange(4) * beams
        got = run(lib, logits, total, seq0, beams, in_place=True, end_token=5)
        check(got, logits, total, seq0, beams, end_token=5, in_place=True)
        p = got["parent"].reshape(-1)
        assert np.array_equal(p[p], p)


def test_outputs_in_the_place_of_inputs(lib):
    rng = np.random.default_rng(12)
    logits = make(rng, 8, 3001, "bf16")
    total, ended = torch.from_numpy((-rng.random(8)).astype(np.float32)).cuda(), torch.tensor([0, 1, 0, 0, 0, 0, 1, 0], device="cuda", dtype=torch.int32)
    want = run(lib, logits, total.cpu().numpy(), [0, 4, 8], 4, ended=ended.cpu().numpy(), end_token=9)
    parent, token = (torch.zeros(2, 4, device="cuda", dtype=torch.int32) for _ in range(2))
    ws = torch.empty(lib.beam_select_workspace_size([0, 4, 8], 3001, 4), dtype=torch.uint8, device="cuda")
    lib.workspace_init(ws)
    lib.beam_select(logits, total, total, parent, token, seq0=[0, 4, 8], ended=ended, ended_out=ended, end_token=9, ws=ws)
    assert np.array_equal(total.cpu().numpy().reshape(2, 4), want["total_out"]) and np.array_equal(ended.cpu().numpy().reshape(2, 4), want["ended_out"])
    assert np.array_equal(parent.cpu().numpy(), want["parent"]) and np.array_equal(token.cpu().numpy(), want["token"])


def test_one_workspace_captured_and_on_streams(lib):
    """Replays follow their inputs; one workspace serves shapes in turn; a captured call has one of its own."""
    rng = np.random.default_rng(13)
    shapes = [([0, 4], 30000, 4), ([0, 8, 16, 24], 9000, 16), ([0, 1], 300, 1), ([0, 32, 64], 2000, 64)]
    size = max(lib.beam_select_workspace_size(s, v, k) for s, v, k in shapes)
    ws = [torch.empty(size, dtype=torch.uint8, device="cuda") for _ in range(2)]
    for w in ws:
        lib.workspace_init(w)
    torch.cuda.synchronize()
    for _ in range(2):
        for seq0, vocab, n_out in shapes:
            logits, total = make(rng, seq0[-1], vocab, "f16"), -rng.random(seq0[-1])
            check(run(lib, logits, total, seq0, n_out, ws=ws[0]), logits, total, seq0, n_out)
    seq0, vocab, n_out = shapes[1]
    logits, total = make(rng, 24, vocab, "f16"), torch.zeros(24, device="cuda")
    out = [torch.zeros(3, n_out, device="cuda")] + [torch.zeros(3, n_out, device="cuda", dtype=torch.int32) for _ in range(2)]
    lib.beam_select(logits, total, *out, seq0=seq0, ws=ws[1])
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        lib.beam_select(logits, total, *out, seq0=seq0, ws=ws[1])
    for _ in range(3):
        logits.copy_(make(rng, 24, vocab, "f16"))
        total.copy_(torch.from_numpy(-rng.random(24)))
        g.replay()
        want = run(lib, logits, total.cpu().numpy(), seq0, n_out, ws=ws[0])
        assert np.array_equal(out[1].cpu().numpy(), want["parent"]) and np.array_equal(out[2].cpu().numpy(), want["token"])
        assert np.array_equal(out[0].cpu().numpy(), want["total_out"])
