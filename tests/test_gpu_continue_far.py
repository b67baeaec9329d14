"""Attention over a shared prefix and reorder at the largest shapes: rows whose
bytes lie past 32 bits of offset, and as many sequences, prefixes and KV heads
as a call may have."""
import numpy as np
import pytest

import _prefix as P
import _rows as R
from test_gpu_rows_far import far

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")


@pytest.mark.slow
@pytest.mark.parametrize("kind,k,v,base,cap", [
    ("f16", "f16", "f16", 0, 9_000_000),                     # KV head 1 of the first at 4.6 GB, the second at 9.2 GB
    ("bf16", "q8_0", "q4_0", 34_000_000, 300),               # codes of 4 bits at 4.35 GB, of 8 bits at 8.7 GB
    ("f16", "q4_0", "q8_0", 17_000_000, 9_000_000),          # the kernel that reads a long prefix for few columns
    ("f32", "f32", "q8_0", 17_000_000, 300)])                # 17.4 and 4.35 GB
def test_offsets_past_32_bits(lib, kind, k, v, base, cap):
    hd, nq, seqs = 256, 4, 7
    rng = np.random.default_rng(7)
    p, c = P.pair(lib, rng, shared=[200, 90], rows=[20] * seqs, n_kv=2, hd=hd, types=(k, v))
    seq0 = [0, 4, seqs]
    newest = P.follow(p, c, seq0)
    row0 = [base, base + 2 * cap + 3]
    _, _, prefix = far(lib, p, row0, [cap, 300])
    _, _, own = far(lib, c, [base + 700 * s for s in range(seqs)], [300] * seqs)
    for tokens in (1, 3, 200):
        t = [tokens] * seqs
        tok0 = np.arange(seqs + 1, dtype=np.int32) * tokens
        pos = np.repeat(newest, tokens).astype(np.int32)
        q = R.act(rng.standard_normal((seqs * tokens, nq, hd)), kind)
        out, lse = torch.empty_like(q), torch.empty(seqs * tokens, nq, device="cuda")
        ws = c.ws(lib.attend_prefix_workspace_size(prefix, own, nq, tok0, seq0))
        lib.attend_prefix(prefix, own, q, out, torch.from_numpy(pos).cuda(), seq0=seq0, tok0=tok0, lse=lse, ws=ws)
        assert lib.device_status(ws) == lib.OK, t
        want = P.expected(p, c, seq0, R.host(q), pos, tok0, nq)
        P.check(R.host(out), R.host(lse), want, kind, kind != "f32", 220, hd, q_exact=kind == "f16", k_exact=k == "f16")


@pytest.mark.slow
@pytest.mark.parametrize("k,v,base,cap", [("f16", "f16", 0, 9_000_000), ("q8_0", "q4_0", 34_000_000, 300), ("f32", "q8_0", 17_000_000, 300)])
def test_reorder_past_32_bits(lib, k, v, base, cap):
    rng = np.random.default_rng(9)
    c = R.Cache(lib, rng, rows=[200, 90, 77], cap=[260, 260, 260], n_kv=2, hd=256, k_type=k, v_type=v)
    row0 = [base, base + 2 * cap + 3, base + 2 * cap + 1000]
    d, live, cache = far(lib, c, row0, [cap, 300, 300])
    for parent in ([1, 0, 2], [2, 2, 2], [0, 0, 1]):
        for cc in (cache, c.cache):
            ws = c.ws(lib.reorder_workspace_size([cc]))
            lib.reorder([cc], torch.tensor(parent, device="cuda", dtype=torch.int32), ws=ws)
            assert lib.device_status(ws) == lib.OK
        assert torch.equal(live, c.d["n_live"])
        for s, n in enumerate(live.tolist()):
            for g in range(2):
                a, b = c.row0[s] + g * c.cap[s], row0[s] + g * int(cache.capacity[s])
                for name, t in d.items():
                    if t is not None:
                        assert torch.equal(t[b:b + n].view(torch.uint8), c.d[name][a:a + n].view(torch.uint8)), name


@pytest.mark.parametrize("kind,k,v", [("f16", "f16", "f16"), ("bf16", "q4_0", "q8_0"), ("f32", "f32", "f32")])
@pytest.mark.parametrize("prefixes", [1, 128, 40])
@pytest.mark.parametrize("n_kv", [8, 7])
def test_as_many_segments_as_a_call_may_have(lib, kind, k, v, prefixes, n_kv):
    """128 sequences x 8 KV heads on one prefix, on one each, and ragged."""
    rng = np.random.default_rng(n_kv)
    rows = [int(x) for x in rng.integers(0, 12, 128)]
    shared = [int(x) for x in rng.integers(0, 200, prefixes)]
    cuts = np.sort(rng.integers(0, 129, prefixes - 1)) if prefixes < 128 else np.arange(1, 128)
    seq0 = [0] + [int(x) for x in cuts] + [128]
    tokens = [int(x) for x in rng.choice([0, 1, 1, 1, 2, 4], 128)]
    p, c = P.pair(lib, rng, shared=shared, rows=rows, n_kv=n_kv, hd=64, types=(k, v))
    newest = P.follow(p, c, seq0)
    tok0 = np.concatenate([[0], np.cumsum(tokens)]).astype(np.int32)
    pos = np.concatenate([n - np.arange(t)[::-1] for n, t in zip(newest, tokens)]).astype(np.int32)
    q = R.act(rng.standard_normal((len(pos), 2 * n_kv, 64)), kind)
    ws = c.ws(lib.attend_prefix_workspace_size(p.cache, c.cache, 2 * n_kv, tok0, seq0))
    for window, sink in ((0, 0), (25, 2)):
        out, lse = torch.empty_like(q), torch.empty(len(pos), 2 * n_kv, device="cuda")
        lib.attend_prefix(p.cache, c.cache, q, out, torch.from_numpy(pos).cuda(), seq0=seq0, tok0=tok0, lse=lse, window=window, sink=sink, ws=ws)
        assert lib.device_status(ws) == lib.OK
        want = P.expected(p, c, seq0, R.host(q), pos, tok0, 2 * n_kv, window, sink)
        P.check(R.host(out), R.host(lse), want, kind, kind != "f32", 220, 64, q_exact=kind == "f16", k_exact=k == "f16")
