"""Append and attention at the largest shapes: segments whose bytes lie past 32
bits of offset, and as many sequences and KV heads as a call may have."""
import numpy as np
import pytest

import _rows as R

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")


def far(lib, c, row0, cap):
    """c's live rows in planes whose sequences begin at rows row0 with `cap` rows a segment; the rest is left as it was
    allocated."""
    rows = max(r + c.n_kv * n for r, n in zip(row0, cap))
    d = {n: None if t is None else torch.empty((rows,) + tuple(t.shape[1:]), dtype=t.dtype, device="cuda") for n, t in c.d.items()
         if n != "n_live"}
    for s in range(len(c.rows)):
        for g in range(c.n_kv):
            a, b = c.row0[s] + g * c.cap[s], row0[s] + g * cap[s]
            for n, t in d.items():
                if t is not None:
                    t[b:b + c.rows[s]].copy_(c.d[n][a:a + c.rows[s]])
    live = c.d["n_live"].clone()
    return d, live, lib.LayerCache(k=d["k"], v=d["v"], k_scale=d["k_scale"], v_scale=d["v_scale"], pos=d["pos"], n_live=live,
                                   seq_row0=row0, capacity=cap, head_dim=c.hd, n_kv_heads=c.n_kv, k_type=c.k_type, v_type=c.v_type)


@pytest.mark.slow
@pytest.mark.parametrize("kind,k,v,base,cap", [
    ("f16", "f16", "f16", 0, 9_000_000),                     # KV head 1 of sequence 0 at 4.6 GB, sequence 1 at 9.2 GB
    ("bf16", "q8_0", "q4_0", 34_000_000, 300),               # codes of 4 bits at 4.35 GB, of 8 bits at 8.7 GB
    ("f32", "f32", "q8_0", 17_000_000, 300)])                # 17.4 and 4.35 GB
def test_offsets_past_32_bits(lib, kind, k, v, base, cap):
    hd, nq = 256, 4
    rng = np.random.default_rng(7)
    c = R.Cache(lib, rng, rows=[200, 90], cap=[260, 150], n_kv=2, hd=hd, k_type=k, v_type=v)
    row0 = [base, base + 2 * cap + 3]
    d, live, cache = far(lib, c, row0, [cap, 300])
    rope = lib.Rope(head_dim=hd, theta=1e4)
    for tokens in (1, 2, 30):
        tok0 = np.array([0, tokens, 2 * tokens], np.int32)
        new = R.act(rng.standard_normal((2 * tokens, nq + 4, hd)), kind)
        pos = np.concatenate([c.last(s) + 1 + np.arange(tokens) for s in range(2)]).astype(np.int32)
        p = torch.from_numpy(pos).cuda()
        q = new[:, :nq].contiguous()
        # the same rows in both caches
        for cc in (cache, c.cache):
            ws = c.ws(lib.workspace_size(c.cache, 0))
            out_q = torch.empty_like(q)
            lib.append_qkv(rope, cc, q, new[:, nq:nq + 2], new[:, nq + 2:], p, ws=ws, q_out=out_q, tok0=tok0)
            assert lib.device_status(ws) == lib.OK
        assert torch.equal(live, c.d["n_live"])
        for s in range(2):
            for g in range(2):
                a, b = c.row0[s] + g * c.cap[s] + c.rows[s], row0[s] + g * int(cache.capacity[s]) + c.rows[s]
                for n, t in d.items():
                    if t is not None:
                        assert torch.equal(t[b:b + tokens].view(torch.uint8), c.d[n][a:a + tokens].view(torch.uint8)), n
        c.rows = [r + tokens for r in c.rows]
        c.h = {n: None if t is None else t.cpu().numpy() for n, t in c.d.items()}
        out, lse = torch.empty_like(q), torch.empty(2 * tokens, nq, device="cuda")
        ws = c.ws(lib.attend_workspace_size(cache, nq, tok0))
        lib.attend(cache, out_q, out, p, tok0=tok0, lse=lse, ws=ws)
        assert lib.device_status(ws) == lib.OK
        want = R.attend_expected(c, R.host(out_q), pos, tok0, nq)
        R.check_attend(R.host(out), R.host(lse), want, kind, kind != "f32", 260, hd, q_exact=kind == "f16", k_exact=k == "f16")


@pytest.mark.parametrize("kind,k,v", [("f16", "f16", "f16"), ("bf16", "q4_0", "q8_0"), ("f32", "f32", "f32")])
@pytest.mark.parametrize("n_kv", [8, 7])
def test_as_many_segments_as_a_call_may_have(lib, kind, k, v, n_kv):
    """128 sequences x 8 KV heads, ragged, some without rows or tokens, decode steps and a few prompts in one call, with and
    without a window; the rows were appended by one call, too."""
    rng = np.random.default_rng(n_kv)
    rows = [int(x) for x in rng.integers(0, 60, 128)]
    rows[0], rows[64], rows[127] = 0, 300, 59
    tokens = [int(x) for x in rng.choice([0, 1, 1, 1, 2, 4], 128)]
    tokens[5], tokens[127] = 20, 9
    hd, nq, n = 64, 2 * n_kv, sum(tokens)
    c = R.Cache(lib, rng, rows=rows, cap=[r + t for r, t in zip(rows, tokens)], n_kv=n_kv, hd=hd, k_type=k, v_type=v)
    tok0 = np.concatenate([[0], np.cumsum(tokens)]).astype(np.int32)
    pos = np.concatenate([c.last(s) + 1 + np.arange(t) for s, t in enumerate(tokens)]).astype(np.int32)
    p = torch.from_numpy(pos).cuda()
    new = R.act(rng.standard_normal((n, nq + 2 * n_kv, hd)), kind)
    q = torch.empty(n, nq, hd, device="cuda", dtype=new.dtype)
    ws = c.ws(lib.workspace_size(c.cache, 0))
    lib.append_qkv(lib.Rope(head_dim=hd, theta=1e4), c.cache, new[:, :nq], new[:, nq:nq + n_kv], new[:, nq + n_kv:], p, ws=ws,
                   q_out=q, tok0=tok0)
    assert lib.device_status(ws) == lib.OK
    c.rows = [r + t for r, t in zip(rows, tokens)]
    assert c.d["n_live"].tolist() == c.rows
    c.h = {name: None if t is None else t.cpu().numpy() for name, t in c.d.items()}
    ws = c.ws(lib.attend_workspace_size(c.cache, nq, tok0))
    for window, sink in ((0, 0), (25, 2)):
        out, lse = torch.empty_like(q), torch.empty(n, nq, device="cuda")
        lib.attend(c.cache, q, out, p, tok0=tok0, lse=lse, window=window, sink=sink, ws=ws)
        assert lib.device_status(ws) == lib.OK
        want = R.attend_expected(c, R.host(q), pos, tok0, nq, window, sink)
        R.check_attend(R.host(out), R.host(lse), want, kind, kind != "f32", max(c.rows), hd, q_exact=kind == "f16", k_exact=k == "f16")
