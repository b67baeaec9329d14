"""Shared builders of the tests of attention over a shared prefix: both caches,
one joint softmax in 64 bits, and the tolerances of the joined results."""
import numpy as np

import _rows as R
from oracle import attend_oracle as A


def pair(lib, rng, *, shared, rows, n_kv, hd, types, own_types=None, gaps=True, spare=5, own_spare=None, spread=1.0):
    """(prefix cache of shared[i] rows, cache of rows[s] own rows whose positions follow() moves behind the prefixes')."""
    k, v = types
    ok, ov = own_types or types
    p = R.Cache(lib, rng, rows=shared, cap=[n + spare for n in shared], n_kv=n_kv, hd=hd, k_type=k, v_type=v, gaps=gaps, spread=spread)
    room = spare if own_spare is None else own_spare
    c = R.Cache(lib, rng, rows=rows, cap=[n + room for n in rows], n_kv=n_kv, hd=hd, k_type=ok, v_type=ov, gaps=gaps, spread=spread)
    return p, c


def follow(p, c, seq0):
    """Moves the own rows' positions behind their prefix's; the position of each sequence's newest row."""
    import torch
    newest = []
    for i in range(len(seq0) - 1):
        for s in range(seq0[i], seq0[i + 1]):
            for g in range(c.n_kv):
                r0 = c.row0[s] + g * c.cap[s]
                c.h["pos"][r0:r0 + c.rows[s]] += p.last(i) + 1
            newest.append(c.last(s) if c.rows[s] else p.last(i) + 1)
    c.d["pos"].copy_(torch.from_numpy(c.h["pos"]))
    return newest


def expected(p, c, seq0, q, pos, tok0, nq, window=0, sink=0, scale=None):
    """As _rows.attend_expected, over both caches."""
    G = nq // c.n_kv
    n_tok = len(pos)
    out, lse = np.zeros((n_tok, nq, c.hd)), np.full((n_tok, nq), -np.inf)
    sum_abs, mag, vmax = np.zeros((n_tok, nq, c.hd)), np.zeros((n_tok, nq)), np.zeros((n_tok, nq))
    for i in range(len(seq0) - 1):
        for g in range(c.n_kv):
            pk, pv, pp = p.values("k", i, g), p.values("v", i, g), p.seg("pos", i, g)
            for s in range(seq0[i], seq0[i + 1]):
                k, v = np.concatenate([pk, c.values("k", s, g)]), np.concatenate([pv, c.values("v", s, g)])
                where = np.concatenate([pp, c.seg("pos", s, g)])
                for t in range(tok0[s], tok0[s + 1]):
                    h = slice(g * G, (g + 1) * G)
                    o, l, w, m = A.attend_rows(q[t, h], pos[t], k, v, where, window, min(sink, len(pp)), scale)
                    seen = w.sum(0) > 0
                    vv = np.where(np.isfinite(v), v, 0) if not seen.all() else v
                    out[t, h], lse[t, h], sum_abs[t, h] = o, l, w @ np.abs(vv)
                    mag[t, h] = m.max(-1, initial=0.0)
                    vmax[t, h] = np.abs(vv[seen]).max(initial=0.0)
    return out, lse, sum_abs, mag, vmax


def check(got, got_lse, want, kind, tensor, rows, hd, q_exact=True, k_exact=True):
    """_rows.check_attend's tolerances of either part, and what joining them adds. A part's log-sum-exp l is off by dl =
    dS + (rows / 32 + 64) 2^-24 of its sum and 4 x 2^-24 |l| of its own roundings, of which the weight e^(l - lse) moves
    the result: |l| e^(l - lse) <= |lse| + 1 for l <= lse. Weights then move by a factor within exp(+-2 dl); the join's
    exponentials, sums and products are 8 roundings of 2^-24 more."""
    out, lse, sum_abs, mag, vmax = want
    U24 = R.U24
    big = np.abs(np.where(np.isfinite(lse), lse, 0)) + 1
    dl = (rows / 32 + 64) * U24 + 4 * U24 * big
    join = np.expm1(2 * dl) + 8 * U24
    dS = (hd + 2) * U24 * mag
    if tensor:
        dS = dS + R.U16 * mag * ((not q_exact) + (not k_exact))
    rel = np.expm1(4 * dS) + (rows / 32 + 64) * U24 + (2 * R.U16 if tensor else 0.0) + join
    tol = rel[..., None] * sum_abs + (rows * U24 * vmax)[..., None] * (1.0 if tensor else 0.0)
    tol = tol + R.HALF_STEP[kind] * (np.abs(out) + tol) + 2.0 ** -24
    blown = ~np.isfinite(out)
    assert np.array_equal(blown, ~np.isfinite(got)) if k_exact else np.isfinite(got[~blown]).all()
    with np.errstate(invalid="ignore"):
        bad = np.where(blown, False, np.abs(got - out) > tol)
        assert not bad.any(), f"{bad.sum()} of {bad.size} outputs off, worst {np.nanmax(np.abs(got - out) / tol):.2f} tolerances"
        if got_lse is not None:
            seen = np.isfinite(lse)
            assert np.array_equal(got_lse == -np.inf, lse == -np.inf) and np.isfinite(got_lse[seen]).all()
            tl = (hd + 2) * U24 * mag + 2 * dl                     # the keys' exact values, whatever their type
            assert np.all(np.abs(got_lse - lse)[seen] <= tl[seen]), np.max((np.abs(got_lse - lse) / tl)[seen])
