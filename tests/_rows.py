"""Shared builders of the tests of rotation, append and attention: a layer's
cache on the host, its device copy, and the library's view of it."""
import numpy as np

from oracle import attend_oracle as A

U16, U24 = 2.0 ** -11, 2.0 ** -24
HALF_STEP = {"f32": 2.0 ** -24, "f16": 2.0 ** -11, "bf16": 2.0 ** -8}


def act(x, kind):
    """float32 numpy -> CUDA tensor of the activation type."""
    import torch
    return torch.from_numpy(np.ascontiguousarray(x, np.float32)).cuda().to(
        {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}[kind])


def host(t):
    return t.detach().float().cpu().numpy().astype(np.float64)


class Cache:
    """One layer's cache: rows[s] live rows of sequence s, cap[s] physical ones; rows past the live ones and the
    space between sequences hold NaN / junk that must never matter."""

    def __init__(self, lib, rng, *, rows, cap, n_kv, hd, k_type, v_type, gaps=True, spread=1.0, guard=3):
        import torch
        self.rows, self.cap, self.n_kv, self.hd, self.k_type, self.v_type = list(rows), list(cap), n_kv, hd, k_type, v_type
        self.row0, at = [], guard
        for c in cap:
            self.row0.append(at)
            at += n_kv * c + guard
        total = at
        self.h = {}
        for name, kind in (("k", k_type), ("v", v_type)):
            data, scale = A.hold((rng.standard_normal((total, hd)) * spread).astype(np.float32), kind)
            self.h[name], self.h[name + "_scale"] = data, scale
        self.h["pos"] = np.full(total, 2 ** 30, np.int32)
        self.h["n_live"] = np.asarray(rows, np.int32)
        live = np.zeros(total, bool)
        for s, n in enumerate(rows):
            for g in range(n_kv):
                r0 = self.row0[s] + g * cap[s]
                step = rng.integers(1, 6, n) if gaps else np.ones(n, np.int64)
                p = np.cumsum(step) - 1
                if n:
                    p = p - p[-1] + (5 * n if gaps else n - 1)
                self.h["pos"][r0:r0 + n] = p
                live[r0:r0 + n] = True
        for name in ("k", "v"):
            if self.h[name].dtype.kind == "f":
                self.h[name][~live] = np.nan
            else:
                self.h[name + "_scale"][~live] = np.nan
        self.d = {n: torch.from_numpy(a.copy()).cuda() if a is not None else None for n, a in self.h.items()}
        self.lib = lib
        self.cache = lib.LayerCache(k=self.d["k"], v=self.d["v"], k_scale=self.d["k_scale"], v_scale=self.d["v_scale"],
                                    pos=self.d["pos"], n_live=self.d["n_live"], seq_row0=self.row0, capacity=self.cap,
                                    head_dim=hd, n_kv_heads=n_kv, k_type=k_type, v_type=v_type)

    def seg(self, name, s, g, n=None):
        r0 = self.row0[s] + g * self.cap[s]
        a = self.h[name]
        return None if a is None else a[r0:r0 + (self.rows[s] if n is None else n)]

    def last(self, s):
        """Position of the newest row (the same for every KV head), -1 when there is none."""
        n = self.rows[s]
        return int(self.h["pos"][self.row0[s] + n - 1]) if n else -1

    def values(self, name, s, g):
        kind = self.k_type if name == "k" else self.v_type
        return A.values(self.seg(name, s, g), self.seg(name + "_scale", s, g), kind)

    def ws(self, size):
        import torch
        w = torch.empty(size, dtype=torch.uint8, device="cuda")
        self.lib.workspace_init(w)
        return w


def attend_expected(c, q, pos, tok0, nq, window=0, sink=0, scale=None):
    """(out, lse, tolerance of out per value without the output's own rounding, tolerance of lse) for queries q
    float64 [tokens][nq][hd]. `pieces` of the tolerance: see check_attend."""
    G = nq // c.n_kv
    n_tok = len(pos)
    out, lse = np.zeros((n_tok, nq, c.hd)), np.full((n_tok, nq), -np.inf)
    sum_abs, mag, vmax = np.zeros((n_tok, nq, c.hd)), np.zeros((n_tok, nq)), np.zeros((n_tok, nq))
    for s in range(len(c.rows)):
        for g in range(c.n_kv):
            k, v = c.values("k", s, g), c.values("v", s, g)
            p = c.seg("pos", s, g)
            for t in range(tok0[s], tok0[s + 1]):
                h = slice(g * G, (g + 1) * G)
                o, l, w, m = A.attend_rows(q[t, h], pos[t], k, v, p, window, sink, scale)
                seen = w.sum(0) > 0
                vv = np.where(np.isfinite(v), v, 0) if not seen.all() else v
                out[t, h], lse[t, h], sum_abs[t, h] = o, l, w @ np.abs(vv)
                mag[t, h] = m.max(-1, initial=0.0)
                vmax[t, h] = np.abs(vv[seen]).max(initial=0.0)
    return out, lse, sum_abs, mag, vmax


def check_attend(got, got_lse, want, kind, tensor, rows, hd, q_exact=True, k_exact=True):
    """Tolerances by counting roundings.
    Logits: fp32 sums of hd products are off by at most (hd + 2) 2^-24 of the sum of moduli (mag); on the tensor
    cores a query not exact in fp16 and a dequantised key add half a step of fp16 each, 2^-11 mag. An error dS of
    the logits moves each weight by a factor within exp(+-2 dS).
    Weights: fp32 exponentials and sums, (rows / 32 + 64) 2^-24 at most; on the tensor cores the weight (times the
    value's block scale) and a dequantised value are rounded to fp16 once each, 2 x 2^-11, with 2^-24 vmax a row
    for weights below fp16's normal range (largest weight 1, so the sum of weights is at least 1).
    Output: half a step of its type."""
    out, lse, sum_abs, mag, vmax = want
    dS = (hd + 2) * U24 * mag
    if tensor:
        dS = dS + U16 * mag * ((not q_exact) + (not k_exact))
    rel = np.expm1(2 * dS) + (rows / 32 + 64) * U24 + (2 * U16 if tensor else 0.0)
    tol = rel[..., None] * sum_abs + (rows * U24 * vmax)[..., None] * (1.0 if tensor else 0.0)
    tol = tol + HALF_STEP[kind] * (np.abs(out) + tol) + 2.0 ** -24
    # A token that sees a junk row has no finite value. Over quantised keys it has no defined one either: a block's
    # sum of codes times an infinite scale is an infinity of the sum's sign, possibly -inf (weight 0), where the sum
    # of products has infinities of both signs.
    blown = ~np.isfinite(out)
    if k_exact:
        assert np.array_equal(blown, ~np.isfinite(got))
    else:
        assert np.isfinite(got[~blown]).all()
    bad = np.where(blown, False, np.abs(got - out) > tol)
    assert not bad.any(), f"{bad.sum()} of {bad.size} outputs off, worst {np.max(np.abs(got - out) / tol):.2f} tolerances"
    if got_lse is not None:
        seen = np.isfinite(lse)
        if k_exact:
            assert np.array_equal(seen, np.isfinite(got_lse)) and np.array_equal(got_lse == -np.inf, lse == -np.inf)
        else:
            assert np.isfinite(got_lse[seen]).all() and np.all(got_lse[lse == -np.inf] == -np.inf)
        tl = dS + (rows / 32 + 64) * U24 + U24 * 4 * np.abs(np.where(seen, lse, 0))
        assert np.all(np.abs(got_lse - lse)[seen] <= tl[seen]), np.max((np.abs(got_lse - lse) / tl)[seen])
