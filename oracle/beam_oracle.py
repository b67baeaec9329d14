"""Plain 64-bit forms of one step of beam search and of the caches that follow
it. Test infrastructure (numpy, float64), sharing nothing with the library:
every continuation is valued and the whole list sorted.
"""
from __future__ import annotations

import numpy as np


def values(logits, total, ended=None, end_token=-1):
    """v [beams][vocab] float64 of every continuation."""
    x = np.asarray(logits, np.float64)
    out = np.full(x.shape, -np.inf)
    for b, row in enumerate(x):
        t = float(total[b])
        if not np.isfinite(t):
            continue
        if ended is not None and ended[b]:
            out[b, end_token] = t
            continue
        top = row.max()
        if np.isnan(row).any() or not np.isfinite(top):
            continue
        out[b] = t + row - (top + np.log(np.exp(row - top).sum()))
    return out


def choose(v, first, n_out, in_place=False, logits=None):
    """The n_out best of a group's values v [beams][vocab]: (beam index among all, token, value) by place. logits: of equal
    values, those of a beam keep their logits' order."""
    beams, vocab = v.shape
    flat = v.reshape(-1)
    x = np.where(v > -np.inf, 0.0 if logits is None else logits, -np.inf).reshape(-1)
    best = [int(i) for i in np.lexsort((np.arange(flat.size), -x, np.arange(flat.size) // vocab, -flat))[:n_out]]
    if in_place:
        place, rest = {}, []
        for i in best:
            if i // vocab in place:
                rest.append(i)
            else:
                place[i // vocab] = i
        for p in range(beams):
            if p not in place:
                place[p] = rest.pop(0)
        best = [place[p] for p in range(beams)]
    return [(first + i // vocab, i % vocab, flat[i]) for i in best]


def reorder(planes, n_live, parent, seq_row0, capacity, n_kv):
    """Planes {name: rows [rows][...]} and n_live [n_seqs] after every sequence took its parent's live rows."""
    out = {k: a.copy() for k, a in planes.items()}
    for s, p in enumerate(parent):
        n = int(n_live[p])
        for g in range(n_kv):
            a, b = seq_row0[s] + g * capacity[s], seq_row0[p] + g * capacity[p]
            for k in out:
                out[k][a:a + n] = planes[k][b:b + n]
    return out, np.asarray([n_live[p] for p in parent], np.int32)
