"""What is measured of decoding several continuations of one prompt over the library's caches.

Three operators of a loop in which sequences branch from shared prompts (beam search, several answers to one question):

* ``prefix``   attention of the new tokens over the rows of the prompt, held once for all sequences that share it, and
  over each sequence's own rows behind it;
* ``select``   the best continuations of a group of beams: log-probabilities of the vocabulary, running totals, the
  best (beam, token) pairs, each surviving beam in its own place where that is asked for;
* ``reorder``  the caches of the beams follow their parents, in every layer.

``run`` computes them in elementary torch operations where ``own`` is false, and calls the library where it is true.
"""
import math

import numpy as np
import torch

own = False

DTYPE = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


# ------------------------------------------------------------------------------------------------ the cases

def listed():
    return [
        # four beams of one short prompt: latency
        dict(name="prefix_step_short", op="prefix", type="f16", heads=32, kv=8, hd=128, prefixes=1, seqs=4, tokens=1,
             prefix=777, rows=20, spread=0.3, k="f16", v="f16", window=0, sink=0, evicted=False),
        # thirty-two answers to one long prompt, one step
        dict(name="prefix_step_f16", op="prefix", type="f16", heads=32, kv=8, hd=128, prefixes=1, seqs=32, tokens=1,
             prefix=32768, rows=700, spread=0.5, k="f16", v="f16", window=0, sink=0, evicted=True),
        # sixty-four samples of a longer prompt held in 8 bits, after its pass
        dict(name="prefix_step_q8", op="prefix", type="bf16", heads=32, kv=8, hd=128, prefixes=1, seqs=64, tokens=1,
             prefix=65536, rows=300, spread=0.5, k="q8_0", v="q8_0", window=0, sink=0, evicted=True),
        # beam search over a batch of ragged prompts held in 4 bits
        dict(name="prefix_beams_q4", op="prefix", type="bf16", heads=32, kv=8, hd=128, prefixes=6, seqs=48, tokens=1,
             prefix=20011, rows=257, spread=0.6, k="q4_0", v="q4_0", window=0, sink=0, evicted=True),
        # wide heads, a sliding window and first rows that stay visible, two tokens a step
        dict(name="prefix_window_hd256", op="prefix", type="f16", heads=16, kv=4, hd=256, prefixes=4, seqs=24, tokens=2,
             prefix=30000, rows=1000, spread=0.5, k="f16", v="f16", window=4096, sink=4, evicted=True),
        # eight questions of a few hundred tokens behind one document
        dict(name="prefix_chunk", op="prefix", type="f16", heads=32, kv=8, hd=128, prefixes=1, seqs=8, tokens=300,
             prefix=16384, rows=300, spread=0.4, k="f16", v="f16", window=0, sink=0, evicted=False),
        # four beams of a small vocabulary: latency
        dict(name="select_step", op="select", type="f16", groups=1, beams=4, vocab=32000, n_out=4, ragged=False,
             in_place=True, ended=0.0, first=False),
        # a batch of searches over a large vocabulary
        dict(name="select_batch", op="select", type="bf16", groups=16, beams=8, vocab=151936, n_out=8, ragged=False,
             in_place=True, ended=0.1, first=False),
        # wide searches of several widths, an odd vocabulary, twice as many candidates as beams
        dict(name="select_wide_f32", op="select", type="f32", groups=4, beams=32, vocab=50021, n_out=64, ragged=True,
             in_place=False, ended=0.0, first=False),
        # one layer of one search: latency
        dict(name="reorder_layer", op="reorder", layers=1, groups=1, beams=4, kv=8, hd=128, rows=300, k="f16", v="f16"),
        # every layer of a model, four searches of eight beams
        dict(name="reorder_model", op="reorder", layers=36, groups=4, beams=8, kv=8, hd=128, rows=401, k="f16", v="f16"),
        # the same in 8 and 4 bits, one wide search
        dict(name="reorder_model_q", op="reorder", layers=36, groups=1, beams=32, kv=8, hd=128, rows=1003, k="q8_0", v="q4_0"),
    ]


HEADS = ((32, 8, 128), (16, 4, 256), (8, 2, 64), (16, 2, 96), (28, 4, 128), (12, 12, 64))


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("prefix", "prefix", "select", "reorder"))
    if op == "select":
        beams = _log(rng, 1, 32)
        groups = _log(rng, 1, max(1, 128 // beams))
        vocab = _log(rng, 1000, 152000)
        in_place = rng.random() < 0.5
        return dict(op=op, type=rng.choice(("f16", "bf16", "f32")), groups=groups, beams=beams, vocab=vocab,
                    n_out=beams if in_place else rng.randrange(1, min(64, 2 * beams) + 1), ragged=not in_place and rng.random() < 0.5,
                    in_place=in_place, ended=rng.choice((0.0, 0.3)), first=rng.random() < 0.2)
    heads, kv, hd = rng.choice(HEADS)
    if op == "reorder":
        beams = _log(rng, 2, 32)
        layers, groups = _log(rng, 1, 36), _log(rng, 1, max(1, min(128 // beams, 1024 // (kv * beams))))
        rows = _log(rng, 1, max(2, min(4000, 36 * 32 * 8 * 400 // (layers * groups * beams * kv) * 128 // hd)))
        return dict(op=op, layers=layers, groups=groups, beams=beams, kv=kv, hd=hd, rows=rows,
                    k=rng.choice(("f16", "q8_0", "q4_0", "f32")), v=rng.choice(("f16", "q8_0", "q4_0")))
    window, sink = rng.choice(((0, 0), (0, 0), (_log(rng, 16, 8192), rng.choice((0, 1, 4, 64)))))
    kind = rng.choice(("step", "step", "step", "few", "chunk", "f32"))
    seqs = _log(rng, 1, 64)
    case = dict(op=op, type=rng.choice(("f16", "bf16")), heads=heads, kv=kv, hd=hd, prefixes=1, seqs=seqs, tokens=1, prefix=1,
                rows=_log(rng, 1, 1500), spread=rng.choice((0.0, 0.3, 0.7)), k=rng.choice(("f16", "q8_0", "q4_0")),
                v=rng.choice(("f16", "q8_0", "q4_0")), window=window, sink=sink, evicted=rng.random() < 0.7)
    if kind in ("step", "few"):
        case["prefixes"] = rng.randrange(1, min(seqs, 6) + 1)
        case["prefix"] = _log(rng, 1, 64000 // case["prefixes"])
        if kind == "few":
            case["tokens"] = rng.randrange(2, 10)
    elif kind == "chunk":
        case.update(seqs=rng.randrange(1, 7), tokens=_log(rng, 17, 300), prefix=_log(rng, 1, 12000), evicted=False)
    else:
        case.update(type="f32", k=rng.choice(("f32", "f32", "q8_0")), v="f32", seqs=_log(rng, 1, 8), tokens=rng.choice((1, 1, 3)),
                    prefix=_log(rng, 3, 4000))
    case["rows"] = max(case["rows"], case["tokens"])
    return case


# ------------------------------------------------------------------------------------------------ shapes

def _spread(n, s, spread, salt):
    return n - int(n * spread * ((s * 0.6180339887 + salt) % 1.0))


def _offsets(counts):
    return np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)


def _sharers(case):
    """Sequences of each prefix: near equal shares."""
    p, n = case["prefixes"], case["seqs"]
    return [n * (i + 1) // p - n * i // p for i in range(p)]


def _tokens(case):
    return [max(1, _spread(case["tokens"], s, case["spread"], 0.11)) for s in range(case["seqs"])]


def _own_rows(case):
    """Own live rows of each sequence, the new tokens among them."""
    return [max(t, _spread(case["rows"], s, case["spread"], 0.37)) for s, t in enumerate(_tokens(case))]


def _prefix_rows(case):
    return [max(1, _spread(case["prefix"], s, case["spread"], 0.23)) for s in range(case["prefixes"])]


def _widths(case):
    """Beams of each group."""
    return [max(1, _spread(case["beams"], g, 0.5 if case["ragged"] else 0.0, 0.4)) for g in range(case["groups"])]


def _beam_rows(case):
    """Live rows of each group's beams: they grow together."""
    return [max(1, _spread(case["rows"], g, 0.3, 0.7)) for g in range(case["groups"])]


def _row_bytes(kind, hd):
    return {"f32": 4 * hd, "f16": 2 * hd, "q8_0": hd + hd // 16, "q4_0": hd // 2 + hd // 16}[kind]


GAP = 1.0 + 0.25 * 4.5       # mean distance of old rows: a quarter of them have 1 .. 8 evicted tokens before them


def work(case):
    if case["op"] == "select":
        size = 4 if case["type"] == "f32" else 2
        beams = sum(_widths(case))
        return {"bytes": beams * (case["vocab"] * size + 8) + 12 * case["groups"] * case["n_out"], "flops": 4 * beams * case["vocab"]}
    if case["op"] == "reorder":
        row = _row_bytes(case["k"], case["hd"]) + _row_bytes(case["v"], case["hd"]) + 4
        moved = 0
        for g, n in enumerate(_beam_rows(case)):
            p = _family(case, g)
            away = [b for b in range(case["beams"]) if p[b] != b]
            moved += n * (len(away) + len({p[b] for b in away}))
        return {"bytes": case["layers"] * (case["kv"] * row * moved + 4 * case["groups"] * case["beams"]), "flops": 0}
    size = 4 if case["type"] == "f32" else 2
    hd, heads, kv, w = case["hd"], case["heads"], case["kv"], case["window"]
    t, own_n, pre, m = _tokens(case), _own_rows(case), _prefix_rows(case), _sharers(case)
    pairs, read, s = 0.0, 0.0, 0
    for p in range(case["prefixes"]):
        most = 0
        for _ in range(m[p]):
            near, far = own_n[s] - (t[s] - 1) / 2, pre[p]
            if w:
                near = min(near, w)
                left = max(0.0, w - own_n[s])
                close = min(far, 512) if case["evicted"] else far
                far = min(far, (left if left <= close else close + (left - close) / GAP) + min(far, case["sink"]))
            pairs += t[s] * (near + far)
            read += min(own_n[s], near + t[s])
            most = max(most, far)
            s += 1
        read += most
    b = kv * read * (_row_bytes(case["k"], hd) + _row_bytes(case["v"], hd))
    b += sum(t) * heads * (2 * hd * size + 4) + 4 * sum(t)
    return {"bytes": int(b), "flops": int(4 * hd * heads * pairs)}


# ------------------------------------------------------------------------------------------------ inputs

def _family(case, g):
    """Which beam each of a group's places comes from after one step: every surviving beam stays in its place, the
    places of the others go to second children. Between a quarter and three quarters of the beams survive."""
    n = case["beams"]
    keep = max(1, round(n * (0.25 + 0.5 * ((g * 0.6180339887 + 0.5) % 1.0))))
    alive = sorted(range(n), key=lambda b: (b * 0.7548776662 + g * 0.31) % 1.0)[:keep]
    return [b if b in alive else alive[(7 * b + g) % keep] for b in range(n)]


def _normal(gen, *shape):
    return torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32)


def _hold(x, kind):
    """x [..., hd] float32 as planes of the cache: (data, scale or None)."""
    if kind in ("f32", "f16"):
        return x.to(DTYPE[kind]), None
    b = x.reshape(*x.shape[:-1], x.shape[-1] // 32, 32)
    if kind == "q8_0":
        d = b.abs().amax(-1, keepdim=True) / 127.0
        code = torch.round(b / torch.where(d > 0, d, torch.ones_like(d))).clamp(-127, 127)
        return code.to(torch.int8).reshape(x.shape), d.squeeze(-1).half()
    d = b.gather(-1, b.abs().argmax(-1, keepdim=True)) / -8.0
    code = torch.floor(b / torch.where(d == 0, torch.ones_like(d), d) + 8.5).clamp(0, 15)
    code = torch.where(d == 0, torch.full_like(code, 8.0), code).to(torch.uint8)
    data = code[..., :16] | (code[..., 16:] << 4)
    return data.reshape(*x.shape[:-1], x.shape[-1] // 2), (d + 0.0).squeeze(-1).half()


def _values(data, scale, kind):
    """The float32 values that planes of the cache stand for."""
    if kind in ("f32", "f16"):
        return data.float()
    if kind == "q8_0":
        b = data.float().reshape(*scale.shape, 32)
    else:
        b = data.reshape(*scale.shape, 16)
        b = torch.cat([(b & 15).float(), (b >> 4).float()], -1) - 8.0
    return (b * scale.float()[..., None]).reshape(*scale.shape[:-1], scale.shape[-1] * 32)


def _planes(gen, case, n, cap):
    """Keys and values of n sequences of cap rows."""
    planes = {}
    for name, kind in (("k", case["k"]), ("v", case["v"])):
        x = torch.empty(n, case["kv"], cap, case["hd"], device="cuda", dtype=torch.float32 if kind == "f32" else torch.float16)
        x.normal_(generator=gen)
        planes[name], planes[name + "_scale"] = (x, None) if kind == "f16" else _hold(x.float(), kind)
    return planes


def _positions(gen, case, rows, cap, evicted, near):
    """Positions of the rows of a cache, from 0 up: as an eviction leaves them (old rows thinned out head by head, the
    newest ones all there) or one after the other; and each sequence's next position."""
    n = len(rows)
    live = torch.tensor(rows, device="cuda")[:, None, None]
    at = torch.arange(cap, device="cuda")[None, None]
    gap = torch.ones(n, case["kv"], cap, device="cuda")
    if evicted:
        u = torch.rand(gap.shape, generator=gen, device="cuda")
        gap = torch.where((at < live - near) & (u < 0.25), 2.0 + torch.floor(u * 32.0), gap)
    pos = torch.cumsum(gap.double(), -1).long()
    nxt = (3 if evicted else 1) * live
    pos = pos - pos.gather(-1, (live - 1).expand(n, case["kv"], 1)) + nxt - 1
    return torch.where(at < live, pos, torch.zeros_like(pos)), nxt[:, 0, 0]


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    st = {"case": case}
    if case["op"] == "select":
        widths, v, dt = _widths(case), case["vocab"], DTYPE[case["type"]]
        n = sum(widths)
        # most of the vocabulary far below a few likely tokens; beams of a group differ in their totals
        x = _normal(gen, n, v) * 2.0
        likely = torch.randint(0, v, (n, 24), generator=gen, device="cuda")
        x.scatter_add_(1, likely, 4.0 + 6.0 * torch.rand(n, 24, generator=gen, device="cuda"))
        st["seq0"], st["logits"] = _offsets(widths), x.to(dt)
        st["total"] = -20.0 - 3.0 * torch.rand(n, generator=gen, device="cuda")
        if case["first"]:                                  # the first step: one beam of each group stands for all
            st["total"][:] = -math.inf
            st["total"][torch.from_numpy(st["seq0"][:-1]).cuda().long()] = 0.0
        st["ended"] = (torch.rand(n, generator=gen, device="cuda") < case["ended"]).int() if case["ended"] else None
        st["end_token"] = 2
        for name, kind in (("total_out", torch.float32), ("parent", torch.int32), ("token", torch.int32), ("ended_out", torch.int32)):
            st[name] = torch.empty(case["groups"], case["n_out"], device="cuda", dtype=kind)
        st["plan"] = _plan(st) if own else None
        return st
    if case["op"] == "reorder":
        layers, n, kv, hd = case["layers"], case["groups"] * case["beams"], case["kv"], case["hd"]
        rows = [r for r in _beam_rows(case) for _ in range(case["beams"])]
        cap = max(rows) + 36
        parts = [_planes(gen, case, n, cap) for _ in range(layers)]
        st["planes"] = {k: None if parts[0][k] is None else torch.stack([p[k] for p in parts]) for k in parts[0]}
        del parts
        st["planes"]["pos"] = (torch.arange(cap, device="cuda", dtype=torch.int32) +
                               torch.randint(0, 9, (layers, n, kv, 1), generator=gen, device="cuda", dtype=torch.int32)).contiguous()
        st["n_live"] = torch.tensor(rows, device="cuda", dtype=torch.int32).repeat(layers, 1)
        st["seq0"] = _offsets([case["beams"]] * case["groups"])
        st["parent"] = torch.tensor([g * case["beams"] + b for g in range(case["groups"]) for b in _family(case, g)],
                                    device="cuda", dtype=torch.int32)
        st["cap"], st["row0"] = cap, np.arange(n, dtype=np.int64) * kv * cap
        st["plan"] = _plan(st) if own else None
        return st
    heads, kv, hd, dt = case["heads"], case["kv"], case["hd"], DTYPE[case["type"]]
    t, rows, pre, m = _tokens(case), _own_rows(case), _prefix_rows(case), _sharers(case)
    n, seqs = sum(t), case["seqs"]
    st["n"], st["tok0"], st["seq0"] = n, _offsets(t), _offsets(m)
    st["cap"], st["prefix_cap"] = max(rows) + 37, max(pre) + 21
    st["row0"] = np.arange(seqs, dtype=np.int64) * kv * st["cap"]
    st["prefix_row0"] = np.arange(case["prefixes"], dtype=np.int64) * kv * st["prefix_cap"]
    st["prefix"], st["own"] = _planes(gen, case, case["prefixes"], st["prefix_cap"]), _planes(gen, case, seqs, st["cap"])
    pos, behind = _positions(gen, case, pre, st["prefix_cap"], case["evicted"], 512)
    st["prefix"]["pos"] = pos.int().contiguous()
    of = torch.repeat_interleave(torch.arange(case["prefixes"], device="cuda"), torch.tensor(m, device="cuda"))
    pos, nxt = _positions(gen, case, rows, st["cap"], case["evicted"] and case["rows"] > 600, max(t))
    live = torch.tensor(rows, device="cuda")
    pos = torch.where(torch.arange(st["cap"], device="cuda")[None, None] < live[:, None, None], pos + behind[of][:, None, None], pos)
    st["own"]["pos"] = pos.int().contiguous()
    seq = torch.repeat_interleave(torch.arange(seqs, device="cuda"), torch.tensor(t, device="cuda"))
    st["seq"], st["at"] = seq, torch.arange(n, device="cuda") - torch.from_numpy(st["tok0"][:-1]).cuda().long()[seq]
    st["pos"] = ((behind[of] + nxt - torch.tensor(t, device="cuda"))[seq] + st["at"]).int()
    st["n_live"], st["prefix_live"] = live.int(), torch.tensor(pre, device="cuda", dtype=torch.int32)
    heat = torch.exp(torch.rand(1, heads, 1, generator=gen, device="cuda") * 2.0 - 0.7)   # flat heads and peaked ones
    st["q"] = (_normal(gen, n, heads, hd) * heat).to(dt)
    st["out"] = torch.empty(n, heads, hd, device="cuda", dtype=dt)
    st["lse"] = torch.empty(n, heads, device="cuda", dtype=torch.float32)
    st["plan"] = _plan(st) if own else None
    return st


# ------------------------------------------------------------------------------------------------ the library's calls

def _cache(tria, case, planes, n_live, row0, cap):
    return tria.LayerCache(k=planes["k"], v=planes["v"], k_scale=planes["k_scale"], v_scale=planes["v_scale"], pos=planes["pos"],
                           n_live=n_live, seq_row0=row0, capacity=[cap] * len(row0), head_dim=case["hd"],
                           n_kv_heads=case["kv"], k_type=case["k"], v_type=case["v"])


def _plan(st):
    """What a program over the library keeps: the caches, the workspace."""
    import kv_cache_eviction_tria_gb300 as tria
    case = st["case"]
    plan = {"tria": tria}
    if case["op"] == "select":
        size = tria.beam_select_workspace_size(st["seq0"], case["vocab"], case["n_out"])
    elif case["op"] == "reorder":
        plan["caches"] = [_cache(tria, case, {k: None if x is None else x[i] for k, x in st["planes"].items()},
                                 st["n_live"][i], st["row0"], st["cap"]) for i in range(case["layers"])]
        size = tria.reorder_workspace_size(plan["caches"], st["seq0"])
    else:
        plan["prefix"] = _cache(tria, case, st["prefix"], st["prefix_live"], st["prefix_row0"], st["prefix_cap"])
        plan["own"] = _cache(tria, case, st["own"], st["n_live"], st["row0"], st["cap"])
        size = tria.attend_prefix_workspace_size(plan["prefix"], plan["own"], case["heads"], st["tok0"], st["seq0"])
    plan["ws"] = torch.empty(size, device="cuda", dtype=torch.uint8)
    tria.workspace_init(plan["ws"])
    return plan


def _own_run(st):
    plan, case = st["plan"], st["case"]
    tria = plan["tria"]
    if case["op"] == "select":
        tria.beam_select(st["logits"], st["total"], st["total_out"], st["parent"], st["token"], seq0=st["seq0"], ended=st["ended"],
                         ended_out=st["ended_out"], end_token=st["end_token"], in_place=case["in_place"], ws=plan["ws"])
        return _selected(st)
    if case["op"] == "reorder":
        tria.reorder(plan["caches"], st["parent"], seq0=st["seq0"], ws=plan["ws"])
        return _moved(st)
    tria.attend_prefix(plan["prefix"], plan["own"], st["q"], st["out"], st["pos"], seq0=st["seq0"], tok0=st["tok0"],
                       lse=st["lse"], window=case["window"], sink=case["sink"], ws=plan["ws"])
    return {"out": st["out"], "lse": st["lse"]}


def _selected(st):
    return {name: st[name] for name in ("total_out", "parent", "token", "ended_out")}


def _moved(st):
    out = {k: x for k, x in st["planes"].items() if x is not None}
    out["n_live"] = st["n_live"]
    return out


# ------------------------------------------------------------------------------------------------ the plain forms

def run(state):
    if own:
        return _own_run(state)
    return {"select": _select, "reorder": _reorder, "prefix": _prefix}[state["case"]["op"]](state)


def _settled(parent, token, total, first, width):
    """A group's choices (best first), each beam's best one in the beam's own place, the others in the places left."""
    local = parent - first
    n = len(local)
    earlier = (local[:, None] == local[None, :]) & torch.ones(n, n, device="cuda", dtype=torch.bool).tril(-1)
    stays = ~earlier.any(1)
    place = torch.empty_like(local)
    place[stays] = local[stays]
    taken = torch.zeros(width, device="cuda", dtype=torch.bool)
    taken[local[stays]] = True
    place[~stays] = torch.nonzero(~taken).flatten()
    back = torch.argsort(place)
    return parent[back], token[back], total[back]


def _select(st):
    case, v = st["case"], st["case"]["vocab"]
    x = st["logits"].double()                              # neighbouring totals differ by less than 32 bits hold
    top = x.amax(1, keepdim=True)
    total = x - top - torch.log(torch.exp(x - top).sum(1, keepdim=True)) + st["total"].double()[:, None]
    if st["ended"] is not None:                            # a search that is over goes on as it is
        over = st["ended"].bool()
        total = total.masked_fill(over[:, None], -math.inf)
        total[:, st["end_token"]] = torch.where(over, st["total"].double(), total[:, st["end_token"]])
    seq0 = st["seq0"].tolist()
    for g in range(case["groups"]):
        a, b = seq0[g], seq0[g + 1]
        val, at = torch.sort(total[a:b].flatten(), descending=True, stable=True)
        val, at = val[:case["n_out"]], at[:case["n_out"]]
        parent, token = a + torch.div(at, v, rounding_mode="floor"), at % v
        if case["in_place"]:
            parent, token, val = _settled(parent, token, val, a, b - a)
        st["total_out"][g], st["parent"][g], st["token"][g] = val.float(), parent.int(), token.int()
    ended = st["token"] == st["end_token"]
    if st["ended"] is not None:
        ended = ended | (st["ended"][st["parent"].long()] != 0)
    st["ended_out"].copy_(ended.int())
    return _selected(st)


def _reorder(st):
    case, parent = st["case"], st["parent"].long()
    live = st["n_live"][:, parent]
    row = torch.arange(st["cap"], device="cuda")
    moves = (row < live[:, :, None]) & (parent != torch.arange(len(parent), device="cuda"))[None, :, None]
    for x in st["planes"].values():
        if x is not None:
            m = moves[:, :, None, :, None] if x.dim() == 5 else moves[:, :, None]
            x.copy_(torch.where(m, x[:, parent], x))
    st["n_live"].copy_(live)
    return _moved(st)


def _sees(case, pos_rows, p, n_live, sink):
    row = torch.arange(pos_rows.shape[-1], device="cuda")
    see = (row < n_live) & (pos_rows <= p)
    if case["window"]:
        see = see & ((p - pos_rows < case["window"]) | (row < sink))
    return see


def _softmax(logit, v):
    """(largest logit, sum of weights, weighted sum of v) of the last axis."""
    top = logit.amax(-1, keepdim=True)
    e = torch.exp(logit - top.masked_fill(top == -math.inf, 0.0))
    return top, e.sum(-1, keepdim=True), e.flatten(-3, -2) @ v


def _prefix(st):
    case = st["case"]
    hd, heads, kv, seqs, n = case["hd"], case["heads"], case["kv"], case["seqs"], st["n"]
    group, dt, tok0, seq0 = heads // kv, DTYPE[case["type"]], st["tok0"], st["seq0"]
    q = st["q"].float().reshape(n, kv, group, hd).permute(1, 0, 2, 3) * hd ** -0.5     # [kv][token][group][hd]
    # the shared rows: all tokens of a prefix's sequences together
    parts = []
    for p in range(case["prefixes"]):
        a, b = int(tok0[seq0[p]]), int(tok0[seq0[p + 1]])
        x = {k: None if y is None else y[p] for k, y in st["prefix"].items()}
        logit = (q[:, a:b].reshape(kv, -1, hd) @ _values(x["k"], x["k_scale"], case["k"]).transpose(-1, -2)).reshape(kv, b - a, group, -1)
        see = _sees(case, x["pos"][:, None], st["pos"][a:b][None, :, None], st["prefix_live"][p], case["sink"])
        top, total, out = _softmax(logit.masked_fill(~see[:, :, None], -math.inf), _values(x["v"], x["v_scale"], case["v"]))
        parts.append((top, total, out.reshape(kv, b - a, group, hd)))
        del logit, see
    top, total, out = (torch.cat(x, 1) for x in zip(*parts))
    # each sequence's own rows
    tm = int(st["at"].max()) + 1
    own_q = torch.zeros(seqs, kv, tm, group, hd, device="cuda", dtype=torch.float32)
    own_q[st["seq"], :, st["at"]] = q.permute(1, 0, 2, 3)
    at = torch.full((seqs, tm), -1, device="cuda", dtype=torch.int32)
    at[st["seq"], st["at"]] = st["pos"]
    x = st["own"]
    logit = (own_q.reshape(seqs, kv, tm * group, hd) @ _values(x["k"], x["k_scale"], case["k"]).transpose(-1, -2)).reshape(seqs, kv, tm, group, -1)
    see = _sees(case, x["pos"][:, :, None], at[:, None, :, None], st["n_live"][:, None, None, None], 0)
    t2, l2, o2 = _softmax(logit.masked_fill(~see[:, :, :, None], -math.inf), _values(x["v"], x["v_scale"], case["v"]))
    o2 = o2.reshape(seqs, kv, tm, group, hd)
    t2, l2, o2 = (y.permute(0, 2, 1, 3, 4)[st["seq"], st["at"]].permute(1, 0, 2, 3) for y in (t2, l2, o2))
    both = torch.maximum(top, t2)
    base = both.masked_fill(both == -math.inf, 0.0)
    w1, w2 = torch.exp(top - base), torch.exp(t2 - base)
    total = total * w1 + l2 * w2
    out = (out * w1 + o2 * w2) / torch.where(total > 0, total, torch.ones_like(total))
    st["out"].copy_(out.permute(1, 0, 2, 3).reshape(n, heads, hd).to(dt))
    st["lse"].copy_((both + torch.log(total)).squeeze(-1).permute(1, 0, 2).reshape(n, heads))
    return {"out": st["out"], "lse": st["lse"]}


# ------------------------------------------------------------------------------------------------ in 64 bits

def exact(case, seed):
    st = prepare(case, seed)
    f64 = torch.float64
    if case["op"] == "reorder":                            # values are moved, row by row
        out = {"n_live": None}
        for name, x in st["planes"].items():
            if x is None:
                continue
            out[name] = x.to(f64) if x.dtype.is_floating_point else None
            if out[name] is not None:
                for s, p in enumerate(st["parent"].tolist()):
                    n = int(st["n_live"][0, p])
                    out[name][:, s, :, :n] = x[:, p, :, :n].to(f64)
        return out
    if case["op"] == "select":
        out = np.empty((case["groups"], case["n_out"]))
        seq0, v = st["seq0"].tolist(), case["vocab"]
        for g in range(case["groups"]):
            x = st["logits"][seq0[g]:seq0[g + 1]].to(f64).cpu().numpy()
            t = st["total"][seq0[g]:seq0[g + 1]].to(f64).cpu().numpy()
            big = x.max(1)
            y = x + (t - big - np.log(np.exp(x - big[:, None]).sum(1)))[:, None]
            if st["ended"] is not None:
                for b in np.flatnonzero(st["ended"][seq0[g]:seq0[g + 1]].cpu().numpy()):
                    y[b], y[b, st["end_token"]] = -np.inf, t[b]
            y = y.reshape(-1)
            # the best ones, equal ones by their index
            cut = np.partition(y, len(y) - case["n_out"])[len(y) - case["n_out"]]
            some = np.flatnonzero(y >= cut)
            best = some[np.lexsort((some, -y[some]))][:case["n_out"]]
            if case["in_place"]:
                places, rest = {}, []
                for c in best:
                    if c // v in places:
                        rest.append(c)
                    else:
                        places[c // v] = c
                free = [b for b in range(case["n_out"]) if b not in places]
                places.update(zip(free, rest))
                best = np.array([places[b] for b in range(case["n_out"])])
            out[g] = y[best]
        return {"total_out": torch.from_numpy(out).cuda(), "parent": None, "token": None, "ended_out": None}
    hd, heads, kv = case["hd"], case["heads"], case["kv"]
    group = heads // kv

    def held(data, scale, kind):
        if kind[0] == "f":
            return data.to(f64)
        s = scale.to(f64).repeat_interleave(32, -1)
        if kind == "q8_0":
            return data.to(f64) * s
        b = data.reshape(*scale.shape, 16).to(torch.int64)
        return (torch.cat([b % 16, b // 16], -1).reshape(*scale.shape[:-1], hd).to(f64) - 8) * s

    def rows(cache, live, s, g):
        n = int(live[s])
        return [held(cache[x][s, g, :n], None if cache[x + "_scale"] is None else cache[x + "_scale"][s, g, :n], case[x]) for x in ("k", "v")] + \
            [cache["pos"][s, g, :n].long()]

    out = torch.zeros(st["n"], heads, hd, device="cuda", dtype=f64)
    lse = torch.full((st["n"], heads), -math.inf, device="cuda", dtype=f64)
    tok0, seq0 = st["tok0"].tolist(), st["seq0"].tolist()
    for p in range(case["prefixes"]):
        for g in range(kv):
            pk, pv, pp = rows(st["prefix"], st["prefix_live"].tolist(), p, g)
            for s in range(seq0[p], seq0[p + 1]):
                a, b = tok0[s], tok0[s + 1]
                k, v, where = rows(st["own"], st["n_live"].tolist(), s, g)
                k, v, where = torch.cat([pk, k]), torch.cat([pv, v]), torch.cat([pp, where])[None]
                at = st["pos"][a:b].long()[:, None]
                hidden = where > at
                if case["window"]:
                    old = at - where >= case["window"]
                    old[:, :min(case["sink"], len(pp))] = False
                    hidden = hidden | old
                x = torch.einsum("thd,nd->thn", st["q"][a:b, g * group:(g + 1) * group].to(f64), k) / math.sqrt(hd)
                x[hidden[:, None].expand_as(x)] = -math.inf
                total = torch.logsumexp(x, -1)
                lse[a:b, g * group:(g + 1) * group] = total
                w = torch.exp(x - torch.where(total == -math.inf, 0.0, total)[..., None])
                out[a:b, g * group:(g + 1) * group] = torch.einsum("thn,nd->thd", w, v)
    return {"out": out, "lse": lse}
