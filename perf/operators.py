"""What is measured of the operators around the cache: making its rows and reading them.

Three operators of a decode loop over the library's cache layout:

* ``rotate``  rotary positions with the per-head norm of queries and keys in the same pass;
* ``append``  the same, written into the cache: queries out, keys and values quantised to the cache's type behind
  the live rows of every KV head;
* ``attend``  attention of the new queries over the cache (per-head rows and positions, as an eviction leaves them),
  with a sliding window and first rows that stay visible, over fp16, q8_0, q4_0 and fp32 rows.

``run`` computes them in elementary torch operations where ``own`` is false, and calls the library where it is true.
"""
import math

import numpy as np
import torch

own = False

DTYPE = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
EPS = 1e-6


# ------------------------------------------------------------------------------------------------ the cases

def listed():
    return [
        # one decode step of one sequence of a Qwen3-8B layer: latency
        dict(name="rotate_step", op="rotate", type="f16", heads=32, kv=8, hd=128, nonrot=0, layout="half",
             scaling="none", norm=True, tokens=1, first=32768, fused=True),
        # a long prompt, far positions, part of the head rotated, interleaved pairs stored as halves
        dict(name="rotate_prompt", op="rotate", type="bf16", heads=32, kv=8, hd=128, nonrot=32,
             layout="interleaved_to_half", scaling="yarn", norm=True, tokens=8191, first=120000, fused=True),
        # one decode step of one sequence into a q8_0 cache: latency
        dict(name="append_step_q8", op="append", type="f16", heads=32, kv=8, hd=128, nonrot=0, layout="half",
             scaling="none", norm=True, seqs=1, tokens=1, rows=6272, spread=0.0, k="q8_0", v="q8_0"),
        # one decode step of a full batch into a 4-bit cache
        dict(name="append_batch_q4", op="append", type="f16", heads=32, kv=8, hd=128, nonrot=0, layout="half",
             scaling="none", norm=True, seqs=64, tokens=1, rows=2048, spread=0.5, k="q4_0", v="q4_0"),
        # ragged prompts of a batch: q8_0 keys, 4-bit values
        dict(name="append_prompts", op="append", type="bf16", heads=32, kv=8, hd=128, nonrot=0, layout="half",
             scaling="bands", norm=True, seqs=8, tokens=4096, rows=0, spread=0.6, k="q8_0", v="q4_0"),
        # a short cache and one token: latency
        dict(name="attend_step_short", op="attend", type="f16", heads=32, kv=8, hd=128, seqs=1, tokens=1, rows=777,
             spread=0.0, k="f16", v="f16", window=0, sink=0, evicted=True),
        # a decode step of eight long sequences, fp16
        dict(name="attend_step_f16", op="attend", type="f16", heads=32, kv=8, hd=128, seqs=8, tokens=1, rows=32768,
             spread=0.4, k="f16", v="f16", window=0, sink=0, evicted=True),
        # the same over a cache held in 4 bits, twice as long
        dict(name="attend_step_q4", op="attend", type="bf16", heads=32, kv=8, hd=128, seqs=8, tokens=1, rows=65536,
             spread=0.4, k="q4_0", v="q4_0", window=0, sink=0, evicted=True),
        # a layer with a sliding window and first rows that stay visible, a batch of q8_0 caches, two tokens a step
        dict(name="attend_window_q8", op="attend", type="f16", heads=32, kv=8, hd=128, seqs=24, tokens=2, rows=20011,
             spread=0.3, k="q8_0", v="q8_0", window=4096, sink=4, evicted=True),
        # wide heads, long ragged batch
        dict(name="attend_step_hd256", op="attend", type="bf16", heads=16, kv=4, hd=256, seqs=8, tokens=1,
             rows=98304, spread=0.6, k="f16", v="f16", window=0, sink=0, evicted=True),
        # a whole prompt
        dict(name="attend_prompt", op="attend", type="f16", heads=32, kv=8, hd=128, seqs=1, tokens=8192, rows=8192,
             spread=0.0, k="f16", v="f16", window=0, sink=0, evicted=False),
        # two chunks of prompts behind evicted 4-bit / q8_0 rows, ragged
        dict(name="attend_chunk_q4", op="attend", type="bf16", heads=32, kv=8, hd=128, seqs=2, tokens=2000,
             rows=20500, spread=0.5, k="q8_0", v="q4_0", window=0, sink=0, evicted=True),
    ]


HEADS = ((32, 8, 128), (16, 4, 256), (8, 2, 64), (16, 2, 96), (28, 4, 128), (12, 12, 64))


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("rotate", "append", "attend", "attend"))
    heads, kv, hd = rng.choice(HEADS)
    if op == "rotate":
        return dict(op=op, type=rng.choice(("f16", "bf16", "f32")), heads=heads, kv=kv, hd=hd,
                    nonrot=rng.choice((0, hd // 2, hd // 4)), layout=rng.choice(("half", "interleaved", "interleaved_to_half")),
                    scaling=rng.choice(("none", "linear", "ntk", "yarn", "bands")), norm=rng.random() < 0.7,
                    tokens=_log(rng, 1, 8191), first=rng.randrange(0, 200000), fused=rng.random() < 0.7)
    if op == "append":
        one = rng.random() < 0.5   # a decode step, or prompts
        tokens = 1 if one else _log(rng, 2, 4096)
        seqs = _log(rng, 1, 100) if one else _log(rng, 1, 8)
        return dict(op=op, type=rng.choice(("f16", "bf16", "f32")), heads=heads, kv=kv, hd=hd,
                    nonrot=rng.choice((0, hd // 2)), layout=rng.choice(("half", "interleaved_to_half")),
                    scaling=rng.choice(("none", "yarn", "bands")), norm=rng.random() < 0.7, seqs=seqs, tokens=tokens,
                    rows=_log(rng, 1, 4000) if rng.random() < 0.7 else 0, spread=rng.choice((0.0, 0.5, 0.9)),
                    k=rng.choice(("f16", "q8_0", "q4_0") if one else ("f16", "q8_0")), v=rng.choice(("f16", "q8_0", "q4_0")))
    kind = rng.choice(("step", "step", "few", "chunk", "f32"))
    window, sink = rng.choice(((0, 0), (0, 0), (_log(rng, 16, 8192), rng.choice((0, 1, 4, 64)))))
    case = dict(op=op, type=rng.choice(("f16", "bf16")), heads=heads, kv=kv, hd=hd, seqs=1, tokens=1, rows=1,
                spread=rng.choice((0.0, 0.3, 0.7)), k=rng.choice(("f16", "q8_0", "q4_0")),
                v=rng.choice(("f16", "q8_0", "q4_0")), window=window, sink=sink, evicted=True)
    if kind in ("step", "few"):
        case["seqs"] = _log(rng, 1, 64)
        case["rows"] = _log(rng, 1, max(2, min(100000, 400000 // case["seqs"])))
        if kind == "few":
            case["tokens"] = rng.randrange(2, 10)
            case["rows"] += case["tokens"]
    elif kind == "chunk":
        case["tokens"] = _log(rng, 17, 2000)
        case["seqs"] = rng.choice((1, 1, 2, 3))
        case["rows"] = case["tokens"] + (0 if rng.random() < 0.3 else _log(rng, 1, 12000))
    else:
        case.update(type="f32", k=rng.choice(("f32", "f32", "q8_0")), v="f32", seqs=_log(rng, 1, 8),
                    tokens=rng.choice((1, 1, 3)), rows=_log(rng, 3, 4000))
    return case


# ------------------------------------------------------------------------------------------------ shapes

def _spread(n, s, spread, salt):
    return n - int(n * spread * ((s * 0.6180339887 + salt) % 1.0))


def _tokens(case):
    """New tokens of each sequence."""
    if case["op"] == "rotate":
        return [case["tokens"]]
    return [max(1, _spread(case["tokens"], s, case["spread"], 0.11)) for s in range(case["seqs"])]


def _rows(case):
    """Live rows of each sequence: before the call (append), with the new tokens among them (attend)."""
    t = _tokens(case)
    if case["op"] == "append":
        return [_spread(case["rows"], s, case["spread"], 0.37) for s in range(case["seqs"])]
    return [max(t[s], _spread(case["rows"], s, case["spread"], 0.37)) for s in range(case["seqs"])]


def _row_bytes(kind, hd):
    return {"f32": 4 * hd, "f16": 2 * hd, "q8_0": hd + hd // 16, "q4_0": hd // 2 + hd // 16}[kind]


def work(case):
    size = 4 if case["type"] == "f32" else 2
    hd, heads, kv = case["hd"], case["heads"], case["kv"]
    t = _tokens(case)
    if case["op"] == "rotate":
        n = t[0] * (heads + kv) * hd
        return {"bytes": 2 * n * size + 4 * t[0], "flops": (9 if case["norm"] else 6) * n}
    if case["op"] == "append":
        n = sum(t)
        b = n * hd * size * (2 * heads + 2 * kv) + n * kv * (_row_bytes(case["k"], hd) + _row_bytes(case["v"], hd) + 4)
        b += n * kv * hd * size * ((case["k"] not in ("f16", "f32")) + (case["v"] not in ("f16", "f32")))  # the held values
        return {"bytes": b, "flops": n * hd * (9 * heads + 12 * kv)}
    rows, pairs, read = _rows(case), 0.0, 0.0
    for s in range(case["seqs"]):
        n, w = rows[s], case["window"]
        first = n - t[s] + 1                               # rows that the first of the new tokens sees without a window
        if w:
            # rows lie GAP positions apart on average behind the newest ones
            near = max(512, t[s]) if case["evicted"] else n
            cut = min(n, w if w <= near else near + (w - near) / GAP)
            see = min(n, cut + case["sink"])
            pairs += t[s] * min(see, (first + n) / 2)
            read += min(n, see + t[s] - 1)
        else:
            pairs += t[s] * (first + n) / 2
            read += n
    b = kv * read * (_row_bytes(case["k"], hd) + _row_bytes(case["v"], hd))
    b += sum(t) * heads * (2 * hd * size + 4) + 4 * sum(t)
    return {"bytes": int(b), "flops": int(4 * hd * heads * pairs)}


# ------------------------------------------------------------------------------------------------ inputs

GAP = 1.0 + 0.25 * 4.5       # mean distance of old rows: a quarter of them have 1 .. 8 evicted tokens before them


def _omega(case):
    """Rotation per position of each pair, and the factor on the rotated dims."""
    rot = case["hd"] - case["nonrot"]
    theta, factor, ctx = 1e6, 4.0, 32768.0
    f = np.arange(rot // 2, dtype=np.float64)
    kind = case["scaling"]
    if kind == "ntk":
        theta = theta * factor ** (rot / (rot - 2.0))
    w = theta ** (-2.0 * f / rot)
    if kind == "linear":
        return w / factor, 1.0
    if kind == "yarn":
        def dim(turns):
            return rot * math.log(ctx / (turns * 2 * math.pi)) / (2 * math.log(theta))
        lo, hi = max(math.floor(dim(32.0)), 0), min(math.ceil(dim(1.0)), rot - 1)
        ramp = np.clip((f - lo) / max(hi - lo, 0.001), 0.0, 1.0)
        return w / factor * ramp + w * (1 - ramp), 0.1 * math.log(factor) + 1.0
    if kind == "bands":
        turns = ctx * w / (2 * math.pi)                     # of the pair over the original context
        keep = np.clip((turns - 1.0) / (4.0 - 1.0), 0.0, 1.0)
        return w / factor * (1 - keep) + w * keep, 1.0
    return w, 1.0


def _normal(gen, *shape):
    return torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32)


def _hold(x, kind):
    """x [..., hd] float32 as planes of the cache: (data, scale or None)."""
    if kind in ("f32", "f16"):
        return x.to(DTYPE[kind]), None
    b = x.reshape(*x.shape[:-1], x.shape[-1] // 32, 32)
    if kind == "q8_0":
        d = b.abs().amax(-1, keepdim=True) / 127.0
        y = b / torch.where(d > 0, d, torch.ones_like(d))
        code = (torch.sign(y) * torch.floor(y.abs().double() + 0.5).float()).clamp(-127, 127)
        return code.to(torch.int8).reshape(x.shape), d.squeeze(-1).half()
    at = b.abs().argmax(-1, keepdim=True)
    d = b.gather(-1, at) / -8.0
    zero = d == 0
    y = b / torch.where(zero, torch.ones_like(d), d)
    code = torch.floor(y + 8.5).clamp(0, 15)
    code = torch.where(zero, torch.full_like(code, 8.0), code).to(torch.uint8)
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


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    hd, heads, kv, dt = case["hd"], case["heads"], case["kv"], DTYPE[case["type"]]
    t = _tokens(case)
    n = sum(t)
    st = {"case": case, "n": n, "tok0": np.concatenate([[0], np.cumsum(t)]).astype(np.int32)}
    if case["op"] != "attend":
        # the projections of n tokens, as one product leaves them: queries, keys, values side by side
        qkv = (_normal(gen, n, heads + 2 * kv, hd) * torch.exp(0.5 * _normal(gen, 1, heads + 2 * kv, hd))).to(dt)
        st["q"], st["k"], st["v"] = qkv[:, :heads], qkv[:, heads:heads + kv], qkv[:, heads + kv:]
        if case["op"] == "rotate" and not case["fused"]:
            st["q"], st["k"] = st["q"].contiguous(), st["k"].contiguous()
        st["q_norm"] = (1.0 + 0.2 * _normal(gen, hd)) if case["norm"] else None
        st["k_norm"] = (1.0 + 0.2 * _normal(gen, hd)) if case["norm"] else None
        w, st["mscale"] = _omega(case)
        st["omega"] = torch.from_numpy(w).cuda()
        st["q_out"] = torch.empty(n, heads, hd, device="cuda", dtype=dt)
    if case["op"] == "rotate":
        st["pos"] = torch.arange(case["first"], case["first"] + n, device="cuda", dtype=torch.int32)
        st["k_out"] = torch.empty(n, kv, hd, device="cuda", dtype=dt)
        st["plan"] = _plan(st) if own else None
        return st
    seqs, rows = case["seqs"], _rows(case)
    cap = max(rows) if case["op"] == "attend" else max(a + b for a, b in zip(rows, t))
    cap = cap + 37                                         # physical rows behind the live ones
    seq = torch.repeat_interleave(torch.arange(seqs, device="cuda"), torch.tensor(t, device="cuda"))
    st["seq"], st["at"] = seq, torch.arange(n, device="cuda") - torch.from_numpy(st["tok0"][:-1]).cuda().long()[seq]
    st["cap"], st["n_max"], st["t_max"] = cap, max(rows), max(t)
    st["row0"] = np.arange(seqs, dtype=np.int64) * kv * cap
    live = torch.tensor(rows, device="cuda", dtype=torch.int32)
    if case["op"] == "append":
        st["n_before"], st["n_live"] = live, live.clone()
        st["pos"] = (2 * live.long()[seq] + st["at"]).int()
        planes = {}
        for name, kind in (("k", case["k"]), ("v", case["v"])):
            width = {"f32": hd, "f16": hd, "q8_0": hd, "q4_0": hd // 2}[kind]
            kind_dt = {"f32": torch.float32, "f16": torch.float16, "q8_0": torch.int8, "q4_0": torch.uint8}[kind]
            planes[name] = torch.zeros(seqs, kv, cap, width, device="cuda", dtype=kind_dt)
            planes[name + "_scale"] = torch.zeros(seqs, kv, cap, hd // 32, device="cuda", dtype=torch.float16) if kind[0] == "q" else None
            st[name + "_held"] = torch.empty(n, kv, hd, device="cuda", dtype=dt) if kind[0] == "q" else None
        planes["pos"] = torch.zeros(seqs, kv, cap, device="cuda", dtype=torch.int32)
        st.update(planes=planes)
        st["plan"] = _plan(st) if own else None
        return st
    # the cache an eviction leaves: old rows thinned out head by head, the newest ones all there
    gap = torch.ones(seqs, kv, cap, device="cuda")
    last = live.long()[:, None, None]
    if case["evicted"]:
        near = torch.clamp(torch.tensor(t, device="cuda"), min=512)[:, None, None]
        old = torch.arange(cap, device="cuda")[None, None] < last - near
        u = torch.rand(gap.shape, generator=gen, device="cuda")
        gap = torch.where(old & (u < 0.25), 2.0 + torch.floor(u * 32.0), gap)
    pos = torch.cumsum(gap.double(), -1).long()
    pos = pos - pos.gather(-1, (last - 1).expand(seqs, kv, 1)) + (4 * last if case["evicted"] else last) - 1
    pos = torch.where(torch.arange(cap, device="cuda")[None, None] < last, pos, torch.zeros_like(pos))
    newest = (4 if case["evicted"] else 1) * live.long() - 1
    tl = torch.tensor(t, device="cuda")
    st["pos"] = (newest[seq] - tl[seq] + 1 + st["at"]).int()
    heat = torch.exp(torch.rand(1, heads, 1, generator=gen, device="cuda") * 2.0 - 0.7)   # flat heads and peaked ones
    st["q"] = (_normal(gen, n, heads, hd) * heat).to(dt)
    planes = {"pos": pos.int().contiguous()}
    for name, kind in (("k", case["k"]), ("v", case["v"])):
        x = torch.empty(seqs, kv, cap, hd, device="cuda", dtype=torch.float16 if kind != "f32" else torch.float32).normal_(generator=gen)
        planes[name], planes[name + "_scale"] = _hold(x.float(), kind) if kind != "f16" else (x, None)
        del x
    st.update(planes=planes, n_live=live, out=torch.empty(n, heads, hd, device="cuda", dtype=dt),
              lse=torch.empty(n, heads, device="cuda", dtype=torch.float32))
    st["plan"] = _plan(st) if own else None
    return st


# ------------------------------------------------------------------------------------------------ the library's calls

def _plan(st):
    """What a program over the library keeps: the rotation, the cache, the workspace."""
    import kv_cache_eviction_tria_gb300 as tria
    case = st["case"]
    plan = {"tria": tria}
    if case["op"] != "attend":
        plan["rope"] = tria.Rope(head_dim=case["hd"], nonrot_dim=case["nonrot"], theta=1e6, layout=case["layout"],
                                 scaling=case["scaling"], factor=4.0, orig_ctx=32768)
    if case["op"] != "rotate":
        p = st["planes"]
        plan["cache"] = tria.LayerCache(k=p["k"], v=p["v"], k_scale=p["k_scale"], v_scale=p["v_scale"], pos=p["pos"],
                                        n_live=st["n_live"], seq_row0=st["row0"], capacity=[st["cap"]] * case["seqs"],
                                        head_dim=case["hd"], n_kv_heads=case["kv"], k_type=case["k"], v_type=case["v"])
        size = tria.attend_workspace_size(plan["cache"], case["heads"], st["tok0"]) if case["op"] == "attend" \
            else tria.workspace_size(plan["cache"], 0)
        plan["ws"] = torch.empty(size, device="cuda", dtype=torch.uint8)
        tria.workspace_init(plan["ws"])
    return plan


def _own_run(st):
    plan, case = st["plan"], st["case"]
    tria = plan["tria"]
    if case["op"] == "rotate":
        tria.rotate(plan["rope"], [(st["q"], st["q_out"], st["q_norm"]), (st["k"], st["k_out"], st["k_norm"])], st["pos"], eps=EPS)
        return {"q": st["q_out"], "k": st["k_out"]}
    if case["op"] == "append":
        tria.append_qkv(plan["rope"], plan["cache"], st["q"], st["k"], st["v"], st["pos"], q_out=st["q_out"], tok0=st["tok0"],
                        n_before=st["n_before"], q_norm=st["q_norm"], k_norm=st["k_norm"], eps=EPS,
                        k_held=st["k_held"], v_held=st["v_held"], ws=plan["ws"])
        return _appended(st)
    tria.attend(plan["cache"], st["q"], st["out"], st["pos"], tok0=st["tok0"], lse=st["lse"], window=case["window"],
                sink=case["sink"], ws=plan["ws"])
    return {"out": st["out"], "lse": st["lse"]}


def _appended(st):
    p = st["planes"]
    out = {"q": st["q_out"], "pos": p["pos"], "n_live": st["n_live"]}
    for name in ("k", "v"):
        if st[name + "_held"] is None:
            out[name] = p[name]
        else:
            out[name], out[name + "_scale"] = st[name + "_held"], p[name + "_scale"]
    return out


# ------------------------------------------------------------------------------------------------ the plain forms

def _turned(st, x, norm):
    """x [n, h, hd] normed and rotated, float32."""
    case = st["case"]
    rot = case["hd"] - case["nonrot"]
    x = x.float()
    if norm is not None:
        x = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS) * norm
    angle = st["pos"].double()[:, None] * st["omega"]       # far positions need the 64 bits
    c, s = (torch.cos(angle) * st["mscale"]).float()[:, None], (torch.sin(angle) * st["mscale"]).float()[:, None]
    if case["layout"] == "half":
        a, b = x[..., :rot // 2], x[..., rot // 2:rot]
    else:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
    a, b = a * c - b * s, a * s + b * c
    y = torch.stack([a, b], -1).flatten(-2) if case["layout"] == "interleaved" else torch.cat([a, b], -1)
    return torch.cat([y, x[..., rot:]], -1)


def _visible(st, pos_rows, p, n_live):
    """Which rows [..., N] the tokens at positions p [..., 1] see."""
    case = st["case"]
    row = torch.arange(pos_rows.shape[-1], device="cuda")
    see = (row < n_live) & (pos_rows <= p)
    if case["window"]:
        see = see & ((p - pos_rows < case["window"]) | (row < case["sink"]))
    return see


def run(state):
    if own:
        return _own_run(state)
    st, case = state, state["case"]
    dt = DTYPE[case["type"]]
    if case["op"] == "rotate":
        st["q_out"].copy_(_turned(st, st["q"], st["q_norm"]))
        st["k_out"].copy_(_turned(st, st["k"], st["k_norm"]))
        return {"q": st["q_out"], "k": st["k_out"]}
    hd, heads, kv, seqs = case["hd"], case["heads"], case["kv"], case["seqs"]
    p = st["planes"]
    if case["op"] == "append":
        st["q_out"].copy_(_turned(st, st["q"], st["q_norm"]))
        row = st["n_before"].long()[st["seq"]] + st["at"]
        for name, kind, x in (("k", case["k"], _turned(st, st["k"], st["k_norm"])), ("v", case["v"], st["v"].float())):
            data, scale = _hold(x, kind)
            p[name][st["seq"], :, row] = data
            if scale is not None:
                p[name + "_scale"][st["seq"], :, row] = scale
                st[name + "_held"].copy_(_values(data, scale, kind))
        p["pos"][st["seq"], :, row] = st["pos"][:, None].expand(st["n"], kv)
        st["n_live"].copy_(st["n_before"] + torch.bincount(st["seq"], minlength=seqs))
        return _appended(st)
    n, tm, group = st["n_max"], st["t_max"], heads // kv
    q = torch.zeros(seqs, tm, heads, hd, device="cuda", dtype=torch.float32)
    q[st["seq"], st["at"]] = st["q"].float()
    q = q.reshape(seqs, tm, kv, group, hd).permute(0, 2, 1, 3, 4).reshape(seqs, kv, tm * group, hd)
    pq = torch.full((seqs, tm), -1, device="cuda", dtype=torch.int32)
    pq[st["seq"], st["at"]] = st["pos"]
    scales = [None if p[x] is None else p[x][:, :, :n] for x in ("k_scale", "v_scale")]
    logit = q @ _values(p["k"][:, :, :n], scales[0], case["k"]).transpose(-1, -2)
    logit = (logit * hd ** -0.5).reshape(seqs, kv, tm, group, n)
    see = _visible(st, p["pos"][:, :, None, :n], pq[:, None, :, None], st["n_live"][:, None, None, None])
    logit = logit.masked_fill(~see[:, :, :, None], -math.inf)
    top = logit.amax(-1, keepdim=True)
    e = torch.exp(logit - top.masked_fill(top == -math.inf, 0.0))
    total = e.sum(-1, keepdim=True)
    out = (e.reshape(seqs, kv, tm * group, n) @ _values(p["v"][:, :, :n], scales[1], case["v"])).reshape(seqs, kv, tm, group, hd)
    out = out / torch.where(total > 0, total, torch.ones_like(total))
    lse = (top + torch.log(total)).squeeze(-1)
    st["out"].copy_(out.permute(0, 2, 1, 3, 4).reshape(seqs, tm, heads, hd)[st["seq"], st["at"]].to(dt))
    st["lse"].copy_(lse.permute(0, 2, 1, 3).reshape(seqs, tm, heads)[st["seq"], st["at"]])
    return {"out": st["out"], "lse": st["lse"]}


# ------------------------------------------------------------------------------------------------ in 64 bits

def exact(case, seed):
    st = prepare(case, seed)
    hd, heads, kv = case["hd"], case["heads"], case["kv"]
    f64 = torch.float64

    def held(data, scale, kind):
        if kind[0] == "f":
            return data.to(f64)
        s = scale.to(f64).repeat_interleave(32, -1)
        if kind == "q8_0":
            return data.to(f64) * s
        b = data.reshape(*scale.shape, 16).to(torch.int64)
        return (torch.cat([b % 16, b // 16], -1).reshape(*scale.shape[:-1], hd).to(f64) - 8) * s

    if case["op"] != "attend":
        rot = hd - case["nonrot"]
        z = torch.polar(torch.full_like(st["omega"], st["mscale"])[None], st["pos"].to(f64)[:, None] * st["omega"][None])[:, None]

        def turned(x, w):
            x = x.to(f64)
            if w is not None:
                x = x / torch.sqrt((x * x).sum(-1, keepdim=True) / hd + EPS) * w.to(f64)
            if case["layout"] == "half":
                c = torch.complex(x[..., :rot // 2], x[..., rot // 2:rot]) * z
                y = torch.cat([c.real, c.imag], -1)
            else:
                c = torch.view_as_complex(x[..., :rot].reshape(*x.shape[:-1], rot // 2, 2).contiguous()) * z
                y = torch.view_as_real(c).reshape(*x.shape[:-1], rot) if case["layout"] == "interleaved" else torch.cat([c.real, c.imag], -1)
            return torch.cat([y, x[..., rot:]], -1)

        q, k = turned(st["q"], st["q_norm"]), turned(st["k"], st["k_norm"])
        if case["op"] == "rotate":
            return {"q": q, "k": k}
        out = {"q": q, "pos": None, "n_live": None}
        rows = st["n_before"].long()[st["seq"]] + st["at"]
        for name, kind, x in (("k", case["k"], k), ("v", case["v"], st["v"].to(f64))):
            if kind[0] == "f":
                plane = torch.zeros(st["planes"][name].shape, device="cuda", dtype=f64)
                plane[st["seq"], :, rows] = x
                out[name] = plane
                continue
            b = x.reshape(st["n"], kv, hd // 32, 32)
            if kind == "q8_0":
                d = b.abs().amax(-1) / 127
                code = b / torch.where(d == 0, 1.0, d)[..., None]
                code = torch.sign(code) * torch.floor(code.abs() + 0.5)
            else:
                big, small = b.amax(-1), b.amin(-1)
                # the value of the largest modulus; of two equal ones the first
                first = b.gather(-1, b.abs().argmax(-1, keepdim=True)).squeeze(-1)
                d = torch.where(big == -small, first, torch.where(big > -small, big, small)) / -8
                code = torch.clamp(torch.floor(b / torch.where(d == 0, 1.0, d)[..., None] + 8.5), 0, 15) - 8
                code = torch.where((d == 0)[..., None], 0.0, code)
            stored = d.half().to(f64)
            scale = torch.zeros(st["planes"][name + "_scale"].shape, device="cuda", dtype=f64)
            scale[st["seq"], :, rows] = d
            out[name], out[name + "_scale"] = (code * stored[..., None]).reshape(st["n"], kv, hd), scale
        return out
    out = torch.zeros(st["n"], heads, hd, device="cuda", dtype=f64)
    lse = torch.full((st["n"], heads), -math.inf, device="cuda", dtype=f64)
    p, group = st["planes"], heads // kv
    live, tok0 = st["n_live"].tolist(), st["tok0"].tolist()
    for s in range(case["seqs"]):
        n, a, b = live[s], tok0[s], tok0[s + 1]
        for g in range(kv):
            k = held(p["k"][s, g, :n], None if p["k_scale"] is None else p["k_scale"][s, g, :n], case["k"])
            v = held(p["v"][s, g, :n], None if p["v_scale"] is None else p["v_scale"][s, g, :n], case["v"])
            where = p["pos"][s, g, :n].long()[None]
            at = st["pos"][a:b].long()[:, None]
            hidden = where > at
            if case["window"]:
                old = at - where >= case["window"]
                old[:, :case["sink"]] = False
                hidden = hidden | old
            x = torch.einsum("thd,nd->thn", st["q"][a:b, g * group:(g + 1) * group].to(f64), k) / math.sqrt(hd)
            x[hidden[:, None].expand_as(x)] = -math.inf
            total = torch.logsumexp(x, -1)
            lse[a:b, g * group:(g + 1) * group] = total
            w = torch.exp(x - torch.where(total == -math.inf, 0.0, total)[..., None])
            out[a:b, g * group:(g + 1) * group] = torch.einsum("thn,nd->thd", w, v)
    return {"out": out, "lse": lse}
