"""One workspace for all calls of a beam search, one after the other: every
result has the bits that it has when each call gets a workspace of its own. There are more
segments (sequences x KV heads) than groups may hold beams, and their rows
reach across CTAs, so that the calls' counters and parts lie side by side."""
import numpy as np
import pytest

import _prefix as P
import _rows as R

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")


class Search:
    """Beams over shared prompts: append, attention over both caches and over the own rows, choice, reorder."""

    def __init__(self, lib, cfg, steps):
        self.lib, self.cfg = lib, cfg
        rng = np.random.default_rng(cfg["beams"])
        self.groups, self.n_kv, self.hd, self.kind = len(cfg["shared"]), cfg["n_kv"], cfg["hd"], cfg["kind"]
        self.n = n = self.groups * cfg["beams"]
        self.nq = self.n_kv * cfg["group"]
        self.seq0 = [cfg["beams"] * g for g in range(self.groups + 1)]
        rows = [int(x) for x in rng.integers(cfg["least"], cfg["least"] + 60, n)]
        self.p, self.c = P.pair(lib, rng, shared=cfg["shared"], rows=rows, n_kv=self.n_kv, hd=self.hd, types=cfg["prefix"],
                                own_types=cfg["own"], gaps=False, own_spare=steps + 70)
        newest = P.follow(self.p, self.c, self.seq0)
        self.rope = lib.Rope(head_dim=self.hd, theta=1e4)
        qm = rng.standard_normal((1, self.nq, self.hd // 2, 2)).astype(np.float32)
        self.stats = lib.Stats(qm, np.hypot(qm[..., 0], qm[..., 1]), n_kv_heads=self.n_kv, head_dim=self.hd, rope_theta=1e4)
        self.heads = self.nq + 2 * self.n_kv
        self.joint = [R.act(rng.standard_normal((n, self.heads, self.hd)), self.kind) for _ in range(steps)]
        self.logits = [R.act(3 * rng.standard_normal((n, cfg["vocab"])), "bf16") for _ in range(steps)]
        self.pos = torch.tensor(np.asarray(newest) + 1, device="cuda", dtype=torch.int32)
        self.total = torch.zeros(n, device="cuda")
        self.parent = torch.zeros(self.groups, cfg["beams"], device="cuda", dtype=torch.int32)
        self.token = torch.zeros_like(self.parent)
        one = np.arange(n + 1, dtype=np.int32)
        self.sizes = dict(pass_=lib.workspace_size(self.c.cache, cfg["group"]), attend=lib.attend_workspace_size(self.c.cache, self.nq, one),
                          prefix=lib.attend_prefix_workspace_size(self.p.cache, self.c.cache, self.nq, 1, self.seq0),
                          select=lib.beam_select_workspace_size(self.seq0, cfg["vocab"], cfg["beams"]),
                          reorder=lib.reorder_workspace_size([self.c.cache], self.seq0))

    def run(self, steps, ws_of, evict=()):
        """The results of the steps; ws_of(size) gives a call's workspace."""
        lib, c, cfg, out = self.lib, self.c, self.cfg, []
        for i in steps:
            used = [ws_of(self.sizes[k]) for k in ("pass_", "prefix", "attend", "select", "reorder", "pass_")]
            q, o = (torch.full((self.n, self.nq, self.hd), 7.0, device="cuda", dtype=self.joint[i].dtype) for _ in range(2))
            own, lse, own_lse = torch.full_like(o, 7.0), *(torch.full((self.n, self.nq), 7.0, device="cuda") for _ in range(2))
            j, nq, n_kv = self.joint[i], self.nq, self.n_kv
            lib.append_qkv(self.rope, c.cache, j[:, :nq], j[:, nq:nq + n_kv], j[:, nq + n_kv:], self.pos, q_out=q, ws=used[0])
            lib.attend_prefix(self.p.cache, c.cache, q, o, self.pos, seq0=self.seq0, lse=lse, ws=used[1])
            lib.attend(c.cache, q, own, self.pos, lse=own_lse, ws=used[2])
            lib.beam_select(self.logits[i], self.total, self.total, self.parent, self.token, seq0=self.seq0, in_place=True, ws=used[3])
            lib.reorder([c.cache], self.parent, seq0=self.seq0, ws=used[4])
            out += [o, own, lse, own_lse, self.total.clone(), self.parent.clone(), self.token.clone(), c.d["n_live"].clone()]
            self.pos += 1
            if i in evict:
                lib.evict(self.stats, 0, c.cache, lib.Policy(budget_rows=[cfg["least"] // 2] * self.n, window=4, cur_pos=self.pos.tolist()), ws=used[5])
                out.append(c.d["n_live"].clone())
            for w in used:
                assert lib.device_status(w) == lib.OK
        return out + [t.clone() for t in c.d.values() if t is not None]


def once_and_again(lib, cfg, steps, evict=()):
    x = Search(lib, cfg, steps)
    shared = x.c.ws(max(x.sizes.values()))
    got = x.run(range(steps), lambda size: shared, evict)
    y = Search(lib, cfg, steps)
    same(got, y.run(range(steps), y.c.ws, evict))


def same(got, want):
    bits = lambda t: t.contiguous().view(torch.uint8)
    bad = [i for i, (a, b) in enumerate(zip(got, want)) if not torch.equal(bits(a), bits(b))]
    assert not bad, f"results {bad} of {len(want)} differ from those with a workspace for each call"


LOOPS = [dict(kind="f16", prefix=("f16", "f16"), own=("f16", "f16"), n_kv=8, group=2, hd=64, shared=[300], beams=32, vocab=40000, least=20),
         dict(kind="bf16", prefix=("q8_0", "q8_0"), own=("q8_0", "q8_0"), n_kv=8, group=4, hd=128, shared=[300, 77], beams=24, vocab=9001, least=30),
         dict(kind="f16", prefix=("q4_0", "q4_0"), own=("q4_0", "q8_0"), n_kv=8, group=2, hd=64, shared=[700, 9], beams=24, vocab=33000, least=40),
         dict(kind="f32", prefix=("f16", "f16"), own=("f16", "f16"), n_kv=8, group=2, hd=64, shared=[300], beams=32, vocab=9001, least=1200),
         dict(kind="f32", prefix=("q8_0", "f32"), own=("q8_0", "f32"), n_kv=8, group=1, hd=64, shared=[90, 300], beams=24, vocab=9001, least=1100)]


@pytest.mark.parametrize("cfg", LOOPS)
def test_attention_choice_and_reorder(lib, cfg):
    once_and_again(lib, cfg, 4)


@pytest.mark.parametrize("cfg", LOOPS)
def test_with_passes(lib, cfg):
    """The own rows are evicted twice in between: 256 and 384 segments of fp16 or 8-bit keys take the fused pass."""
    x = Search(lib, cfg, 1)
    assert lib.evict_model_fused(x.stats, [0], [x.c.cache]) == (cfg["own"][0] != "q4_0")
    once_and_again(lib, cfg, 4, evict=(1, 2))


def test_searches_of_different_shapes_in_turn(lib):
    """Steps of all of them on one workspace, in a random order."""
    rng = np.random.default_rng(3)
    searches = [Search(lib, cfg, 4) for cfg in LOOPS]
    shared = searches[0].c.ws(max(max(x.sizes.values()) for x in searches))
    turns = rng.permutation(np.repeat(np.arange(len(LOOPS)), 4))
    got, at = [[] for _ in LOOPS], [0] * len(LOOPS)
    for k in turns:
        got[k] += searches[k].run([at[k]], lambda size: shared, evict=(1, 2))
        at[k] += 1
    for cfg, g in zip(LOOPS, got):
        y = Search(lib, cfg, 4)
        same(g, [t for i in range(4) for t in y.run([i], y.c.ws, evict=(1, 2))])


TAG, SCRATCH = 0x9E3779B1, 256 + 4 * 4 * 2048       # the first pass's flags; the words that are zero between calls end here


@pytest.mark.parametrize("rows,n_kv,seqs,k,v", [(300001, 1, 1, "f16", "f16"), (270000, 2, 1, "q8_0", "q4_0"), (40001, 4, 4, "q4_0", "f16"),
                                                (9000, 8, 8, "f16", "q8_0"), (3000, 8, 16, "q8_0", "q8_0")])
def test_a_pass_relies_on_nothing_in_its_scratch(lib, rows, n_kv, seqs, k, v):
    """Flags that look set, counters and histograms that are not zero: cooperative, cluster and fused selections, moves of
    many rounds, and a keep list of the caller's."""
    rng = np.random.default_rng(rows)
    live = [rows - 37 * s for s in range(seqs)]
    hd, group = 64, 2
    qm = rng.standard_normal((1, n_kv * group, hd // 2, 2)).astype(np.float32)
    stats = lib.Stats(qm, np.hypot(qm[..., 0], qm[..., 1]), n_kv_heads=n_kv, head_dim=hd, rope_theta=1e4)
    c = R.Cache(lib, rng, rows=live, cap=[rows] * seqs, n_kv=n_kv, hd=hd, k_type=k, v_type=v)
    first = {name: None if t is None else t.clone() for name, t in c.d.items()}
    size = lib.workspace_size(c.cache, group)
    half = [n // 2 for n in live]
    policies = [lib.Policy(budget_rows=[int(f * n) for n in live], window=16, sink=4, cur_pos=[6 * rows] * seqs) for f in (0.7, 0.3)]
    keep = torch.zeros(c.row0[-1] + n_kv * rows + 3, device="cuda", dtype=torch.int32)
    for s in range(seqs):
        for g in range(n_kv):
            at = c.row0[s] + g * rows
            keep[at:at + half[s]] = torch.from_numpy(np.sort(rng.choice(live[s], half[s], replace=False)).astype(np.int32))
    ends = []
    for fill in (0, TAG, 1):
        out = []
        for call in ("evict", "evict_staged", "compact"):
            for name, t in first.items():
                if t is not None:
                    c.d[name].copy_(t)
            ws = c.ws(size)
            words = ws.view(torch.int32)[SCRATCH // 4:]
            for i, policy in enumerate(policies):                 # the second one's flags carry the second tag
                tag = (i + 1) * fill % 2 ** 32
                words.fill_(tag - 2 ** 32 if tag >= 2 ** 31 else tag)
                if call != "compact":
                    getattr(lib, call)(stats, 0, c.cache, policy, ws=ws)
                elif i == 0:
                    lib.compact(c.cache, lib.Policy(budget_rows=half), keep, ws=ws)
                assert lib.device_status(ws) == lib.OK
                out += [t.clone() for t in c.d.values() if t is not None]
        ends.append(out)
    for other in ends[1:]:
        assert all(torch.equal(a.contiguous().view(torch.uint8), b.contiguous().view(torch.uint8)) for a, b in zip(ends[0], other))
    stats.close()
