"""Beam search as a decode loop runs it: new tokens appended to the beams' own
rows, attention over the shared prompts and those rows, the choice of the next
beams, and every layer's rows behind their parents, with a pass over the own
rows in between. Every step is checked in 64 bits over what stands on the
device; the same loop, captured and replayed, gives the same bits."""
import numpy as np
import pytest

import _prefix as P
import _rows as R
from oracle import beam_oracle as B
from test_gpu_beams import check as check_choice
from test_gpu_reorder import state

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

LOOPS = [dict(k="f16", v="f16", kind="f16", n_kv=2, group=4, hd=128, shared=[300, 77], beams=4, vocab=613, window=0, sink=0),
         dict(k="q8_0", v="q4_0", kind="bf16", n_kv=1, group=8, hd=64, shared=[130, 0, 64], beams=6, vocab=1001, window=90, sink=3),
         dict(k="q4_0", v="q4_0", kind="f16", n_kv=2, group=2, hd=128, shared=[500], beams=32, vocab=97, window=0, sink=0),
         dict(k="f32", v="f32", kind="f32", n_kv=1, group=4, hd=64, shared=[40, 90], beams=2, vocab=50, window=0, sink=0)]


class Loop:
    def __init__(self, lib, cfg, steps, layers=2):
        rng = np.random.default_rng(cfg["hd"] + cfg["beams"])
        self.lib, self.cfg = lib, cfg
        n_kv, hd, kind, beams = cfg["n_kv"], cfg["hd"], cfg["kind"], cfg["beams"]
        self.nq, self.groups = n_kv * cfg["group"], len(cfg["shared"])
        self.n = n = self.groups * beams
        self.seq0 = [beams * g for g in range(self.groups + 1)]
        types = (cfg["k"], cfg["v"])
        self.pairs = [P.pair(lib, rng, shared=cfg["shared"], rows=[0] * n, n_kv=n_kv, hd=hd, types=types, spare=steps + 3, gaps=False)
                      for _ in range(layers)]
        self.own = [c.cache for _, c in self.pairs]
        self.rope = lib.Rope(head_dim=hd, theta=1e4)
        heads = self.nq + 2 * n_kv
        self.table = [R.act(rng.standard_normal((cfg["vocab"], heads, hd)), kind) for _ in range(layers)]
        self.joint = torch.zeros(n, heads, hd, device="cuda", dtype=self.table[0].dtype)
        self.to_logits = torch.from_numpy((rng.standard_normal((self.nq * hd, cfg["vocab"])) * 0.3).astype(np.float32)).cuda()
        self.q = [torch.zeros(n, self.nq, hd, device="cuda", dtype=self.joint.dtype) for _ in range(layers)]
        self.out = [torch.zeros_like(self.q[0]) for _ in range(layers)]
        self.lse = [torch.zeros(n, self.nq, device="cuda") for _ in range(layers)]
        self.tok = torch.from_numpy(rng.integers(0, cfg["vocab"], n)).cuda()
        self.pos = torch.from_numpy(np.repeat(cfg["shared"], beams).astype(np.int32)).cuda()
        self.logits = torch.zeros(n, cfg["vocab"], device="cuda")
        self.total = torch.zeros(n, device="cuda")
        self.before = torch.zeros(n, device="cuda")
        self.over, self.over_before = torch.zeros(n, device="cuda", dtype=torch.int32), torch.zeros(n, device="cuda", dtype=torch.int32)
        self.parent = torch.zeros(self.groups, beams, device="cuda", dtype=torch.int32)
        self.token = torch.zeros_like(self.parent)
        p, c = self.pairs[0]
        self.ws = c.ws(max(lib.workspace_size(c.cache, cfg["group"]),
                           lib.attend_prefix_workspace_size(p.cache, c.cache, self.nq, 1, self.seq0),
                           lib.beam_select_workspace_size(self.seq0, cfg["vocab"], beams),
                           lib.reorder_workspace_size(self.own, self.seq0)))

    def attend(self):
        self.before.copy_(self.total)
        self.over_before.copy_(self.over)
        for l, (p, c) in enumerate(self.pairs):
            self.joint.copy_(self.table[l][self.tok])
            if l:
                self.joint[:, :self.nq] += self.out[l - 1]
            j, n_kv = self.joint, c.n_kv
            self.lib.append_qkv(self.rope, c.cache, j[:, :self.nq], j[:, self.nq:self.nq + n_kv], j[:, self.nq + n_kv:], self.pos,
                                q_out=self.q[l], ws=self.ws)
            self.lib.attend_prefix(p.cache, c.cache, self.q[l], self.out[l], self.pos, seq0=self.seq0, lse=self.lse[l],
                                   window=self.cfg["window"], sink=self.cfg["sink"], ws=self.ws)
        torch.mm(self.out[-1].flatten(1).float(), self.to_logits, out=self.logits)

    def choose(self):
        self.lib.beam_select(self.logits, self.total, self.total, self.parent, self.token, seq0=self.seq0, ended=self.over,
                             ended_out=self.over, end_token=0, in_place=True, ws=self.ws)
        self.lib.reorder(self.own, self.parent, seq0=self.seq0, ws=self.ws)
        self.tok.copy_(self.token.flatten())
        self.pos += 1

    def check_attend(self):
        cfg = self.cfg
        tok0, pos = np.arange(self.n + 1), self.pos.cpu().numpy()
        for l, (p, c) in enumerate(self.pairs):
            c.h = {k: None if t is None else t.cpu().numpy() for k, t in c.d.items()}
            c.rows = c.d["n_live"].tolist()
            want = P.expected(p, c, self.seq0, R.host(self.q[l]), pos, tok0, self.nq, cfg["window"], cfg["sink"])
            P.check(R.host(self.out[l]), R.host(self.lse[l]), want, cfg["kind"], cfg["kind"] != "f32", max(p.rows) + max(c.rows), c.hd,
                    q_exact=cfg["kind"] == "f16", k_exact=cfg["k"] == "f16")

    def check_choice(self, planes):
        got = dict(total_out=self.total.view_as(self.parent).cpu().numpy(), parent=self.parent.cpu().numpy(), token=self.token.cpu().numpy(),
                   ended_out=self.over.view_as(self.parent).cpu().numpy())
        check_choice(got, self.logits, self.before.cpu().numpy(), self.seq0, self.cfg["beams"], self.over_before.cpu().numpy(), 0, True)
        for (_, c), (before, live) in zip(self.pairs, planes):
            want, n = B.reorder(before, live, got["parent"].flatten(), c.row0, c.cap, c.n_kv)
            now, n_now = state(c)
            assert np.array_equal(n, n_now) and all(np.array_equal(now[k], want[k]) for k in want)


@pytest.mark.parametrize("cfg", LOOPS)
def test_beam_loop(lib, cfg):
    steps, due, ends = 30, 17, []
    nq, hd = cfg["n_kv"] * cfg["group"], cfg["hd"]
    rng = np.random.default_rng(5)
    qm = rng.standard_normal((2, nq, hd // 2, 2)).astype(np.float32)
    stats = lib.Stats(qm, np.hypot(qm[..., 0], qm[..., 1]), n_kv_heads=cfg["n_kv"], head_dim=hd, rope_theta=1e4)
    for captured in (False, True):
        x = Loop(lib, cfg, steps)
        history = [[] for _ in range(x.n)]                    # each beam's appended tokens
        graph = None
        for i in range(steps):
            fed = x.tok.tolist()
            if not captured:
                x.attend()
                planes = [state(c) for _, c in x.pairs]
                if i % 7 == 0 or i > steps - 3:
                    x.check_attend()
                x.choose()
                x.check_choice(planes)
            else:
                if i == 1:                                    # (the first step ran outside the capture)
                    graph = torch.cuda.CUDAGraph()
                    with torch.cuda.graph(graph):
                        x.attend()
                        x.choose()
                if graph is None:
                    x.attend()
                    x.choose()
                else:
                    graph.replay()
            assert lib.device_status(x.ws) == lib.OK
            old = [h + [t] for h, t in zip(history, fed)]
            history = [list(old[s]) for s in x.parent.flatten().tolist()]
            if i == due - 1:                                  # values are the history's tokens', wherever their rows went
                c = x.pairs[0][1]
                if cfg["v"] in ("f16", "f32") and cfg["kind"] == cfg["v"]:
                    for s in range(x.n):
                        for g in range(c.n_kv):
                            r0 = c.row0[s] + g * c.cap[s]
                            assert torch.equal(c.d["v"][r0:r0 + due], x.table[0][torch.tensor(history[s], device="cuda"), nq + c.n_kv + g])
                pol = lib.Policy(budget_rows=[9] * x.n, window=3, cur_pos=x.pos.tolist())
                for l, own in enumerate(x.own):
                    lib.evict(stats, l, own, pol, ws=x.ws)
                assert lib.device_status(x.ws) == lib.OK and x.pairs[1][1].d["n_live"].tolist() == [9] * x.n
        ends.append((history, x.tok.tolist(), x.total.clone(), x.over.tolist(), x.out[1].clone()))
        x.rope.close()
    (h0, t0, v0, e0, o0), (h1, t1, v1, e1, o1) = ends
    assert h0 == h1 and t0 == t1 and e0 == e1 and torch.equal(v0, v1) and torch.equal(o0, o1)
    stats.close()
