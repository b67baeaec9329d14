"""Rotation, append, attention and the pass as a decode loop runs them: ragged
prompts, then steps, with a pass whenever the schedule says so. Every step's
attention is checked in 64 bits over the cache as it stands on the device, and
every appended row against the projections that made it."""
import numpy as np
import pytest

import _rows as R
from oracle import attend_oracle as A

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

LOOPS = [dict(k="f16", v="f16", kind="f16", n_kv=2, group=4, hd=128, scaling={}, layout="half", window=0, sink=0),
         dict(k="q8_0", v="q4_0", kind="bf16", n_kv=1, group=8, hd=64, layout="interleaved_to_half", window=40, sink=4,
              scaling=dict(scaling="yarn", factor=4.0, orig_ctx=64)),
         dict(k="q4_0", v="q4_0", kind="f16", n_kv=2, group=2, hd=128, layout="half", window=0, sink=0,
              scaling=dict(scaling="bands", factor=2.0, orig_ctx=128)),
         dict(k="f32", v="f32", kind="f32", n_kv=1, group=4, hd=64, scaling={}, layout="half", window=25, sink=2)]


@pytest.mark.parametrize("cfg", LOOPS)
@pytest.mark.parametrize("captured", [False, True])
def test_decode_loop(lib, cfg, captured):
    n_kv, group, hd, kind = cfg["n_kv"], cfg["group"], cfg["hd"], cfg["kind"]
    nq, prompts, cap, steps = n_kv * group, [37, 5, 20], [120, 100, 90], 70
    seqs = len(prompts)
    rng = np.random.default_rng(hd)
    c = R.Cache(lib, rng, rows=[0] * seqs, cap=cap, n_kv=n_kv, hd=hd, k_type=cfg["k"], v_type=cfg["v"])
    rope = lib.Rope(head_dim=hd, theta=1e4, layout=cfg["layout"], **cfg["scaling"])
    omega, _ = lib.rope_frequencies(head_dim=hd, theta=1e4, layout=cfg["layout"], **cfg["scaling"])
    qm = rng.standard_normal((1, nq, hd // 2, 2)).astype(np.float32)
    stats = lib.Stats(qm, np.hypot(qm[..., 0], qm[..., 1]), n_kv_heads=n_kv, head_dim=hd, omega=omega)
    sch = lib.Schedule(kv_budget=48, divide_length=16, window=8, sink=0)
    state = lib.Sequences(sch, cap)
    ws = c.ws(lib.workspace_size(c.cache, group))
    norms = [torch.from_numpy((1 + 0.2 * rng.standard_normal(hd)).astype(np.float32)).cuda() for _ in range(2)]
    tensor = kind != "f32"

    class Call:
        """The projections of some tokens and the two calls on them."""

        def __init__(self, tokens):
            self.tok0 = np.concatenate([[0], np.cumsum(tokens)]).astype(np.int32)
            n = int(self.tok0[-1])
            self.joint = R.act(np.zeros((n, nq + 2 * n_kv, hd)), kind)
            self.pos = torch.zeros(n, device="cuda", dtype=torch.int32)
            self.q, self.out = torch.zeros(n, nq, hd, device="cuda", dtype=self.joint.dtype), None
            self.out, self.lse = torch.zeros_like(self.q), torch.zeros(n, nq, device="cuda")
            self.held = [torch.zeros(n, n_kv, hd, device="cuda", dtype=self.joint.dtype) for _ in range(2)]
            self.aws = c.ws(lib.attend_workspace_size(c.cache, nq, self.tok0))

        def run(self):
            j = self.joint
            lib.append_qkv(rope, c.cache, j[:, :nq], j[:, nq:nq + n_kv], j[:, nq + n_kv:], self.pos, q_out=self.q,
                           tok0=self.tok0, q_norm=norms[0], k_norm=norms[1], k_held=self.held[0], v_held=self.held[1], ws=ws)
            lib.attend(c.cache, self.q, self.out, self.pos, tok0=self.tok0, lse=self.lse, window=cfg["window"],
                       sink=cfg["sink"], ws=self.aws)

        def check(self):
            assert lib.device_status(ws) == lib.OK and lib.device_status(self.aws) == lib.OK
            c.h = {k: None if t is None else t.cpu().numpy() for k, t in c.d.items()}
            c.rows = c.d["n_live"].tolist()
            pos = self.pos.cpu().numpy()
            for s in range(seqs):                              # the newest rows are the projections'
                t = int(self.tok0[s + 1] - self.tok0[s])
                for g in range(n_kv):
                    for name, held in (("k", self.held[0]), ("v", self.held[1])):
                        want = c.values(name, s, g)[c.rows[s] - t:]
                        got = R.host(held)[self.tok0[s]:self.tok0[s + 1], g]
                        assert np.all(np.abs(got - want) <= R.HALF_STEP[kind] * np.abs(want) + 2.0 ** -25)
                    assert np.array_equal(c.seg("pos", s, g)[c.rows[s] - t:], pos[self.tok0[s]:self.tok0[s + 1]])
            want = R.attend_expected(c, R.host(self.q), pos, self.tok0, nq, cfg["window"], cfg["sink"])
            R.check_attend(R.host(self.out), R.host(self.lse), want, kind, tensor, max(c.rows), hd,
                           q_exact=kind == "f16", k_exact=cfg["k"] == "f16")

    prompt = Call(prompts)
    prompt.joint.copy_(R.act(rng.standard_normal(tuple(prompt.joint.shape)), kind))
    prompt.pos.copy_(torch.from_numpy(np.concatenate([np.arange(p) for p in prompts]).astype(np.int32)))
    prompt.run()
    prompt.check()
    for s, p in enumerate(prompts):
        state.prefill(s, p)
    step = Call([1] * seqs)
    graph = None
    passes = 0
    for i in range(steps):
        step.joint.copy_(R.act(rng.standard_normal(tuple(step.joint.shape)), kind))
        step.pos.copy_(torch.tensor([p + i for p in prompts], dtype=torch.int32))
        if captured and i == 1:                                # (the first step ran outside the capture)
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                step.run()
        if graph is not None:
            graph.replay()
        else:
            step.run()
        if i % 9 == 0 or i > steps - 3:
            step.check()
        due = [state.decode(s) for s in range(seqs)]
        if any(due):
            pol, n_due = state.policy()
            lib.evict(stats, 0, c.cache, pol, ws=ws)
            assert lib.device_status(ws) == lib.OK and n_due == sum(due)
            state.passed()
            passes += 1
            assert c.d["n_live"].tolist() == [state.state(s)["rows"] for s in range(seqs)]
    assert passes >= 3
    stats.close()
    rope.close()


def test_a_step_taken_again_over_rejected_tokens(lib):
    """n_before rewinds: drafts are attended together, the rejected ones written over."""
    rng = np.random.default_rng(1)
    c = R.Cache(lib, rng, rows=[50, 30], cap=[60, 40], n_kv=2, hd=64, k_type="f16", v_type="q8_0", gaps=False)
    rope = lib.Rope(head_dim=64, theta=1e4)
    ws = c.ws(lib.workspace_size(c.cache, 0))

    def draft(tokens, before, seed):
        n = sum(tokens)
        tok0 = np.concatenate([[0], np.cumsum(tokens)]).astype(np.int32)
        j = R.act(np.random.default_rng(seed).standard_normal((n, 8 + 4, 64)), "bf16")
        pos = torch.tensor([b + i for b, t in zip(before, tokens) for i in range(t)], device="cuda", dtype=torch.int32)
        q = torch.zeros(n, 8, 64, device="cuda", dtype=torch.bfloat16)
        lib.append_qkv(rope, c.cache, j[:, :8], j[:, 8:10], j[:, 10:], pos, q_out=q, tok0=tok0,
                       n_before=torch.tensor(before, device="cuda", dtype=torch.int32), ws=ws)
        out = torch.zeros_like(q)
        lib.attend(c.cache, q, out, pos, tok0=tok0, ws=c.ws(lib.attend_workspace_size(c.cache, 8, tok0)))
        return out

    draft([4, 3], [50, 30], 5)
    again = draft([2, 1], [52, 31], 6)                      # two and one of the drafts were kept
    assert c.d["n_live"].tolist() == [54, 32]
    d = R.Cache(lib, np.random.default_rng(1), rows=[50, 30], cap=[60, 40], n_kv=2, hd=64, k_type="f16", v_type="q8_0", gaps=False)
    c, keep = d, c
    draft([4, 3], [50, 30], 5)
    c.d["n_live"].copy_(torch.tensor([52, 31], dtype=torch.int32))
    straight = draft([2, 1], [52, 31], 6)
    assert torch.equal(again, straight) and torch.equal(keep.d["pos"], c.d["pos"])
