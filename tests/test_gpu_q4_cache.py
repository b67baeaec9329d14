"""Caches held in 4 bits through the pass: scores against the 64-bit oracle on
the values that the codes stand for, keep-sets of both evict paths, compacted
planes as exact gathers, and where q4_0 keys are dispatched."""
import numpy as np
import pytest

import _util as U
from oracle import attend_oracle as A
from oracle import tria_oracle as O

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")


def build(n_kv, group, hd, k_type, v_type, n_live, cap, seed=0, nonrot=0):
    rng = np.random.default_rng(seed)
    row0 = np.cumsum([0] + [n_kv * c for c in cap[:-1]]).astype(np.int64)
    rows = int(sum(n_kv * c for c in cap))
    host = {"n_live": np.asarray(n_live, np.int32), "pos": (np.arange(rows) * 3 + 1).astype(np.int32)}
    for name, kind in (("k", k_type), ("v", v_type)):
        scale = np.where(rng.random(hd // 2) < 0.1, 8.0, 1.0)
        x = (rng.standard_normal((rows, hd)) * np.concatenate([scale, scale])).astype(np.float32)
        host[name], host[name + "_scale"] = A.hold(x, kind)
    nq, fc = n_kv * group, (hd - nonrot) // 2
    qm = rng.standard_normal((1, nq, fc, 2)).astype(np.float32)
    qa = (np.hypot(qm[..., 0], qm[..., 1]) + 0.5 * np.abs(rng.standard_normal((1, nq, fc)))).astype(np.float32)
    qn = rng.standard_normal((1, nq, nonrot)).astype(np.float32) if nonrot else None
    return host, row0, qm, qa, qn


def device(lib, host, row0, cap, n_kv, hd, k_type, v_type):
    dev = U.to_device(host)
    return dev, lib.LayerCache(k=dev["k"], v=dev["v"], k_scale=dev["k_scale"], v_scale=dev["v_scale"], pos=dev["pos"],
                               n_live=dev["n_live"], seq_row0=row0, capacity=cap, head_dim=hd, n_kv_heads=n_kv,
                               k_type=k_type, v_type=v_type)


CASES = [dict(n_kv=2, group=4, hd=128, k_type="q4_0", v_type="q4_0", n_live=[300, 1001], cap=[320, 1024]),
         dict(n_kv=1, group=1, hd=64, k_type="q4_0", v_type="f16", n_live=[77], cap=[80]),
         dict(n_kv=3, group=2, hd=96, k_type="q4_0", v_type="q8_0", n_live=[500, 33, 5], cap=[512, 40, 40]),
         dict(n_kv=1, group=8, hd=256, k_type="q4_0", v_type="q4_0", n_live=[400], cap=[400]),
         dict(n_kv=2, group=2, hd=32, k_type="q4_0", v_type="q4_0", n_live=[600], cap=[600]),
         dict(n_kv=1, group=4, hd=128, k_type="q4_0", v_type="q4_0", n_live=[257], cap=[300], nonrot=64),
         dict(n_kv=2, group=4, hd=128, k_type="f16", v_type="q4_0", n_live=[700], cap=[768]),
         dict(n_kv=2, group=4, hd=128, k_type="q8_0", v_type="q4_0", n_live=[700], cap=[768])]


@pytest.mark.parametrize("case", CASES)
def test_scores_and_passes(lib, case):
    n_kv, group, hd, cap, n_live = case["n_kv"], case["group"], case["hd"], case["cap"], case["n_live"]
    nonrot = case.get("nonrot", 0)
    host, row0, qm, qa, qn = build(n_kv, group, hd, case["k_type"], case["v_type"], n_live, cap, seed=hd, nonrot=nonrot)
    st = lib.Stats(qm, qa, n_kv_heads=n_kv, head_dim=hd, rope_theta=1e5, nonrot_dim=nonrot, q_nonrot=qn)
    cur = [5000 + 3 * n for n in n_live]
    budget = [max(8, n // 3) for n in n_live]
    pol = lib.Policy(budget_rows=budget, window=3, sink=2, cur_pos=cur)
    keys = A.values(host["k"], host["k_scale"], case["k_type"])
    omega, mw = O.rope_omega(hd, 1e5, nonrot), O.mlr_weight(qm[0], qa[0])
    dev, cache = device(lib, host, row0, cap, n_kv, hd, case["k_type"], case["v_type"])
    rows = len(host["pos"])
    ws = U.new_workspace(lib, cache, group)
    s_out, raw = torch.zeros(rows, device="cuda"), torch.zeros(rows, group, device="cuda")
    lib.score(st, 0, cache, pol, s_out, raw, ws=ws)
    assert lib.device_status(ws) == lib.OK
    want = {}
    for s, n in enumerate(n_live):
        for g in range(n_kv):
            r = slice(int(row0[s]) + g * cap[s], int(row0[s]) + g * cap[s] + n)
            h = slice(g * group, (g + 1) * group)
            ora_raw = O.raw_scores(keys[r], O.as_complex(qm[0])[h], mw[h], omega, cur[s], O.default_future_offsets(),
                                   **({"q_nonrot": qn[0][h]} if nonrot else {}))
            ora_s = O.gqa_max(O.znorm(ora_raw))
            U.assert_scores_close(raw[r].cpu().numpy(), ora_raw, s_out[r].cpu().numpy(), ora_s, f"seg {s},{g}")
            want[s, g] = (r, ora_s, O.select_keep(ora_s, n, budget[s], 2, 3))
    for name in ("evict", "evict_staged"):
        dev, cache = device(lib, host, row0, cap, n_kv, hd, case["k_type"], case["v_type"])
        ws = U.new_workspace(lib, cache, group)
        getattr(lib, name)(st, 0, cache, pol, ws=ws)
        assert lib.device_status(ws) == lib.OK
        assert dev["n_live"].tolist() == [min(n, b) for n, b in zip(n_live, budget)]
        for (s, g), (r, ora_s, keep) in want.items():
            got_pos = dev["pos"][r].cpu().numpy()[:len(keep)]
            got = (got_pos - 1) // 3 - r.start
            U.assert_keep_sets_match(got, keep, ora_s, n_live[s], budget[s], 2, 3, f"{name} {s},{g}")
            for plane in ("k", "v", "k_scale", "v_scale"):
                if host[plane] is not None:
                    assert dev[plane][r].cpu().numpy()[:len(got)].tobytes() == host[plane][r][got].tobytes(), plane
    st.close()


def test_model_calls_over_q4_keys_take_the_staged_kernels(lib):
    """Many short segments would take the fused kernel; it has no 4-bit scorer."""
    n_live, cap = [200] * 16, [208] * 16
    host, row0, qm, qa, _ = build(8, 4, 128, "q4_0", "q4_0", n_live, cap)
    st = lib.Stats(qm, qa, n_kv_heads=8, head_dim=128, rope_theta=1e6)
    dev, cache = device(lib, host, row0, cap, 8, 128, "q4_0", "q4_0")
    assert lib.evict_model_fused(st, [0], [cache]) is False
    pol = lib.Policy(budget_rows=[100] * 16, window=8, sink=0, cur_pos=[1000] * 16)
    ws = torch.empty(lib.model_workspace_size(cache, 1, 4), dtype=torch.uint8, device="cuda")
    lib.workspace_init(ws)
    lib.evict_model(st, [0], [cache], pol, ws=ws)
    assert lib.device_status(ws) == lib.OK and dev["n_live"].tolist() == [100] * 16
    other, cache2 = device(lib, host, row0, cap, 8, 128, "q4_0", "q4_0")
    lib.evict_staged(st, 0, cache2, pol, ws=U.new_workspace(lib, cache2, 4))
    for name in ("k", "v", "k_scale", "v_scale", "pos"):
        assert torch.equal(dev[name].view(torch.uint8), other[name].view(torch.uint8))
    st.close()
