"""What tria_attend's roundings are, held to bounds that count no others: exact
codes and fp32 scales of keys in decode steps and prompts, bf16 queries, outputs
that do not depend on what else is asked for."""
import numpy as np
import pytest

import _rows as R

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")


def ask(lib, c, q, pos, tok0, *, lse=True, **kw):
    n, nq = q.shape[:2]
    out = torch.full_like(q, 7.0)
    l = torch.full((n, nq), 7.0, device="cuda") if lse else None
    ws = c.ws(lib.attend_workspace_size(c.cache, nq, tok0))
    lib.attend(c.cache, q, out, torch.from_numpy(pos).cuda(), tok0=tok0, lse=l, ws=ws, **kw)
    assert lib.device_status(ws) == lib.OK
    return out, l


def newest(c, tokens):
    tok0 = np.concatenate([[0], np.cumsum(tokens)]).astype(np.int32)
    return tok0, np.concatenate([c.last(s) - np.arange(t)[::-1] for s, t in enumerate(tokens)]).astype(np.int32)


@pytest.mark.parametrize("kind,k,v", [("f16", "q8_0", "q4_0"), ("bf16", "q4_0", "f16"), ("f16", "f16", "q8_0"), ("f32", "q4_0", "f32")])
@pytest.mark.parametrize("hd", [64, 128, 192, 256])
@pytest.mark.parametrize("round_keys", [False, True])
@pytest.mark.parametrize("tokens", [[1, 4], [70, 30]])
def test_outputs_do_not_depend_on_whether_lse_is_asked_for(lib, kind, k, v, hd, round_keys, tokens):
    rng = np.random.default_rng(hd)
    c = R.Cache(lib, rng, rows=[700, 80], cap=[710, 80], n_kv=2, hd=hd, k_type=k, v_type=v)
    tok0, pos = newest(c, tokens)
    q = R.act(rng.standard_normal((int(tok0[-1]), 8, hd)) * 3, kind)
    with_lse, lse = ask(lib, c, q, pos, tok0, round_keys=round_keys)
    without, _ = ask(lib, c, q, pos, tok0, lse=False, round_keys=round_keys)
    assert torch.equal(with_lse, without)
    want = R.attend_expected(c, R.host(q), pos, tok0, 8)
    R.check_attend(R.host(without), R.host(lse), want, kind, kind != "f32", 700, hd, q_exact=kind != "bf16", k_exact=k == "f16")


@pytest.mark.parametrize("k", ["q8_0", "q4_0"])
def test_rounded_keys_are_the_prompts_alone(lib, k):
    """round_keys changes a prompt's bits and leaves decode steps, fp16 keys and fp32 calls as they are."""
    rng = np.random.default_rng(3)
    for kind, kt, tokens, same in (("f16", k, [40], False), ("f16", k, [2], True), ("f16", "f16", [40], True), ("f32", k, [40], True)):
        c = R.Cache(lib, rng, rows=[500], cap=[500], n_kv=1, hd=128, k_type=kt, v_type="f16")
        tok0, pos = newest(c, tokens)
        q = R.act(rng.standard_normal((tokens[0], 4, 128)) * 8, kind)
        a, b = (ask(lib, c, q, pos, tok0, round_keys=r) for r in (False, True))
        assert torch.equal(a[1], b[1]) == same and (torch.equal(a[0], b[0]) or not same)
