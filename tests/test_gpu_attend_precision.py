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


def lost_of_bf16(c, q, scale):
    """A head of bf16 queries whose largest value lies in [2^e, 2^(e + 1)) is taken times 2^-e as fp16, exactly but for
    values whose last place lies under fp16's smallest step: 2^-25 off at most. So a logit is off by at most
    scale 2^(e - 25) sum |k|."""
    top = np.abs(q).max(-1)
    e = np.floor(np.log2(np.where(top > 0, top, 1.0)))
    k = max(np.abs(c.values("k", s, g)).sum(-1).max(initial=0.0) for s in range(len(c.rows)) for g in range(c.n_kv))
    return scale * 2.0 ** (e - 25) * k


@pytest.mark.parametrize("size", [1.0, 1e-4, 1e-6])
@pytest.mark.parametrize("kind", ["f16", "bf16"])
@pytest.mark.parametrize("k,v", [("q8_0", "q8_0"), ("q4_0", "q4_0"), ("q4_0", "f16"), ("q8_0", "q4_0")])
@pytest.mark.parametrize("hd,tokens", [(64, [1, 2]), (128, [1, 4]), (256, [2, 1]), (96, [3, 1]), (64, [70, 30]), (128, [61, 7]),
                                       (256, [40, 9]), (192, [33, 12])])
def test_logits_over_codes_carry_no_rounding_of_keys(lib, k, v, hd, tokens, kind, size):
    """lse within fp32's roundings alone: sums of 2 hd products (keys, and in prompts their remainders) are off by at
    most (2 hd + 3) 2^-24 of the sum of moduli, exponentials and sums of weights by (rows / 32 + 64) 2^-24, the
    logarithm and the last product by 4 x 2^-24 of the result. Block scales around 1, near fp16's smallest normal
    number and below it (a product of code and scale is then a multiple of 2^-24, and so is its remainder)."""
    rng = np.random.default_rng(hd)
    c = R.Cache(lib, rng, rows=[333, 80], cap=[340, 80], n_kv=2, hd=hd, k_type=k, v_type=v)
    c.h["k_scale"][...] = (c.h["k_scale"].astype(np.float32) * np.float32(size)).astype(np.float16)
    c.d["k_scale"].copy_(torch.from_numpy(c.h["k_scale"]))
    tok0, pos = newest(c, tokens)
    q = R.act(rng.standard_normal((int(tok0[-1]), 8, hd)), kind)
    scale = 1.0 / (size * np.sqrt(hd))
    out, lse = ask(lib, c, q, pos, tok0, scale=scale)
    want = R.attend_expected(c, R.host(q), pos, tok0, 8, scale=scale)
    dS = (2 * hd + 3) * R.U24 * want[3]
    if kind == "bf16":
        dS = dS + lost_of_bf16(c, R.host(q), scale)
    tl = dS + (333 / 32 + 64) * R.U24 + 4 * R.U24 * np.abs(want[1])
    off = np.abs(R.host(lse) - want[1])
    assert np.all(off <= tl), np.max(off / tl)
    R.check_attend(R.host(out), R.host(lse), want, kind, True, 333, hd, q_exact=kind == "f16", k_exact=False)


@pytest.mark.parametrize("hd", [64, 128, 256])
def test_logits_of_bf16_queries_over_fp16_keys(lib, hd):
    """bf16 queries over wide ranges: the power of two that takes them into fp16's range costs what lost_of_bf16 says."""
    rng = np.random.default_rng(hd)
    c = R.Cache(lib, rng, rows=[300, 90], cap=[310, 96], n_kv=2, hd=hd, k_type="f16", v_type="f16")
    for tokens in ([1, 3], [50, 20]):
        for heat in (1.0, 1e-20, 1e15):
            tok0, pos = newest(c, tokens)
            x = rng.standard_normal((int(tok0[-1]), 8, hd)) * 2.0 ** rng.integers(-12, 1, (int(tok0[-1]), 8, hd)) * heat
            q = R.act(x, "bf16")
            scale = 1.0 / (heat * np.sqrt(hd))
            out, lse = ask(lib, c, q, pos, tok0, scale=scale)
            want = R.attend_expected(c, R.host(q), pos, tok0, 8, scale=scale)
            tl = (hd + 2) * R.U24 * want[3] + lost_of_bf16(c, R.host(q), scale) + (300 / 32 + 64) * R.U24 + 4 * R.U24 * np.abs(want[1])
            off = np.abs(R.host(lse) - want[1])
            assert np.all(off <= tl), (tokens, heat, np.max(off / tl))


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
