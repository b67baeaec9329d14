"""tria_beam_select where 64 bits of v do not tell continuations apart: those of a
beam keep their logits' order, equal logits their tokens', beams their own;
and log-probabilities near zero."""
import numpy as np
import pytest

import _rows as R
from oracle import beam_oracle as B
from test_gpu_beams import LOG_TOL, check, make, run

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")


@pytest.mark.parametrize("kind", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("vocab", [40, 3000, 40000])
@pytest.mark.parametrize("n_out", [1, 9, 64])
def test_totals_that_hide_the_logits(lib, kind, vocab, n_out):
    """Totals as low as a mask's: v is the total, whatever the logit."""
    rng = np.random.default_rng(vocab + n_out)
    logits = make(rng, 3, vocab, kind)
    total = np.asarray([-1e30, -3e38, -1e30], np.float32)
    exact(run(lib, logits, total, [0, 3], n_out), logits, total, n_out)


@pytest.mark.parametrize("vocab", [40, 3000, 40000])
@pytest.mark.parametrize("size", [1e-17, 1e-30])
def test_logits_that_differ_by_less_than_their_values(lib, vocab, size):
    rng = np.random.default_rng(vocab)
    logits = make(rng, 4, vocab, "f32", size)
    for total in ([0.0, 0.0, -1.0, 0.0], [-2.0, -1.0, -1.0, -2.0]):
        for n_out in (3, 64):
            exact(run(lib, logits, total, [0, 4], n_out), logits, np.asarray(total, np.float32), n_out)


def exact(got, logits, total, n_out):
    x = logits.double().cpu().numpy()
    v = B.values(x, total)
    want = B.choose(v, 0, n_out, logits=x)
    assert got["parent"][0].tolist() == [b for b, _, _ in want] and got["token"][0].tolist() == [t for _, t, _ in want]
    w = np.asarray([val for _, _, val in want])
    assert np.all(np.abs(got["total_out"][0] - w) <= R.U24 * np.abs(w) + LOG_TOL)


@pytest.mark.parametrize("kind", ["f16", "f32"])
@pytest.mark.parametrize("vocab", [40, 9000, 100001])
def test_log_probabilities_near_zero(lib, kind, vocab):
    """Rows with one token that is all but sure, and totals of zero: what is left is the sum's rounding, bounded absolutely."""
    rng = np.random.default_rng(vocab)
    for gap in (3.0, 10.0, 17.0, 40.0):
        logits = make(rng, 4, vocab, kind, 0.5) - gap - np.log(vocab)
        for b in range(4):
            logits[b, (b * 977) % vocab] = 5.0
        check(run(lib, logits, [0.0] * 4, [0, 2, 4], 2), logits, [0.0] * 4, [0, 2, 4], 2)
