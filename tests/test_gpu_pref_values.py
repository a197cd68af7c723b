"""The preference loss at infinite log-ratios: an answer that its model cannot
give (a counted token with log-probability -inf)."""

import math

import numpy as np
import pytest

from oracle import objective as ob
from quantized_rank_fine_amd import qlora as q

from gpu_harness import say
from test_gpu_objective import U, _pref, f32

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("lens", [
    [5, 7, 3, 6, 8, 9],                                  # one workgroup
    [700 + 11 * i for i in range(130)],                  # a workgroup to a pair
    [9001, 3, 64, 30000, 4097, 5],                       # slices
    [i % 5 + 1 for i in range(1400)],                    # the losses by the workspace
])
@pytest.mark.parametrize("kind", ["sigmoid", "hinge"])
@pytest.mark.parametrize("average", [False, True])
def test_impossible_rejected_answer(lens, kind, average):
    """h = +inf: no loss and no gradient, in the sigmoid loss too (without
    smoothing -log sigma(inf) = 0, and 0 of the other term is 0).  The rest of
    the batch is as if the pair's margin were merely wide."""
    say(f"[pref inf] {len(lens) // 2} pairs {kind} average={average}")
    g = np.random.default_rng(len(lens))
    P = len(lens) // 2
    cu = np.concatenate([[0], np.cumsum(lens)])
    lp = -np.abs(g.standard_normal(int(cu[-1]))).astype(np.float32)
    at = int(cu[P + 1])                                  # pair 1's rejected answer
    lp[at] = -np.inf
    beta, margin = f32(0.1), f32(0.25)
    wide = lp.copy()
    wide[at] = -1e9                                      # e^-u is 0 in float64 as well
    rl, rr, rd = ob.pref_loss(kind, wide, None, None, cu, beta, margin, 0.0, average)
    pref = q.pref_struct(q.PREF_SIGMOID if kind == "sigmoid" else q.PREF_HINGE, beta, margin, 0.0,
                         average)
    loss, rw, d = _pref(lp, None, None, cu, pref)
    assert rw[P + 1] == -math.inf and np.isfinite(np.delete(rw, P + 1)).all()
    assert not d[cu[1]:cu[2]].any() and not d[at:cu[P + 2]].any()
    # S is below the longest answer's sum of |logp|: u to 8 u of beta times that, and of margin
    big = max(np.abs(wide[int(a):int(b)][np.isfinite(lp[int(a):int(b)])]).sum()
              for a, b in zip(cu[:-1], cu[1:]))
    tol = 8 * U * (beta * 2 * big + margin + 1)
    assert abs(loss - rl) <= tol
    assert np.all(np.abs(d - rd) <= beta * (tol + 4 * U) / P)


def test_impossible_chosen_answer_is_an_infinite_loss():
    pref = q.pref_struct(q.PREF_SIGMOID, 0.1)
    loss, rw, d = _pref(np.array([-np.inf, -1.0], np.float32), None, None, [0, 1, 2], pref)
    assert loss == math.inf and rw[0] == -math.inf
    assert abs(d[0] + f32(0.1)) <= 4 * U and abs(d[1] - f32(0.1)) <= 4 * U


def test_smoothing_of_an_infinite_margin_is_an_infinite_loss():
    """With smoothing the other term's log is infinite."""
    pref = q.pref_struct(q.PREF_SIGMOID, 0.1, 0.0, 0.125)
    loss, _, d = _pref(np.array([-1.0, -np.inf], np.float32), None, None, [0, 1, 2], pref)
    assert loss == math.inf and abs(d[0] - f32(0.1) * 0.125) <= 4 * U
