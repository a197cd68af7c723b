"""The inverse temperature at the ends of its range."""

import math

import numpy as np
import pytest

from quantized_rank_fine_amd import qlora as q

from test_gpu_objective import U, _dev, _fwd, _policy_logits, f32

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("s", [2.3e38, 1e30, 1e-30, 1e-38])
@pytest.mark.parametrize("V", [5, 5000, 70001])
def test_extreme_scales(s, V):
    """The largest logit alone, or all of them alike: log 2 of two equal ones,
    log of the count where the scale leaves no difference."""
    s = f32(s)
    x = np.full((2, V), -3.0, np.float32)
    x[:, 1] = x[:, 4] = 2.0
    x[:, 2] = 1.0
    y = np.array([4, 2])
    lp, st, h = _fwd(_dev(x), V, "f32", _dev(y), s)
    n = 2 if s > 1 else V
    want = np.array([-math.log(n), -math.log(n) - s])
    tol = (V / 64 + 64) * U * (1 + np.abs(want))
    assert np.all(np.abs(lp.cpu().numpy() - want) <= tol)
    assert np.all(np.abs(h.cpu().numpy() - math.log(n)) <= tol[0] * 3)
    out, l2, dx, _ = _policy_logits(_dev(x), V, "f32", y, s, q.policy_struct(q.OBJ_NLL),
                                    np.array([0.25, 0.0], np.float32))
    got = dx.cpu().numpy().astype(float)
    hot = np.zeros(V)
    hot[4] = 1.0
    p = np.where(x[0] == 2.0, 0.5, 0.0) if n == 2 else np.full(V, 1.0 / V)
    assert np.all(np.abs(got[0] - 0.25 * s * (p - hot)) <= s * (V / 64 + 64) * U)
    assert not got[1].any()
