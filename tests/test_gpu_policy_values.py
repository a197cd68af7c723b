"""The policy objective where its terms nearly vanish, overflow or are
switched off: the KL estimate's digits, infinite log-ratios, coefficients and
advantages of 0."""

import math

import numpy as np
import pytest

from quantized_rank_fine_amd import qlora as q

from gpu_harness import say, torch_dev
from test_gpu_objective import U, _dev, _policy_logits

pytestmark = pytest.mark.gpu


def _loss(pol, logp, adv=None, old=None, ref=None, weight=None):
    """out, dlogp of qlora_policy_loss."""
    torch, dev = torch_dev()
    T = len(logp)
    out, d = torch.full((4,), 9.0, device=dev), torch.full((T,), 9.0, device=dev)
    n = q.qlora_policy_workspace_bytes(T)
    ws = torch.empty(n, dtype=torch.uint8, device=dev) if n else None
    a = [None if v is None else _dev(np.asarray(v, np.float32)) for v in (logp, weight, adv, old,
                                                                         ref)]
    q.qlora_policy_loss(a[0], None, T, a[1], a[2], a[3], a[4], pol, out, d, None, ws, n)
    return out.cpu().numpy().astype(float), d.cpu().numpy().astype(float)


def _k(v):
    """exp(v) - v - 1 in float64, by its series where it cancels."""
    if abs(v) > 1.0:
        return math.expm1(v) - v
    return sum(v ** n / math.factorial(n) for n in range(2, 24))


@pytest.mark.parametrize("sign", [1, -1])
def test_kl_estimate_keeps_its_digits(sign):
    """Relative to k itself, and never below 0.  q = ref - logp is exact here
    for |q| <= 1/2 (logp = -1), else rounded once (at most 3 u of k).  In fp32
    the product q q, the polynomial beside it (its constant 1/2 and a first
    term of at most a sixth of it, five roundings of half an ulp and less) and
    their product err by at most 6 u;
    for larger |q| expm1 (an ulp, 2 u, of its value) and the difference err by
    2 u (e^q + |q|) + u k.  The weight is 1: the sums add a rounding."""
    for size in [2.0 ** -23, 2.0 ** -20, 1e-6, 1e-5, 1e-4, 1e-3, 1e-2, 0.05, 0.1, 0.2, 0.3, 0.4,
                 0.49, 0.499999, 0.5, 0.500001, 0.6, 0.75, 0.99]:
        ref = np.float32(-1.0 + sign * size)
        v = float(ref) + 1.0
        say(f"[kl digits] q={v}")
        out, d = _loss(q.policy_struct(q.OBJ_NLL, kl_coef=1.0), [-1.0], adv=[0.0], ref=[ref])
        want = _k(v)
        rel = 8 * U if abs(v) < 0.5 else 2 * U * (math.exp(v) + abs(v)) / want + 4 * U
        assert out[1] >= 0 and abs(out[1] - want) <= rel * want, v
        assert abs(out[0] - want) <= rel * want
        assert abs(d[0] + math.expm1(v)) <= 4 * U * abs(math.expm1(v))
    out, d = _loss(q.policy_struct(q.OBJ_NLL, kl_coef=1.0), [-1.0], adv=[0.0], ref=[-1.0])
    assert out[1] == 0 and out[0] == 0 and d[0] == 0


def test_kl_estimate_of_far_ratios():
    """exp(q) past fp32, and q infinite, give an infinite estimate, not NaN:
    exp(q) - q - 1 has that limit at both ends."""
    inf = math.inf
    for logp, old, ref in ((-100.0, -100.0, -1.0), (-inf, -1.0, -1.0), (-1.0, -1.0, -inf)):
        out, _ = _loss(q.policy_struct(q.OBJ_CLIP, kl_coef=1.0), [logp, -1.0], old=[old, -1.0],
                       ref=[ref, -1.0])
        assert out[1] == inf and out[0] == inf, (logp, ref)


@pytest.mark.parametrize("kind", [q.OBJ_NLL, q.OBJ_CLIP])
def test_no_kl_coefficient_takes_nothing_from_the_ratio(kind):
    """kl_coef = 0 with a reference (the estimate is reported only): the loss
    and the gradient are those without one, however far the reference is."""
    logp, ref = [-2.0, -100.0, -1.0, -math.inf], [-1.0, -1.0, -math.inf, -1.0]
    old, adv = [-2.1, -100.0, -1.0, -1.0], [1.0, -0.5, 2.0, 0.75]
    w = [0.25, 0.5, 0.125, 0.0625]
    if kind == q.OBJ_NLL:                        # a log-likelihood of -inf is an infinite loss
        logp, ref, old, adv, w = (v[:3] for v in (logp, ref, old, adv, w))
    pol = q.policy_struct(kind)
    a, da = _loss(pol, logp, adv, old, None, w)
    b, db = _loss(pol, logp, adv, old, ref, w)
    assert np.isfinite(a).all() and np.isfinite(da).all()
    assert b[0] == a[0] and np.array_equal(da, db) and b[1] == math.inf


def test_no_advantage_takes_nothing_from_the_policy():
    """An advantage of 0 (all answers of a prompt rewarded alike): no loss, no
    bound and no gradient, whatever the ratio or the log-probability."""
    far = [-1.0, -1.0, -1.0, -math.inf]
    out, d = _loss(q.policy_struct(q.OBJ_CLIP), far, [0.0] * 4, [-101.0, -1.0, -0.5, -1.0])
    assert not out.any() and not d.any()
    out, d = _loss(q.policy_struct(q.OBJ_CLIP, clip_hi=math.inf), far, [0.0, -0.0] * 2,
                   [-200.0, -90.0, -math.inf, -1.0])
    assert not out.any() and not d.any()
    out, d = _loss(q.policy_struct(q.OBJ_NLL), far, [0.0] * 4)
    assert not out.any() and not d.any()


@pytest.mark.parametrize("V", [9, 70001])
def test_policy_logits_of_masked_labels_and_far_ratios(V):
    """The same through the logits: a label at -inf beside kl_coef = 0 and
    beside an advantage of 0, and a ratio past fp32."""
    torch, dev = torch_dev()
    g = np.random.default_rng(V)
    x = g.standard_normal((4, V)).astype(np.float32)
    y = np.array([3, 4, 5, 6])
    x[1, 4] = x[2, 5] = -np.inf
    adv, w = np.array([1.0, 0.0, 0.5, 0.0], np.float32), np.full(4, 0.25, np.float32)
    old = np.array([-math.log(V), -1.0, -1.0, -200.0], np.float32)
    ref = np.full(4, -1.0, np.float32)
    pol = q.policy_struct(q.OBJ_CLIP, 0.2, math.inf, 0.0, 0.0, 0.0)
    out, lp, dx, _ = _policy_logits(_dev(x), V, "f32", y, 1.0, pol, w, adv, old, ref)
    assert np.isfinite(out[0]) and out[1] == math.inf and out[2] == 0
    assert lp[1] == -math.inf and lp[2] == -math.inf
    got = dx.cpu().numpy()
    assert np.isfinite(got).all() and not got[1:].any() and got[0].any()
