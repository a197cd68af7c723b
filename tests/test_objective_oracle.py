"""Pins of the oracle's objectives and generator (no GPU): published values,
closed forms, and every gradient against central differences of its loss."""

import math

import numpy as np
import pytest

from oracle import objective as ob


def test_philox_known_answers():
    """The published known answers of Philox4x32-10 (Salmon et al.'s vectors
    for zero, all-ones and pi-digit inputs)."""
    ff = 0xFFFFFFFF
    assert ob.philox4x32((0, 0, 0, 0), (0, 0)) == (0x6627E8D5, 0xE169C58D, 0xBC57AC4C, 0x9B00DBD8)
    assert ob.philox4x32((ff,) * 4, (ff, ff)) == (0x408F276D, 0x41C83B0E, 0xA20BC7C6, 0x6D5451FD)
    assert ob.philox4x32((0x243F6A88, 0x85A308D3, 0x13198A2E, 0x03707344),
                         (0xA4093822, 0x299F31D0)) == (0xD16CFE09, 0x94FDCCEB, 0x5001E420,
                                                       0x24126EA1)


def test_dropout_rate_and_rows():
    keep, p16 = ob.dropout_keep(64, 100, 0.25, 7, 3)
    assert p16 == 16384
    # 6400 draws: 5 standard deviations of a binomial
    assert abs(keep.mean() - 0.75) < 5 * math.sqrt(0.75 * 0.25 / keep.size)
    part, _ = ob.dropout_keep(64, 100, 0.25, 7, 3, only=[5, 63])
    assert np.array_equal(part, keep[[5, 63]])
    assert ob.dropout_keep(4, 16, 0.0, 1, 1)[0].all()


def test_uniform_row_and_masked_words():
    x = np.zeros((2, 10))
    x[1, 4:] = -np.inf
    lp, m, z, h = ob.token_logp(x, [3, 1])
    assert np.allclose(lp, [-math.log(10), -math.log(4)])
    assert np.allclose(z, [math.log(10), math.log(4)]) and np.allclose(h, z)
    assert np.all(m == 0)
    g = ob.logits_grad(x, [3, 1], [1.0, 1.0], [0.5, 0.5])
    assert np.all(g[1, 4:] == 0) and np.isclose(g[1, 1], 0.75)
    # nothing scored, nothing possible
    assert np.all(ob.token_logp(x, [-100, 10]) == 0)
    x[:] = -np.inf
    assert np.array_equal(ob.token_logp(x, [0, -1])[:, 0], [-np.inf, -np.inf, 0, 0])
    assert np.all(ob.logits_grad(x, [0, 1], [1.0, 1.0], [1.0, 1.0]) == 0)


def _diff(f, x, h=1e-6):
    d = np.zeros_like(x)
    for i in np.ndindex(*x.shape):
        a, b = x.copy(), x.copy()
        a[i] += h
        b[i] -= h
        d[i] = (f(a) - f(b)) / (2 * h)
    return d


def test_logits_grad_is_the_difference_quotient():
    g = np.random.default_rng(1)
    x, y = g.standard_normal((3, 7)) * 2, [2, -100, 6]
    c, e, s = g.standard_normal(3), g.standard_normal(3), 1.3
    f = lambda v: (lambda r: float(c @ r[0] + e @ r[3]))(ob.token_logp(v, y, s))  # noqa: E731
    assert np.allclose(ob.logits_grad(x, y, c, e, s), _diff(f, x), atol=1e-8)


@pytest.mark.parametrize("kind", ["sigmoid", "squared", "hinge"])
@pytest.mark.parametrize("average", [False, True])
def test_pref_grad_is_the_difference_quotient(kind, average):
    g = np.random.default_rng(2)
    cu = [1, 5, 5, 9, 12]                  # the second answer is empty
    lp, ref = -g.random(13), -g.random(13)
    mask = np.array([1, 1, 0, 1, 1, 1, 1, 0, 1, 0, 0, 0, 1])   # the last answer has no token
    a = (cu, 0.3, 0.1, 0.05, average)
    f = lambda v: ob.pref_loss(kind, v, ref, mask, *a)[0]  # noqa: E731
    loss, rewards, grad = ob.pref_loss(kind, lp, ref, mask, *a)
    assert np.allclose(grad, _diff(f, lp), atol=1e-8)
    assert rewards[1] == 0 and rewards[3] == 0 and np.all(grad[[0, 2, 7, 12]] == 0)


def test_pref_closed_forms():
    assert np.isclose(ob.pair_loss("sigmoid", 0.0, 0.1)[0], math.log(2))
    assert np.isclose(ob.pair_loss("sigmoid", 0.0, 0.1)[1], -0.05)
    assert ob.pair_loss("squared", 5.0, 0.1) == (0.0, 0.0)
    assert ob.pair_loss("hinge", 30.0, 0.1) == (0.0, 0.0)


@pytest.mark.parametrize("kind,dual", [("clip", 0.0), ("clip", 1.5), ("nll", 0.0)])
def test_policy_grad_is_the_difference_quotient(kind, dual):
    g = np.random.default_rng(3)
    n = 40
    lp, h = -g.random(n), g.random(n)
    old, ref = lp - g.standard_normal(n) * 0.5, lp + g.standard_normal(n)
    w, adv = g.random(n) * (g.random(n) > 0.2), g.standard_normal(n)
    a = (w, adv, old, ref, 0.2, 0.3, dual, 0.1, 0.01)
    out, dlp, dh = ob.policy_loss(kind, lp, h, *a)
    assert np.allclose(dlp, _diff(lambda v: ob.policy_loss(kind, v, h, *a)[0][0], lp), atol=1e-8)
    assert np.allclose(dh, _diff(lambda v: ob.policy_loss(kind, lp, v, *a)[0][0], h), atol=1e-8)
    # every branch is taken; the KL estimate is not negative
    d = lp - old
    if kind == "clip":
        for far in (d > math.log(1.3), d < math.log(0.8)):
            assert (far & (adv > 0)).any() and (far & (adv < 0)).any()
    assert out[1] >= 0


def test_policy_skips_tokens_of_no_weight():
    nan = float("nan")
    out, g, gh = ob.policy_loss("clip", [nan, -1.0], [nan, 2.0], [0.0, 0.5], [nan, 1.0],
                                [nan, -1.0], [nan, -1.0], ent_coef=0.1)
    assert np.allclose(out, [0.5 * (-1.0 - 0.2), 0, 0, 1.0])
    assert np.allclose(g, [0, -0.5]) and np.allclose(gh, [0, -0.05])
