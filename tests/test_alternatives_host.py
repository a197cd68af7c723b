"""Refusals and workspaces of the top alternatives and the distillation loss
(no GPU), and their oracle against closed forms."""

import math

import numpy as np
import pytest

from oracle import objective as ob
from quantized_rank_fine_amd import qlora as q

P = 0x10000
BAD = P + 1


def _swap(a, **kw):
    return list({**a, **kw}.values())


def test_top_refusals():
    f = q.lib().qlora_token_top
    T, V = 4, 200000
    n = q.qlora_token_top_workspace_bytes(T, V, q.BF16, 8)
    assert n > 0
    a = dict(x=P, ld=V, T=T, V=V, dt=q.BF16, y=P, s=1.0, k=8, ids=P, top=P, lp=P, h=P, ws=P, n=n,
             stream=None)
    for bad in (dict(V=0), dict(T=-1), dict(ld=V - 1), dict(T=(1 << 24) + 1), dict(k=0),
                dict(k=q.MAX_TOP + 1), dict(V=7, ld=7), dict(ld=(1 << 32) + 1)):
        assert f(*_swap(a, **bad)) == 2, bad
    assert f(*_swap(a, dt=2)) == 4
    for s in (0.0, -1.0, math.inf, math.nan, 2.4e38):
        assert f(*_swap(a, s=s)) == 7
    for k in ("x", "ids", "top"):
        assert f(*_swap(a, **{k: None})) == 1, k
    assert f(*_swap(a, y=None)) == 1                       # logp without labels
    for k in ("x", "y", "ids", "top", "lp", "h", "ws"):
        assert f(*_swap(a, **{k: BAD})) == 3, k
    assert f(*_swap(a, x=P + 2, dt=q.F32)) == 3
    assert f(*_swap(a, ws=None)) == 1 and f(*_swap(a, n=n - 1)) == 5
    assert f(*_swap(a, T=0, x=None, ids=None, top=None)) == 0


def test_distill_refusals():
    f = q.lib().qlora_distill_logits
    T, V = 4, 70000
    n = q.qlora_distill_workspace_bytes(T, V, q.BF16, 8)
    assert n > 0
    a = dict(x=P, ld=V, T=T, V=V, dt=q.BF16, s=1.0, w=P, k=8, ids=P, t=P, norm=1, loss=P, kl=P,
             dx=P, ldd=V, ws=P, n=n, stream=None)
    for bad in (dict(V=0), dict(T=-1), dict(ld=V - 1), dict(ldd=V - 1), dict(k=0),
                dict(k=q.MAX_TOP + 1), dict(ldd=(1 << 32) + 1)):
        assert f(*_swap(a, **bad)) == 2, bad
    assert f(*_swap(a, dt=-1)) == 4 and f(*_swap(a, s=0.0)) == 7
    for k in ("x", "ids", "t", "loss", "kl", "dx"):
        assert f(*_swap(a, **{k: None})) == 1, k
    for k in ("x", "w", "ids", "t", "loss", "kl", "dx", "ws"):
        assert f(*_swap(a, **{k: BAD})) == 3, k
    assert f(*_swap(a, dx=P + 2, dt=q.F32)) == 3
    assert f(*_swap(a, ws=None)) == 1 and f(*_swap(a, n=n - 1)) == 5
    assert f(*_swap(a, T=0, loss=None)) == 1
    # in place, rows of another pitch would overwrite logits that are still to be read
    assert f(*_swap(a, ldd=V + 8)) == 2 and f(*_swap(a, ld=V + 8)) == 2


def test_workspaces():
    top, dis = q.qlora_token_top_workspace_bytes, q.qlora_distill_workspace_bytes
    assert top(4096, 32000, q.BF16, 20) == 0 and top(65, 200000, q.F32, 20) == 0
    assert top(1, 200000, q.F32, 20) >= 25 * (12 + 20 * 8)
    assert dis(4096, 32000, q.BF16, 20) == 0 and dis(8193, 32000, q.BF16, 20) >= 9 * 8
    assert dis(100, 70000, q.BF16, 20) >= 100 * (9 * 12 + 8)
    for f in (top, dis):
        assert f(4, 0, q.BF16, 2) == 0 and f(4, 100, 3, 2) == 0 and f(4, 100, q.BF16, 0) == 0
        assert f(4, 100, q.BF16, 65) == 0


def test_oracle_top():
    x = np.array([[1.0, 3.0, 3.0, -np.inf, 2.0], [0.0, -0.0, 0.0, 0.0, -1.0]])
    ids, lp = ob.token_top(x, 4)
    assert ids.tolist() == [[1, 2, 4, 0], [0, 1, 2, 3]]
    z = np.log(np.exp([1.0, 3.0, 3.0, 2.0]).sum())
    assert np.allclose(lp[0], np.array([3, 3, 2, 1]) - z)
    ids, lp = ob.token_top(x, 5)
    assert ids[0, 4] == 3 and lp[0, 4] == -np.inf
    assert ob.token_top(np.array([[np.nan, 1.0, 2.0]]), 2)[0].tolist() == [[2, 1]]


def test_oracle_top_of_nan_beside_a_mask():
    """A NaN is behind a word at -inf, and no word where too few are left."""
    n, i = np.nan, np.inf
    x = np.array([[n, -i, -i, -i], [-i, n, 1.0, n], [n, n, n, n], [-i, n, -i, i]])
    assert ob.token_top(x, 3)[0].tolist() == [[1, 2, 3], [2, 0, -1], [-1, -1, -1], [3, 0, 2]]


@pytest.mark.parametrize("s", [1.0, 0.7])
def test_oracle_distill(s):
    """Against itself the loss is 0 and so is the gradient; one alternative is
    cross-entropy; an unnormalised teacher of weight c is c times that plus
    c ln c; a word named twice counts twice."""
    g = np.random.default_rng(0)
    x = g.standard_normal((1, 6))
    lp = s * x - np.log(np.exp(s * x).sum())
    every = np.arange(6)[None].astype(np.int32)
    loss, kl, d = ob.distill(x, every, lp, [1.0], s)
    assert abs(loss) < 1e-14 and np.abs(d).max() < 1e-14
    loss, _, d = ob.distill(x, np.array([[2]]), np.array([[-3.0]]), [2.0], s)
    want = s * 2.0 * (np.exp(lp) - np.eye(6)[2])
    assert np.isclose(loss, -2 * lp[0, 2]) and np.allclose(d, want)
    half = np.log(np.array([[0.5]]))
    loss, _, d = ob.distill(x, np.array([[2]]), half, [2.0], s, False)
    assert np.isclose(loss, 2 * 0.5 * (np.log(0.5) - lp[0, 2])) and np.allclose(d, 0.5 * want)
    a = ob.distill(x, np.array([[2, 2, -1]]), np.zeros((1, 3)), [1.0], s)
    assert np.allclose(a[2], s * (np.exp(lp) - np.eye(6)[2]))
    assert ob.distill(x, np.array([[-1]]), np.zeros((1, 1)), [1.0], s)[0] == 0
