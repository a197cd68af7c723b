"""Refusals and workspace of the orthogonalised update (no GPU), and its
oracle against closed forms."""

import ctypes
import math

import numpy as np
import pytest

import oracle
from quantized_rank_fine_amd import qlora as q

P = 0x10000
BAD = P + 2


def _call(mats=None, ws=P, short=0, n=None, **hp):
    h = dict(lr=0.1, momentum=0.9, weight_decay=0.0, nesterov=1, steps=5, eps=1e-7,
             coef=q.MUON_COEF)
    h.update(hp)
    h["coef"] = (ctypes.c_double * 3)(*h["coef"])
    arr = q.muon_mats([q.muon_mat(100, 16, P, P, P, P, P)] if mats is None else mats)
    size = q.qlora_muon_workspace_bytes(arr) if len(arr) else 0
    s = q.qlora_muon_hparams(**h)
    return q.lib().qlora_muon_step(len(arr) if n is None else n, arr, ctypes.byref(s), ws,
                                   size - short, None)


def test_refusals():
    mat = lambda **kw: [q.muon_mat(**{**dict(rows=100, cols=16, grad=P, m=P, theta=P,  # noqa: E731
                                             theta_bf16=P, update=P), **kw})]
    for kw in (dict(rows=0), dict(cols=0), dict(rows=-1), dict(rows=257, cols=257),
               dict(rows=(1 << 24) + 1), dict(cols=(1 << 24) + 1)):
        assert _call(mat(**kw)) == 2, kw
        assert q.qlora_muon_workspace_bytes(q.muon_mats(mat(**kw))) == 0
    assert _call(n=-1) == 2 and _call(n=q.MUON_MAX_MATS + 1) == 2
    assert q.lib().qlora_muon_step(1, None, None, P, 1 << 20, None) == 1
    assert q.lib().qlora_muon_step(0, None, None, None, 0, None) == 1      # no hparams
    assert _call(mat(grad=None)) == 1
    assert _call(mat(theta=None)) == 1                                     # a copy of nothing
    for k in ("grad", "m", "theta", "update"):
        assert _call(mat(**{k: BAD})) == 3, k
    assert _call(mat(theta_bf16=P + 1)) == 3
    for kw in (dict(lr=math.nan), dict(momentum=-0.1), dict(momentum=math.inf),
               dict(weight_decay=-1.0), dict(eps=-1e-9), dict(eps=math.nan), dict(steps=0),
               dict(steps=17), dict(steps=9), dict(coef=(math.nan, 0, 0)),
               dict(coef=(1, math.inf, 0)), dict(coef=(-40.0, 1, 1))):
        assert _call(**kw) == 7, kw
    assert _call(mat(scale=math.inf)) == 7
    assert _call(ws=None) == 1 and _call(ws=P + 8) == 3 and _call(short=1) == 5
    assert _call([]) == 0


def test_workspace_depends_on_the_shapes_alone():
    a = q.muon_mats([q.muon_mat(4096, 16, P), q.muon_mat(16, 4096, P)])
    b = q.muon_mats([q.muon_mat(4096, 16, P + 4, P, P), q.muon_mat(16, 4096, P, scale=2)])
    assert q.qlora_muon_workspace_bytes(a) == q.qlora_muon_workspace_bytes(b) > 0
    for shape in ((1, 1), (1 << 24, 1), (1, 1 << 24), (256, 1 << 24), (1 << 24, 256)):
        assert q.qlora_muon_workspace_bytes(q.muon_mats([q.muon_mat(*shape, P)])) > 0
    assert q.qlora_muon_workspace_bytes(q.muon_mats([])) == 0


def test_binding_takes_tensors_and_none():
    m = q.muon_mat(4, 2, 64, None, 128)
    assert (m.grad, m.m, m.theta, m.scale) == (64, None, 128, 1.0)


@pytest.mark.parametrize("shape", [(6, 6), (9, 4), (4, 9)])
def test_oracle_of_orthogonal_and_of_scaled_input(shape):
    """An orthogonal matrix over its norm has all singular values 1 / sqrt(k);
    the input's size does not matter (eps = 0); the cubic polynomial converges
    to the polar factor."""
    g = np.random.default_rng(0)
    u, _, v = np.linalg.svd(g.standard_normal(shape), full_matrices=False)
    k = min(shape)
    s = 1 / math.sqrt(k)
    for _ in range(5):
        s = 3.4445 * s - 4.7750 * s ** 3 + 2.0315 * s ** 5
    assert np.allclose(oracle.orthogonalize(u @ v, eps=0.0), s * (u @ v), atol=1e-13)
    x = g.standard_normal(shape)
    assert np.allclose(oracle.orthogonalize(x, eps=0.0), oracle.orthogonalize(1e9 * x, eps=0.0))
    u, _, v = np.linalg.svd(x, full_matrices=False)
    assert np.allclose(oracle.orthogonalize(x, (1.5, -0.5, 0.0), 60, 0.0), u @ v, atol=1e-12)
    assert not oracle.orthogonalize(0 * x, eps=0.0).any()


def test_oracle_is_the_iteration():
    """The singular values' image is what the products give."""
    g = np.random.default_rng(1)
    for shape in ((12, 5), (5, 12), (7, 7)):
        x = g.standard_normal(shape)
        want = oracle.orthogonalize(x, steps=4, eps=0.25)
        x = x / (np.linalg.norm(x) + 0.25)
        for _ in range(4):
            a = x @ x.T
            x = 3.4445 * x - 4.7750 * a @ x + 2.0315 * a @ a @ x
        assert np.allclose(x, want, atol=1e-13)


def test_oracle_step():
    th, m, x = oracle.muon_step(np.ones((2, 2)), 2 * np.eye(2), np.eye(2), 0.1, 0.5, True, 0.2,
                                scale=3.0)
    assert np.allclose(m, 2.5 * np.eye(2))
    assert np.allclose(x, oracle.orthogonalize(3.25 * np.eye(2)))
    assert np.allclose(th, 1 - 0.1 * (3 * x + 0.2))
