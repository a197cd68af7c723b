"""Refusals and host-side planning of the objectives and the dropout (no GPU):
the documented status comes back before any pointer is touched."""

import ctypes
import math

import pytest

from quantized_rank_fine_amd import qlora as q

P = 0x10000          # aligned for every element
BAD = P + 1          # no element but a byte


@pytest.fixture(scope="module")
def L():
    return q.lib()


def _swap(args, **change):
    return [change.get(k, v) for k, v in args.items()]


def _null_and_align(f, args, required, optional, align):
    """Every required pointer refuses NULL; every pointer refuses BAD."""
    for k in required:
        assert f(*_swap(args, **{k: None})) == 1, k
    for k in required + optional:
        if k in align:
            assert f(*_swap(args, **{k: BAD})) == 3, k


def test_token_logp_refusals(L):
    a = dict(x=P, ld=100, T=4, V=100, dt=q.BF16, y=P, s=1.0, lp=P, st=P, ent=P, ws=P, n=1 << 20,
             stream=None)
    f = L.qlora_token_logp_fwd
    for bad in (dict(V=0), dict(V=(1 << 24) + 1, ld=1 << 25), dict(T=-1), dict(T=(1 << 24) + 1),
                dict(ld=99), dict(ld=(1 << 32) + 1)):
        assert f(*_swap(a, **bad)) == 2, bad
    assert f(*_swap(a, dt=2)) == 4
    for s in (0.0, -1.0, math.inf, math.nan):
        assert f(*_swap(a, s=s)) == 7
    assert f(*_swap(a, T=0, x=None, y=None, lp=None, st=None)) == 0
    _null_and_align(f, a, ["x", "y", "lp", "st"], ["ent"], {"x", "y", "lp", "st", "ent"})
    assert f(*_swap(a, x=P + 2, dt=q.F32)) == 3
    assert q.qlora_token_logp_workspace_bytes(4, 0, q.BF16) == 0
    b = dict(x=P, ld=100, T=4, V=100, dt=q.F32, y=P, s=1.0, st=P, ent=P, g=P, ge=P, dx=P, ldd=100,
             stream=None)
    f = L.qlora_token_logp_bwd
    for bad in (dict(V=0), dict(T=-1), dict(ld=99), dict(ldd=99), dict(ldd=(1 << 32) + 1)):
        assert f(*_swap(b, **bad)) == 2, bad
    assert f(*_swap(b, dt=-1)) == 4
    assert f(*_swap(b, s=0.0)) == 7
    assert f(*_swap(b, T=0)) == 0
    _null_and_align(f, b, ["x", "y", "st", "g", "dx", "ent", "ge"], [],
                    {"x", "y", "st", "g", "dx", "ent", "ge"})


def test_pref_refusals(L):
    ok = q.pref_struct(q.PREF_SIGMOID, 0.1, 0.5, 0.1, True)
    ws = q.qlora_pref_workspace_bytes(2, 100)
    a = dict(lp=P, ref=P, mask=BAD, cu=P, P=2, T=100, pref=ctypes.byref(ok), loss=P, rw=P, d=P,
             ws=P, n=ws, stream=None)
    f = L.qlora_pref_loss
    for bad in (dict(P=0), dict(P=-1), dict(P=(1 << 20) + 1), dict(T=-1), dict(T=(1 << 30) + 1)):
        assert f(*_swap(a, **bad)) == 2, bad
    assert f(*_swap(a, pref=None)) == 1
    for v in ((3, 0.1), (-1, 0.1), (0, 0.0), (0, -0.1), (0, math.inf), (0, math.nan),
              (0, 0.1, math.nan), (0, 0.1, math.inf), (0, 0.1, 0.0, 0.6), (0, 0.1, 0.0, -0.1)):
        assert f(*_swap(a, pref=ctypes.byref(q.pref_struct(*v)))) == 7, v
    _null_and_align(f, a, ["lp", "cu", "loss", "rw", "d"], ["ref"],
                    {"lp", "ref", "cu", "loss", "rw", "d"})
    if ws:
        assert f(*_swap(a, n=ws - 1)) == 5
        assert f(*_swap(a, ws=None)) == 1
    assert q.qlora_pref_workspace_bytes(0, 100) == 0
    assert q.qlora_pref_workspace_bytes(2, -1) == 0


def test_policy_refusals(L):
    ok = q.policy_struct(q.OBJ_CLIP, 0.2, 0.3, 3.0, 0.1, 0.01)
    T = 100000
    ws = q.qlora_policy_workspace_bytes(T)
    assert ws > 0 and q.qlora_policy_workspace_bytes(-1) == 0
    a = dict(lp=P, ent=P, T=T, w=P, adv=P, old=P, ref=P, pol=ctypes.byref(ok), out=P, d=P, dh=P,
             ws=P, n=ws, stream=None)
    f = L.qlora_policy_loss
    bad_values = ((2,), (-1,), (1, -0.1), (1, 1.1), (1, 0.2, -0.1), (1, 0.2, math.nan),
                  (1, 0.2, 0.2, 1.0), (1, 0.2, 0.2, 0.5), (1, 0.2, 0.2, math.inf),
                  (1, 0.2, 0.2, 0.0, math.nan), (1, 0.2, 0.2, 0.0, 0.0, math.inf))
    assert f(*_swap(a, T=-1)) == 2 and f(*_swap(a, T=(1 << 30) + 1)) == 2
    assert f(*_swap(a, pol=None)) == 1
    for v in bad_values:
        assert f(*_swap(a, pol=ctypes.byref(q.policy_struct(*v)))) == 7, v
    _null_and_align(f, a, ["lp", "out", "d"], ["ent", "w", "adv", "old", "ref", "dh"],
                    {"lp", "out", "d", "ent", "w", "adv", "old", "ref", "dh"})
    assert f(*_swap(a, n=ws - 1)) == 5
    assert f(*_swap(a, ws=None)) == 1
    wl = q.qlora_policy_logits_workspace_bytes(4, 100, q.BF16)
    b = dict(x=P, ld=100, T=4, V=100, dt=q.BF16, y=P, s=1.0, w=P, adv=P, old=P, ref=P,
             pol=ctypes.byref(ok), out=P, lp=P, dx=P, ldd=100, ws=P, n=wl, stream=None)
    f = L.qlora_policy_logits
    for bad in (dict(V=0), dict(T=-1), dict(ld=99), dict(ldd=99), dict(T=(1 << 24) + 1)):
        assert f(*_swap(b, **bad)) == 2, bad
    assert f(*_swap(b, dt=3)) == 4
    assert f(*_swap(b, s=math.nan)) == 7
    assert f(*_swap(b, pol=None)) == 1
    for v in bad_values:
        assert f(*_swap(b, pol=ctypes.byref(q.policy_struct(*v)))) == 7, v
    _null_and_align(f, b, ["x", "y", "out", "dx", "ws"], ["w", "adv", "old", "ref", "lp"],
                    {"x", "y", "out", "dx", "w", "adv", "old", "ref", "lp"})
    assert wl > 0 and f(*_swap(b, n=wl - 1)) == 5
    assert q.qlora_policy_logits_workspace_bytes(4, 0, q.BF16) == 0


def test_dropout_refusals(L):
    a = dict(x=P, ldx=64, r=P, ldr=64, rows=4, cols=64, dt=q.BF16, p=0.1, seed=1, ctr=2, y=P,
             ldy=64, stream=None)
    f = L.qlora_dropout
    for bad in (dict(rows=-1), dict(cols=-1), dict(rows=1 << 31), dict(cols=1 << 31), dict(ldx=63),
                dict(ldr=63), dict(ldy=63), dict(ldx=(1 << 32) + 1), dict(ldy=(1 << 32) + 1)):
        assert f(*_swap(a, **bad)) == 2, bad
    assert f(*_swap(a, dt=5)) == 4
    for p in (-0.1, 1.0, 1.5, math.nan):
        assert f(*_swap(a, p=p)) == 7, p
    assert f(*_swap(a, rows=0, x=None, y=None)) == 0
    assert f(*_swap(a, cols=0)) == 0
    _null_and_align(f, a, ["x", "y"], ["r"], {"x", "y", "r"})
    assert f(*_swap(a, dt=q.F32, x=P + 2)) == 3


def test_binding_raises(L):
    with pytest.raises(q.QloraError) as e:
        q.qlora_dropout(P, 64, None, 0, 4, 64, q.BF16, 1.0, 0, 0, P, 64, stream=0)
    assert e.value.status == 7
