"""Refusals and workspace of the linear's elementwise end (no GPU)."""

import ctypes

from quantized_rank_fine_amd import qlora as q

P = 0x10000
BAD = P + 8


def _fwd(ep="ok", lora=None, n_in=256, n_out=192, **kw):
    s = q.nf4_struct(n_in, n_out, P, P, P)
    e = q.epilogue_struct(**kw)
    o = q.qlora_lora(*lora) if lora else None
    n = q.qlora_fwd_workspace_bytes(64, 256, 192, 8)
    return q.lib().qlora_linear_fwd_ep(
        ctypes.byref(s), P, 64, q.BF16, P, P, 8, q.BF16, ctypes.byref(o) if o else None,
        ctypes.byref(e) if ep else None, None if ep == "no y" else P, P, P,
        n - (ep == "short"), None)


def test_forward_refusals():
    assert _fwd(ep=None) == 1
    for a in (-1, 5, 100):
        assert _fwd(act=a) == 7
    for k in ("bias", "mul", "residual", "Z"):
        assert _fwd(**{k: BAD}) == 3, k
    assert _fwd(lora=(float("nan"), 0.0, None)) == 7 and _fwd(lora=(1.0, 0.5, None)) == 7
    assert _fwd(n_in=100) == 2 and _fwd("no y") == 1 and _fwd("short") == 5


def test_gradient_refusals():
    f = q.lib().qlora_ep_bwd
    n = q.qlora_ep_bwd_workspace_bytes(1000, 192)
    assert n > 0
    ok = dict(Z=P, mul=P, dY=P, M=1000, out=192, act=q.BF16, ep=q.EP_SILU, dZ=P, dmul=P, db=P, ws=P,
              n=n, stream=None)
    call = lambda **kw: f(*{**ok, **kw}.values())  # noqa: E731
    for kw in (dict(M=-1), dict(M=(1 << 24) + 1), dict(out=0), dict(out=100), dict(out=(1 << 19) + 64)):
        assert call(**kw) == 2, kw
    assert call(act=2) == 4 and call(ep=5) == 7 and call(ep=-1) == 7
    assert call(dY=None) == 1 and call(Z=None) == 1 and call(mul=None) == 1
    assert call(Z=None, ep=q.EP_NONE) == 1 and call(mul=None, dmul=P) == 1
    for k in ("Z", "mul", "dY", "dZ", "dmul", "db", "ws"):
        assert call(**{k: BAD}) == 3, k
    assert call(ws=None) == 1 and call(n=n - 1) == 5
    assert call(dZ=None, dmul=None, db=None, ws=None, n=0) == 0       # nothing is wanted
    assert call(M=0, Z=None, dY=None, db=None) == 0


def test_workspace():
    w = q.qlora_ep_bwd_workspace_bytes
    assert w(64, 192) == 0 and w(65, 192) == 2 * 192 * 8              # one slab needs none
    assert w(1 << 24, 192) == 256 * 192 * 8
    assert w(0, 192) == 0 and w(-1, 192) == 0 and w(64, 100) == 0 and w(1000, 192, 7) == 0
