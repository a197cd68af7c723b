"""GPU parity of the objectives (token log-probabilities, preference loss,
policy loss) against the float64 oracle.

Tolerances are worst cases of fp32 arithmetic, u = 2^-24 being half an ulp of
1: a sum over V words is at most V / 64 additions in a lane and a few joins
(so (V / 64 + 64) u of itself, which also covers the rounding of the exponents,
weighted by their e), a bf16 result 2^-8 of itself."""

import math

import numpy as np
import pytest

from oracle import objective as ob
from quantized_rank_fine_amd import qlora as q

from gpu_harness import out_to_f64, say, torch_dev

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
f32 = lambda v: float(np.float32(v))  # noqa: E731


def _dev(a):
    torch, dev = torch_dev()
    return None if a is None else torch.from_numpy(np.ascontiguousarray(a)).to(dev)


def _rows(T, V, ld, dt, seed, at=0, big=2.5):
    """Logits [T, V] as a view `at` elements into a buffer of rows of ld, and
    their values in float64."""
    torch, dev = torch_dev()
    g = np.random.default_rng(seed)
    tdt = torch.bfloat16 if dt == "bf16" else torch.float32
    v = (g.standard_normal(at + T * ld) * big).astype(np.float32)
    buf = torch.from_numpy(v).to(tdt).to(dev)
    x = buf[at:].view(T, ld)[:, :V]
    return x, out_to_f64(x.contiguous(), dt).reshape(T, V)


def _fwd(x, ld, dt, labels, s, entropy=True, stream=None):
    torch, dev = torch_dev()
    T, V = x.shape
    qd = q.BF16 if dt == "bf16" else q.F32
    lp = torch.full((T,), 7.0, device=dev)
    st = torch.full((T, 2), 7.0, device=dev)
    h = torch.full((T,), 7.0, device=dev) if entropy else None
    n = q.qlora_token_logp_workspace_bytes(T, V, qd)
    ws = torch.empty(n, dtype=torch.uint8, device=dev) if n else None
    q.qlora_token_logp_fwd(x, ld, T, V, qd, labels, s, lp, st, h, ws, n, stream=stream)
    return lp, st, h


def _tol_rows(V, lp, z):
    """Bounds of logp, z and H."""
    e = (V / 64 + 64) * U
    zt = e + 2 * U * np.abs(z)
    return zt + 3 * U * np.abs(lp), zt, e * (2 + 2 * np.abs(z))


def _tol_grad(x, labels, d, g, gh, s, gerr=0.0):
    """Bound of the gradient d of the coefficients g, gh (g known to gerr)."""
    V = x.shape[1]
    lp, m, z, h = ob.token_logp(x, labels, s)
    with np.errstate(all="ignore"):
        l = s * (x - m[:, None]) - z[:, None]
    l = np.where(np.isfinite(l), l, 0.0)
    p = np.where(np.isfinite(x), np.exp(l), 0.0)
    _, zt, ht = _tol_rows(V, lp, z)
    rel = zt[:, None] + (3 * np.abs(l) + 4) * U
    hot = np.zeros_like(p)
    ok = (np.asarray(labels) >= 0) & (np.asarray(labels) < V)
    hot[ok, np.asarray(labels)[ok]] = 1.0
    G, H = np.abs(g)[:, None], np.abs(gh)[:, None]
    t = G * (p * rel + 3 * U * (hot + p)) + np.broadcast_to(gerr, g.shape)[:, None] * (hot + p)
    size = np.abs(l) + h[:, None]
    t = t + H * p * (rel * (size + 1) + ht[:, None] + 4 * U * size)
    return s * t + 2 * U * np.abs(d) + 1e-36


SHAPES = [  # T, V, ld, dt, s, elements before the first row
    (1, 1, 1, "f32", 1.0, 0), (3, 7, 7, "bf16", 1.0, 1), (2, 8, 8, "bf16", 0.7, 0),
    (5, 63, 65, "f32", 1.25, 3), (4, 2047, 2047, "bf16", 1.0, 5), (3, 2049, 2056, "f32", 2.0, 0),
    (70, 1000, 1000, "bf16", 1.0, 0), (2, 4096, 4097, "bf16", 1.0, 0),
    (6, 32000, 32000, "bf16", 1.0, 0), (2, 50001, 50016, "f32", 1.25, 1),
    (3, 131077, 131077, "bf16", 1.0, 0), (1, 300007, 300007, "f32", 1.0, 0),
    (66, 70003, 70003, "bf16", 1.0, 0),          # more rows than are cut into segments
]


@pytest.mark.parametrize("T,V,ld,dt,s,at", SHAPES)
@pytest.mark.parametrize("ent", [True, False])
def test_logp_forward_and_gradient(T, V, ld, dt, s, at, ent):
    torch, dev = torch_dev()
    say(f"[logp] T={T} V={V} ld={ld} {dt} s={s} at={at} entropy={ent}")
    s = f32(s)
    g = np.random.default_rng(V)
    x, xv = _rows(T, V, ld, dt, V + T, at)
    y = g.integers(0, V, T)
    if T > 3:
        y[1], y[2] = -100, V                       # not scored
    lp, st, h = _fwd(x, ld, dt, _dev(y), s, ent)
    rl, rm, rz, rh = ob.token_logp(xv, y, s)
    tl, tz, th = _tol_rows(V, rl, rz)
    ok = (y >= 0) & (y < V)
    glp, gst = lp.cpu().numpy(), st.cpu().numpy()
    assert np.array_equal(gst[:, 0], rm.astype(np.float32))
    assert np.all(np.abs(gst[:, 1] - rz) <= tz) and np.all(np.abs(glp - rl) <= tl)
    assert np.all(glp[~ok] == 0) and np.all(gst[~ok] == 0)
    if ent:
        assert np.all(np.abs(h.cpu().numpy() - rh) <= th)
    # the gradient into rows of another length, nothing written past V
    cg, ch = g.standard_normal(T).astype(np.float32), g.standard_normal(T).astype(np.float32)
    if T > 4:
        cg[4] = 0.0
    ldd = V + 5
    buf = torch.full((T * ldd + 8,), 3.0, dtype=x.dtype, device=dev)
    dx = buf[1:]
    q.qlora_token_logp_bwd(x, ld, T, V, q.BF16 if dt == "bf16" else q.F32, _dev(y), s, st,
                           h if ent else None, _dev(cg), _dev(ch) if ent else None, dx, ldd)
    torch.cuda.synchronize()
    got = out_to_f64(buf, dt)
    rows = got[1:1 + T * ldd].reshape(T, ldd)
    assert got[0] == 3.0 and np.all(rows[:, V:] == 3.0) and np.all(got[1 + T * ldd:] == 3.0)
    gh = ch.astype(np.float64) if ent else np.zeros(T)
    ref = ob.logits_grad(xv, y, cg.astype(np.float64), gh, s)
    tol = _tol_grad(xv, y, ref, cg.astype(np.float64), gh, s)
    if dt == "bf16":
        tol = tol + 2.0 ** -8 * (np.abs(ref) + tol)
    assert np.all(np.abs(rows[:, :V] - ref) <= tol)
    assert np.all(rows[~ok, :V] == 0)


def _special(V):
    """Rows with masked, infinite, lowest and NaN logits; labels; what each
    row is."""
    g = np.random.default_rng(5)
    low = float(np.float32(-3.3895314e38))             # bf16's lowest value
    base = (g.standard_normal((9, V)) * 2).astype(np.float32)
    x, y = base.copy(), np.full(9, 3)
    x[0, V // 2:] = -np.inf                            # masked words
    x[1] = -np.inf                                     # nothing possible
    x[2] = low                                         # all at the lowest value: uniform
    x[3, :] = low
    x[3, 3] = 1.0                                      # one word left
    x[4, 3] = -np.inf                                  # the label itself is masked
    x[5, V - 1] = np.nan
    x[6, 1] = np.inf
    x[7] = np.nan
    x[8, :] = -np.inf
    x[8, 3] = -5.0                                     # one possible word
    return x, y


@pytest.mark.parametrize("V", [13, 4100, 70001])
@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_logp_special_rows(V, dt):
    torch, dev = torch_dev()
    say(f"[logp special] V={V} {dt}")
    xs, y = _special(V)
    T = len(y)
    x = _dev(xs).to(torch.bfloat16 if dt == "bf16" else torch.float32)
    xv = out_to_f64(x, dt).reshape(T, V)
    lp, st, h = _fwd(x, V, dt, _dev(y), 1.5)
    rl, rm, rz, rh = ob.token_logp(xv, y, 1.5)
    assert rl[4] == -np.inf and rl[1] == -np.inf and abs(rl[3]) == 0
    tl, tz, th = _tol_rows(V, np.where(np.isfinite(rl), rl, 0), np.where(np.isfinite(rz), rz, 0))
    for got, ref, tol in ((lp, rl, tl), (st[:, 0], rm, 0 * tl), (st[:, 1], rz, tz), (h, rh, th)):
        v = got.cpu().numpy().astype(np.float64)
        assert np.array_equal(np.isnan(v), np.isnan(ref))
        assert np.array_equal(v[np.isinf(ref)], ref[np.isinf(ref)])
        f = np.isfinite(ref)
        assert np.all(np.abs(v[f] - ref[f]) <= tol[f] + 1e-30)
    cg, ch = np.full(T, 0.5, np.float32), np.full(T, 0.25, np.float32)
    dx = torch.empty_like(x)
    qd = q.BF16 if dt == "bf16" else q.F32
    q.qlora_token_logp_bwd(x, V, T, V, qd, _dev(y), 1.5, st, h, _dev(cg), _dev(ch), dx, V)
    got = out_to_f64(dx, dt).reshape(T, V)
    ref = ob.logits_grad(xv, y, cg.astype(np.float64), ch.astype(np.float64), 1.5)
    for t in range(T):
        if t in (5, 6, 7):
            assert np.isnan(got[t]).all()
            continue
        tol = _tol_grad(xv[t:t + 1], y[t:t + 1], ref[t:t + 1], cg[t:t + 1].astype(float),
                        ch[t:t + 1].astype(float), 1.5)[0]
        tol = tol + (2.0 ** -8 * np.abs(ref[t]) if dt == "bf16" else 0)
        assert np.all(np.abs(got[t] - ref[t]) <= tol), t
    assert np.all(got[1] == 0)
    # the fused objective on the same rows: no finite row is touched by another
    out, l2, d2, _ = _policy_logits(x, V, dt, y, 1.5, q.policy_struct(q.OBJ_NLL),
                                    np.full(T, 1.0 / T, np.float32))
    got = out_to_f64(d2, dt).reshape(T, V)
    ref = ob.logits_grad(xv, y, np.full(T, -1.0 / T), np.zeros(T), 1.5)
    assert np.all(got[1] == 0) and np.isnan(got[5]).all() and np.isnan(got[7]).all()
    for t in (0, 2, 3, 4, 8):
        tol = _tol_grad(xv[t:t + 1], y[t:t + 1], ref[t:t + 1], np.array([1.0 / T]), np.zeros(1),
                        1.5)[0] + 2.0 ** -23 / T
        tol = tol + (2.0 ** -8 * np.abs(ref[t]) if dt == "bf16" else 0)
        assert np.all(np.abs(got[t] - ref[t]) <= tol), t


def test_logp_gradient_in_place_far_into_memory():
    """Offsets past 2^32 elements (and 2^33 bytes), the gradient replacing
    the logits: rows near the start, the middle and the end."""
    torch, dev = torch_dev()
    T, V, ld = 66000, 65, 65600
    say(f"[logp far] T={T} V={V} ld={ld}")
    x = torch.zeros(T * ld, dtype=torch.bfloat16, device=dev).view(T, ld)
    some = [0, 1, 32767, 65471, T - 2, T - 1]
    vals = torch.from_numpy(np.random.default_rng(8).standard_normal((6, V)).astype(np.float32))
    for r, v in zip(some, vals):
        x[r, :V] = v.to(torch.bfloat16).to(dev)
    xv = np.stack([out_to_f64(x[r, :V].contiguous(), "bf16") for r in some])
    y = torch.arange(T, device=dev) % V
    ys = [r % V for r in some]
    lp, st, h = _fwd(x[:, :V], ld, "bf16", y, 1.0)
    rl, _, rz, _ = ob.token_logp(xv, ys)
    assert np.all(np.abs(lp[some].cpu().numpy() - rl) <= _tol_rows(V, rl, rz)[0])
    g = torch.ones(T, device=dev)
    q.qlora_token_logp_bwd(x, ld, T, V, q.BF16, y, 1.0, st, None, g, None, x, ld)
    ref = ob.logits_grad(xv, ys, np.ones(6), np.zeros(6))
    got = np.stack([out_to_f64(x[r, :V].contiguous(), "bf16") for r in some])
    tol = _tol_grad(xv, ys, ref, np.ones(6), np.zeros(6), 1.0)
    assert np.all(np.abs(got - ref) <= tol + 2.0 ** -8 * np.abs(ref))
    assert not x[T - 1, V:].any() and not x[T - 2, V:].any()


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_more_rows_than_a_grid_dimension(dt):
    """70000 rows of 9 words: every row's gradient, of the logits and of the
    policy objective, against the formula (float64, all rows at once)."""
    torch, dev = torch_dev()
    T, V = 70000, 9
    x, xv = _rows(T, V, V, dt, 12)
    g = np.random.default_rng(13)
    y, c = g.integers(0, V, T), g.standard_normal(T).astype(np.float32)
    lp, st, _ = _fwd(x, V, dt, _dev(y), 1.0)
    e = np.exp(xv - xv.max(1, keepdims=True))
    z = np.log(e.sum(1))
    rl = xv[np.arange(T), y] - xv.max(1) - z
    assert np.all(np.abs(lp.cpu().numpy() - rl) <= _tol_rows(V, rl, z)[0])
    p = e / e.sum(1, keepdims=True)
    hot = np.eye(V)[y]
    ref = c[:, None] * (hot - p)
    tol = np.abs(c)[:, None] * (p * 120 * U + 4 * U) + (2.0 ** -8 * np.abs(ref)
                                                       if dt == "bf16" else 0)
    dx = torch.empty_like(x)
    q.qlora_token_logp_bwd(x, V, T, V, q.BF16 if dt == "bf16" else q.F32, _dev(y), 1.0, st, None,
                           _dev(c), None, dx, V)
    assert np.all(np.abs(out_to_f64(dx, dt).reshape(T, V) - ref) <= tol)
    out, _, d2, _ = _policy_logits(x, V, dt, y, 1.0, q.policy_struct(q.OBJ_NLL), -c)
    assert np.all(np.abs(out_to_f64(d2, dt).reshape(T, V) - ref) <= tol)
    want = (c * rl).sum()
    assert abs(out[0] - want) <= 2 * U * (np.abs(want) + (np.abs(c) * (np.abs(rl) + 100)).sum())


@pytest.mark.parametrize("V", [40, 70001])
def test_rows_without_a_gradient_are_not_read(V):
    """A coefficient of 0: a row of zeros, whatever its logits hold (prompt
    tokens under a mask), out of place and in place."""
    torch, dev = torch_dev()
    x, _ = _rows(3, V, V, "bf16", 21)
    y = np.array([1, 2, 3])
    _, st, h = _fwd(x, V, "bf16", _dev(y), 1.0)
    x[1] = float("nan")
    dx = torch.full_like(x, 7.0)
    g = torch.tensor([1.0, 0.0, -1.0], device=dev)
    q.qlora_token_logp_bwd(x, V, 3, V, q.BF16, _dev(y), 1.0, st, None, g, None, dx, V)
    assert not dx[1].any() and bool(torch.isfinite(dx).all()) and dx[0].any() and dx[2].any()
    keep = dx.clone()
    q.qlora_token_logp_bwd(x, V, 3, V, q.BF16, _dev(y), 1.0, st, None, g, None, x, V)
    assert torch.equal(x, keep)


# ------------------------------------------------------------ policy loss

def _policy_inputs(T, seed, dual=0.0, lo=0.2, hi=0.28):
    """logp, entropy, weight, adv, old, ref (fp32); log-ratios away from the
    places where a bound begins to hold."""
    g = np.random.default_rng(seed)
    lp = -np.abs(g.standard_normal(T) * 1.5).astype(np.float32)
    d = g.standard_normal(T) * np.where(g.random(T) < 0.2, 1.0, 0.2)
    for e in [math.log1p(-lo), math.log1p(hi)] + ([math.log(dual)] if dual else []):
        d = np.where(np.abs(d - e) < 1e-3, d + 2e-3, d)
    w = (g.random(T) * (g.random(T) > 0.2) / T).astype(np.float32)
    return dict(logp=lp, entropy=(1 + g.random(T)).astype(np.float32), weight=w,
                adv=g.standard_normal(T).astype(np.float32), old=(lp - d).astype(np.float32),
                ref=(lp + g.standard_normal(T) * 0.5).astype(np.float32))


def _token_tol(c, kl, ent, lperr=0.0):
    """Per token: bounds of the loss and of dlogp before the weight, when
    logp is known to lperr."""
    one = np.ones(len(c["logp"]))
    a = np.abs(c["adv"].astype(float)) if c["adv"] is not None else one
    lp = c["logp"].astype(float)
    d = np.zeros_like(lp) if c["old"] is None else lp - c["old"]
    r = np.exp(d)
    k = np.zeros_like(lp) if c["ref"] is None else c["ref"] - lp
    h = 0 * one if c["entropy"] is None else np.abs(c["entropy"])
    slope = a * (r + np.abs(lp)) + abs(kl) * (np.exp(k) + 1)
    t = 8 * U * (a * (r + 1.4) * (1 + np.abs(d)) + a * np.abs(lp)
                 + abs(kl) * (np.exp(k) + 1 + np.abs(k)) * (1 + np.abs(k)) + abs(ent) * h)
    return t + (slope + a) * lperr, t + slope * lperr, 8 * U * (np.exp(k) + 1 + np.abs(k)) + \
        (np.exp(k) + 1) * lperr


CASES = [  # kind, dual, kl, ent, inputs left out
    ("clip", 0.0, 0.1, 0.0, ()), ("clip", 3.0, 0.04, 0.01, ()), ("clip", 1.2, 0.0, 0.02, ("ref",)),
    ("nll", 0.0, 0.1, 0.0, ("old",)), ("nll", 0.0, 0.0, 0.0, ("adv", "old", "ref", "entropy")),
    ("clip", 0.0, 0.1, 0.0, ("old", "weight", "entropy")), ("clip", 3.0, 0.1, 0.0, ("adv",)),
]


@pytest.mark.parametrize("T", [0, 1, 63, 1000, 4096, 4097, 70001])
@pytest.mark.parametrize("kind,dual,kl,ent,none", CASES)
def test_policy_loss(T, kind, dual, kl, ent, none):
    torch, dev = torch_dev()
    say(f"[policy] T={T} {kind} dual={dual} without {none}")
    c = _policy_inputs(T, T + 3, dual)
    for k in none:
        c[k] = None
    lo, hi, kl, ent, dual = f32(0.2), f32(0.28), f32(kl), f32(ent), f32(dual)
    ref_out, rg, rh = ob.policy_loss(kind, *[c[k] for k in ("logp", "entropy", "weight", "adv",
                                                            "old", "ref")], lo, hi, dual, kl, ent)
    if c["weight"] is not None:                # what a token of no weight holds is not read
        off = c["weight"] == 0
        for k in ("logp", "entropy", "adv", "old", "ref"):
            if c[k] is not None:
                c[k] = np.where(off, np.float32(np.nan), c[k])
    t = {k: _dev(v) for k, v in c.items()}
    # entered one token into larger arrays: 4-byte alignment only
    t = {k: None if v is None else torch.cat([v.new_zeros(1), v])[1:] for k, v in t.items()}
    pol = q.policy_struct(q.OBJ_CLIP if kind == "clip" else q.OBJ_NLL, lo, hi, dual, kl, ent)
    out = torch.full((4,), 9.0, device=dev)
    d = torch.full((T + 2,), 9.0, device=dev)
    dh = torch.full((T + 2,), 9.0, device=dev) if c["entropy"] is not None else None
    n = q.qlora_policy_workspace_bytes(T)
    ws = torch.empty(n, dtype=torch.uint8, device=dev) if n else None
    q.qlora_policy_loss(t["logp"], t["entropy"], T, t["weight"], t["adv"], t["old"], t["ref"], pol,
                        out, d[1:], None if dh is None else dh[1:], ws, n)
    got, go = d.cpu().numpy().astype(float), out.cpu().numpy().astype(float)
    assert got[0] == 9.0 and got[-1] == 9.0
    w = np.ones(T) if c["weight"] is None else c["weight"].astype(float)
    clean = {k: None if v is None else np.nan_to_num(v) for k, v in c.items()}
    tl, tg, tk = _token_tol(clean, kl, ent)
    assert np.all(np.abs(got[1:-1] - rg) <= w * tg + 2 * U * np.abs(rg))
    if dh is not None:
        assert np.all(np.abs(dh.cpu().numpy()[1:-1] - rh) <= 2 * U * np.abs(rh))
    absum = np.array([(w * tl).sum(), (w * tk).sum(), 0.0, 0.0])
    assert np.all(np.abs(go - ref_out) <= absum + 2 * U * (np.abs(ref_out) + w.sum()))


def _policy_logits(x, ld, dt, y, s, pol, w, adv=None, old=None, ref=None, inplace=False):
    torch, dev = torch_dev()
    T, V = x.shape
    qd = q.BF16 if dt == "bf16" else q.F32
    out, lp = torch.full((4,), 9.0, device=dev), torch.full((T,), 9.0, device=dev)
    dx = x if inplace else torch.empty(T, V, dtype=x.dtype, device=dev)
    ldd = ld if inplace else V
    n = q.qlora_policy_logits_workspace_bytes(T, V, qd)
    ws = torch.empty(n, dtype=torch.uint8, device=dev)
    args = (x, ld, T, V, qd, _dev(y), s, _dev(w), _dev(adv), _dev(old), _dev(ref), pol)
    q.qlora_policy_logits(*args, out, lp, dx, ldd, ws, n)
    torch.cuda.synchronize()
    return out.cpu().numpy().astype(float), lp.cpu().numpy().astype(float), dx, args


@pytest.mark.parametrize("T,V,ld,dt,s,at", SHAPES)
@pytest.mark.parametrize("kind,ent", [("clip", 0.02), ("nll", 0.0)])
def test_policy_logits(T, V, ld, dt, s, at, kind, ent):
    torch, dev = torch_dev()
    say(f"[policy logits] T={T} V={V} ld={ld} {dt} s={s} at={at} {kind}")
    s, lo, hi, kl, ent = f32(s), f32(0.2), f32(0.28), f32(0.1), f32(ent)
    g = np.random.default_rng(V + 1)
    x, xv = _rows(T, V, ld, dt, V + T + 1, at)
    y = g.integers(0, V, T)
    lp, m, z, h = ob.token_logp(xv, y, s)
    c = _policy_inputs(T, V, 0.0)
    w = (0.25 + g.random(T)).astype(np.float32) / T
    if T > 4:
        y[1], y[2], w[3] = -100, V, 0.0
    d = c["logp"] - c["old"].astype(float)
    old, ref = (lp - d).astype(np.float32), (lp + (c["ref"] - c["logp"])).astype(np.float32)
    adv = c["adv"]
    if kind == "nll":
        adv = old = ref = None
    on = (y >= 0) & (y < V) & (w != 0)
    weight = w * on
    ro, rg, rgh = ob.policy_loss(kind, lp, h, weight, adv, old, ref, lo, hi, 0.0, kl, ent)
    rd = ob.logits_grad(xv, np.where(on, y, -1), rg, rgh, s)
    pol = q.policy_struct(q.OBJ_CLIP if kind == "clip" else q.OBJ_NLL, lo, hi, 0.0, kl, ent)
    out, glp, dx, _ = _policy_logits(x, ld, dt, y, s, pol, w, adv, old, ref)
    tl, tz, th = _tol_rows(V, lp, z)
    assert np.all(np.abs(glp - lp * on) <= tl * on)
    inputs = dict(logp=lp, entropy=h, adv=adv, old=old, ref=ref)
    tloss, tg, tk = _token_tol(inputs, kl, ent, tl)
    gerr = weight * tg + 2 * U * np.abs(rg)
    tol = _tol_grad(xv, np.where(on, y, -1), rd, rg, rgh, s, gerr)
    if dt == "bf16":
        tol = tol + 2.0 ** -8 * (np.abs(rd) + tol)
    got = out_to_f64(dx, dt).reshape(T, V)
    assert np.all(np.abs(got - rd) <= tol)
    assert np.all(got[~on] == 0)
    absum = np.array([(weight * (tloss + abs(ent) * th)).sum(), (weight * tk).sum(), 0.0,
                      (weight * th).sum()])
    # the sums themselves: each token's term rounded to fp32, added in fp64
    terms = weight.sum() * (4 + np.abs(ro).max() / max(weight.sum(), 1e-30)) + \
        (weight * (np.abs(lp) + h)).sum()
    assert np.all(np.abs(out - ro) <= absum + 4 * U * terms)
    # the same bits again, and in place
    out2, lp2, dx2, _ = _policy_logits(x, ld, dt, y, s, pol, w, adv, old, ref, inplace=True)
    assert np.array_equal(out, out2) and np.array_equal(glp, lp2)
    assert np.array_equal(out_to_f64(dx2.contiguous(), dt).reshape(T, V), got)


@pytest.mark.parametrize("V", [50, 70001])
def test_policy_logits_of_nothing(V):
    """No tokens, and tokens of which none is scored or weighted: zeros."""
    torch, dev = torch_dev()
    pol = q.policy_struct(q.OBJ_CLIP, kl_coef=0.1, ent_coef=0.1)
    out = torch.full((4,), 9.0, device=dev)
    q.qlora_policy_logits(None, V, 0, V, q.BF16, None, 1.0, None, None, None, None, pol, out, None,
                          None, V, None, 0)
    assert not out.any()
    x, _ = _rows(4, V, V, "f32", 3)
    x[:] = float("nan")
    y, w = np.array([-100, V, 0, 5]), np.array([1, 1, 0, 0], np.float32)
    out, lp, dx, _ = _policy_logits(x, V, "f32", y, 1.0, pol, w, adv=np.full(4, np.nan, np.float32))
    assert not out.any() and not lp.any() and not dx.any()
    lp, st, h = _fwd(x[:2].contiguous(), V, "f32", _dev(y[:2]), 1.0)
    assert not lp.any() and not st.any() and not h.any()


def test_policy_logits_gradient_is_the_difference_quotient():
    """Against central differences of the oracle's loss (float64), by logit."""
    T, V = 3, 11
    x, xv = _rows(T, V, V, "f32", 77)
    y, w = np.array([2, 5, 10]), np.array([0.5, 0.25, 0.25], np.float32)
    adv = np.array([1.0, -2.0, 0.5], np.float32)
    old = ref = (ob.token_logp(xv, y)[0] + np.array([0.05, -0.1, 0.02])).astype(np.float32)
    pol = q.policy_struct(q.OBJ_CLIP, 0.2, 0.2, 0.0, 0.5, 0.125)
    _, _, dx, _ = _policy_logits(x, V, "f32", y, 1.0, pol, w, adv, old, ref)

    def loss(v):
        lp, _, _, h = ob.token_logp(v, y)
        return ob.policy_loss("clip", lp, h, w, adv, old, ref, f32(0.2), f32(0.2), 0.0, 0.5,
                              0.125)[0][0]

    got = dx.cpu().numpy().astype(float)
    eps = 1e-5
    for i in np.ndindex(T, V):
        a, b = xv.copy(), xv.copy()
        a[i] += eps
        b[i] -= eps
        # the quotient's own error: eps^2 times a third derivative of order 10
        assert abs(got[i] - (loss(a) - loss(b)) / (2 * eps)) <= 1e-8 + 200 * U


# -------------------------------------------------------- preference loss

def _pref(lp, ref, mask, cu, pref):
    torch, dev = torch_dev()
    T, P = len(lp), (len(cu) - 1) // 2
    loss, rw = torch.full((1,), 9.0, device=dev), torch.full((2 * P,), 9.0, device=dev)
    d = torch.full((T + 2,), 9.0, device=dev)
    n = q.qlora_pref_workspace_bytes(P, T)
    ws = torch.full((n,), 255, dtype=torch.uint8, device=dev) if n else None
    pad = lambda a, z: None if a is None else torch.cat([z, _dev(a)])[1:]  # noqa: E731
    z4, z1 = torch.zeros(1, device=dev), torch.zeros(1, dtype=torch.uint8, device=dev)
    q.qlora_pref_loss(pad(lp, z4), pad(ref, z4), pad(mask, z1), _dev(np.asarray(cu, np.int64)), P,
                      T, pref, loss, rw, d[1:], ws, n)
    got = d.cpu().numpy().astype(float)
    assert got[0] == 9.0 and got[-1] == 9.0
    return float(loss), rw.cpu().numpy().astype(float), got[1:-1]


PREF_KINDS = {"sigmoid": q.PREF_SIGMOID, "squared": q.PREF_SQUARED, "hinge": q.PREF_HINGE}
LENGTHS = {
    "one token": [1, 1], "empty": [0, 0], "half empty": [5, 0, 0, 7],
    "short": [3, 1, 64, 65, 200, 17], "many": list(range(0, 200)),
    "long": [9001, 1, 30000, 4097], "very long": [150000, 70001],
    "pairs": [700 + 11 * i for i in range(130)], "many short": [i % 90 for i in range(700)],
    "crowd": [i % 5 for i in range(1400)],
}


@pytest.mark.parametrize("name", LENGTHS)
@pytest.mark.parametrize("kind", PREF_KINDS)
@pytest.mark.parametrize("average", [False, True])
@pytest.mark.parametrize("ref,masked", [(True, True), (False, False)])
def test_pref_loss(name, kind, average, ref, masked):
    say(f"[pref] {name} {kind} average={average} ref={ref} mask={masked}")
    g = np.random.default_rng(len(name) + 10 * average)
    lens = np.array(LENGTHS[name])
    if name in ("many", "pairs", "many short", "crowd"):
        lens = g.permutation(lens)
    before, after = (3, 5) if masked else (0, 0)        # tokens outside every answer
    cu = before + np.concatenate([[0], np.cumsum(lens)])
    T = int(cu[-1]) + after
    lp = -np.abs(g.standard_normal(T)).astype(np.float32)
    rf = (lp + 0.1 * g.standard_normal(T)).astype(np.float32) if ref else None
    mask = (g.random(T) > 0.3).astype(np.uint8) * 2 if masked else None
    if masked:
        a = int(cu[len(lens) // 2])
        mask[a:int(cu[len(lens) // 2 + 1])] = 0          # an answer without a counted token
    beta, margin, smooth = f32(0.1), f32(0.25), f32(0.05)
    rl, rr, rd = ob.pref_loss(kind, lp, rf, mask, cu, beta, margin, smooth, average)
    if masked:
        lp[mask == 0] = np.nan                           # what is masked is not read
    pref = q.pref_struct(PREF_KINDS[kind], beta, margin, smooth, average)
    loss, rw, d = _pref(lp, rf, mask, cu, pref)
    # bounds: S is a sum of fp32 differences, then rounded; h a difference of two S
    dif = np.nan_to_num(np.abs(lp - (rf if ref else 0)))
    P, tol_s, cnt = len(lens) // 2, [], []
    for i in range(2 * P):
        k = slice(int(cu[i]), int(cu[i + 1]))
        n = k.stop - k.start if mask is None else int((mask[k] != 0).sum())
        cnt.append(max(1, n) if average else 1)
        tol_s.append(2 * U * (dif[k].sum() / cnt[-1] + abs(rr[i] / beta)))
    tol_s, cnt = np.array(tol_s), np.array(cnt)
    assert np.all(np.abs(rw - rr) <= beta * tol_s + 2 * U * np.abs(rr))
    h = (rr[:P] - rr[P:]) / beta
    th = tol_s[:P] + tol_s[P:] + U * np.abs(h)
    if kind == "squared":
        e = np.abs(h - 0.5 / beta)
        et = th + U * (np.abs(h) + 10 / 2 + e)
        tl, td = et * (2 * e + et) + 4 * U * e * e, 2 * et + 4 * U * e
    else:
        u = np.abs(beta * h - margin)
        ut = beta * th + 3 * U * (np.abs(beta * h) + margin + u)
        tl, td = ut + 8 * U * (1 + u), beta * (ut + 8 * U)
        if kind == "hinge":
            assert np.all(np.abs(beta * h - margin - 1.0) > ut)      # no pair at the corner
            td = 2 * U * beta + 0 * u
    assert abs(loss - rl) <= tl.mean() + 2 * U * abs(rl)
    for i in range(2 * P):
        k = slice(int(cu[i]), int(cu[i + 1]))
        t = td[i % P] / P / cnt[i]
        assert np.all(np.abs(d[k] - rd[k]) <= t + 4 * U * np.abs(rd[k])), i
    assert np.all(d[:before] == 0) and np.all(d[T - after:] == 0)
    if masked:
        assert np.all(d[mask == 0] == 0)
    # fixed order: the same bits again
    again = _pref(lp, rf, mask, cu, pref)
    assert again[0] == loss and np.array_equal(again[1], rw) and np.array_equal(again[2], d)


def test_pref_offsets_outside_the_tokens():
    """cu past either end is taken as the end; nothing is read beyond it."""
    lp = -np.ones(10, np.float32)
    pref = q.pref_struct(q.PREF_SIGMOID, 0.5)
    loss, rw, d = _pref(lp, None, None, [-4, 6, 99], pref)
    assert np.allclose(rw, [-3.0, -2.0]) and np.all(d[:6] == d[0]) and np.all(d[6:] == -d[0])
    rl, _, rd = ob.pref_loss("sigmoid", lp, None, None, [0, 6, 10], 0.5)
    assert abs(loss - rl) <= 16 * U and np.all(np.abs(d - rd) <= 16 * U)
    # a decreasing pair is an empty answer
    _, rw, _ = _pref(lp, None, None, [0, 6, 2], pref)
    assert rw[1] == 0


def test_pref_without_tokens():
    torch, dev = torch_dev()
    loss, rw = torch.full((1,), 9.0, device=dev), torch.full((4,), 9.0, device=dev)
    n = q.qlora_pref_workspace_bytes(2, 0)
    ws = torch.empty(n, dtype=torch.uint8, device=dev) if n else None
    cu = torch.zeros(5, dtype=torch.int64, device=dev)
    q.qlora_pref_loss(None, None, None, cu, 2, 0, q.pref_struct(q.PREF_SIGMOID, 0.1), loss, rw,
                      None, ws, n)
    assert abs(float(loss) - math.log(2)) <= 4 * U and not rw.any()


# ----------------------------------------------------- graphs and streams

@pytest.mark.parametrize("T,V", [(5, 1000), (3, 40000), (3, 140001)])
def test_graph_replays_and_another_stream(T, V):
    """The whole chain (scoring, preference loss, gradient; policy loss from
    tokens and from logits) captured on a side stream: every replay gives the
    eager bits."""
    torch, dev = torch_dev()
    say(f"[objective graph] T={T} V={V}")
    x, _ = _rows(T, V, V, "bf16", 3)
    y = torch.arange(T, device=dev) * 7 % V
    cu = torch.tensor([0, 1, T], device=dev)
    e = lambda *n: torch.empty(*n, device=dev)  # noqa: E731
    lp, st, h, loss, rw, g, dx = e(T), e(T, 2), e(T), e(1), e(2), e(T), torch.empty_like(x)
    out, out2, d2, dx2, l2 = e(4), e(4), e(T), torch.empty_like(x), e(T)
    pref, pol = q.pref_struct(q.PREF_SIGMOID, 0.1), q.policy_struct(q.OBJ_CLIP, ent_coef=0.01)
    sizes = (q.qlora_token_logp_workspace_bytes(T, V, q.BF16), q.qlora_pref_workspace_bytes(1, T),
             q.qlora_policy_workspace_bytes(T), q.qlora_policy_logits_workspace_bytes(T, V, q.BF16))
    ws = [torch.empty(max(n, 16), dtype=torch.uint8, device=dev) for n in sizes]

    def step():
        q.qlora_token_logp_fwd(x, V, T, V, q.BF16, y, 1.0, lp, st, h, ws[0], sizes[0])
        q.qlora_pref_loss(lp, None, None, cu, 1, T, pref, loss, rw, g, ws[1], sizes[1])
        q.qlora_token_logp_bwd(x, V, T, V, q.BF16, y, 1.0, st, None, g, None, dx, V)
        q.qlora_policy_loss(lp, h, T, None, None, None, None, pol, out, d2, None, ws[2], sizes[2])
        q.qlora_policy_logits(x, V, T, V, q.BF16, y, 1.0, None, None, None, None, pol, out2, l2,
                              dx2, V, ws[3], sizes[3])

    outs = (lp, st, h, loss, rw, g, dx, out, out2, d2, dx2, l2)
    step()
    torch.cuda.synchronize()
    want = [t.float().cpu().numpy().copy() for t in outs]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for rep in range(3):
        for t in outs:
            t.fill_(float("nan"))
        for w in ws:
            w.fill_(255)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for k, (t, v) in enumerate(zip(outs, want)):
            assert np.array_equal(t.float().cpu().numpy(), v), (rep, k)
