"""GPU parity of the row kernels where words are masked by a large finite
value: every count of wavefronts, chunks and segments to a row, scales at which
the mask's product with the inverse temperature rounds up and down.

Tolerances as in test_gpu_objective.py.  A row of nothing but the mask is
summed against c m rounded to fp32, c = s log2 e, which leaves off = c m -
round(c m), at most half an ulp: logs of sums are then up to off + log2 V, and
their roundings (one of the log, one of ln 2 times off, one of the difference)
count against that.  A p below the least normal number, 2^-126, is 0 (exp2 has
no subnormal results), which is all that is lost of it."""

import numpy as np
import pytest

from oracle import objective as ob
from quantized_rank_fine_amd import qlora as q

from gpu_harness import out_to_f64, say, torch_dev
from test_gpu_objective import (U, _dev, _fwd, _policy_logits, _special, _tol_grad, _tol_rows,
                                _token_tol, f32)

pytestmark = pytest.mark.gpu

MASKS = [-1e8, -1e9, -2e9, -1e10, -1e12, -1e15]
SCALES = [1.0, 1 / 0.6, 2.5, 5.0]
WIDTHS = [513, 4096, 12001, 40000, 70003]


def _rows(V, dt, seed):
    """Five rows to a mask: its tail, all but a scattered hundredth, all but
    three words, all words, and every second word; labels (live but in the
    fourth), and masked labels."""
    torch, dev = torch_dev()
    g = np.random.default_rng(seed)
    x = (g.standard_normal((5 * len(MASKS), V)) * 2).astype(np.float32)
    y, y_masked = np.zeros(len(x), np.int64), np.zeros(len(x), np.int64)
    for i, mask in enumerate(MASKS):
        gone = np.zeros((5, V), bool)
        gone[0, V - V // 8:] = True
        gone[1] = g.random(V) > 0.01
        gone[2] = True
        gone[2, g.integers(0, V, 3)] = False
        gone[3] = True
        gone[4, ::2] = True
        gone[1, V // 3] = gone[1, V // 2] = False
        x[5 * i:5 * i + 5][gone] = mask
        for j in range(5):
            y_masked[5 * i + j] = np.flatnonzero(gone[j])[1]
            y[5 * i + j] = 7 if j == 3 else np.flatnonzero(~gone[j])[-1]
    t = torch.from_numpy(x).to(dev).to(torch.bfloat16 if dt == "bf16" else torch.float32)
    return t, out_to_f64(t, dt).reshape(x.shape), y, y_masked


def _tols(xv, V, lp, z, s):
    """Bounds of logp, z and H."""
    tl, tz, th = _tol_rows(V, lp, z)
    cm = np.abs(s * xv.max(1)) * 1.4427
    off = np.where(cm < 2.0 ** 31, 2.0 ** (np.floor(np.log2(np.maximum(cm, 1.0))) - 24), 0.0)
    e = (V / 64 + 64) * U
    return tl + 6 * U * off, tz + 6 * U * off, th + 2 * e * off


def _lost(xv, m, z, h, g, gh, s):
    """The most that a p of less than 2^-126 is worth in the gradient."""
    l = s * (xv - m[:, None]) - z[:, None]
    l = np.where(l < -87.0, np.maximum(l, -104.0), 0.0)   # (none below 2^-150: 0 to start with)
    size = np.abs(l) + h[:, None]
    return np.where(l < 0, s * (np.abs(g)[:, None] + np.abs(gh)[:, None] * size) * 2.0 ** -126, 0.0)


@pytest.mark.parametrize("V", WIDTHS)
@pytest.mark.parametrize("s", SCALES)
@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_logp_of_rows_with_finite_masks(V, s, dt):
    say(f"[logp masks] V={V} s={s} {dt}")
    s = f32(s)
    x, xv, y, y_masked = _rows(V, dt, V)
    T, torch = len(y), torch_dev()[0]
    qd = q.BF16 if dt == "bf16" else q.F32
    for labels in (y, y_masked):
        lp, st, h = _fwd(x, V, dt, _dev(labels), s)
        rl, rm, rz, rh = ob.token_logp(xv, labels, s)
        tl, tz, th = _tols(xv, V, rl, rz, s)
        assert np.array_equal(st.cpu().numpy()[:, 0], rm.astype(np.float32))
        assert np.all(np.abs(st.cpu().numpy()[:, 1] - rz) <= tz)
        assert np.all(np.abs(lp.cpu().numpy() - rl) <= tl)
        assert np.all(np.abs(h.cpu().numpy() - rh) <= th)
        # without the entropy: the same bits
        lp2, st2, _ = _fwd(x, V, dt, _dev(labels), s, False)
        assert torch.equal(lp, lp2) and torch.equal(st, st2)
        g = np.random.default_rng(V + 1)
        cg, ch = g.standard_normal(T).astype(np.float32), g.standard_normal(T).astype(np.float32)
        dx = torch.empty_like(x)
        q.qlora_token_logp_bwd(x, V, T, V, qd, _dev(labels), s, st, h, _dev(cg), _dev(ch), dx, V)
        ref = ob.logits_grad(xv, labels, cg.astype(float), ch.astype(float), s)
        tol = _tol_grad(xv, labels, ref, cg.astype(float), ch.astype(float), s)
        # z and H to their own bounds, where those are wider
        p = np.exp(s * (xv - rm[:, None]) - rz[:, None])
        wide = (np.abs(cg) + np.abs(ch) * (1 + rz))[:, None] * p * (tz + th)[:, None]
        tol = tol + s * wide + _lost(xv, rm, rz, rh, cg, ch, s)
        if dt == "bf16":
            tol = tol + 2.0 ** -8 * (np.abs(ref) + tol)
        assert np.all(np.abs(out_to_f64(dx, dt).reshape(T, V) - ref) <= tol)


@pytest.mark.parametrize("V", WIDTHS)
@pytest.mark.parametrize("s", SCALES)
@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("ent", [0.0, 0.02])
def test_policy_of_rows_with_finite_masks(V, s, dt, ent):
    """The fused objective, with and without an entropy term: the sums, the
    scores and the gradient."""
    say(f"[policy masks] V={V} s={s} {dt} ent={ent}")
    s, ent, kl, lo, hi = f32(s), f32(ent), f32(0.1), f32(0.2), f32(0.28)
    x, xv, y, _ = _rows(V, dt, V + 2)
    T = len(y)
    lp, m, z, h = ob.token_logp(xv, y, s)
    g = np.random.default_rng(V + 3)
    w, adv = ((0.25 + g.random(T)) / T).astype(np.float32), g.standard_normal(T).astype(np.float32)
    old, ref = (lp + 0.05).astype(np.float32), (lp - 0.1).astype(np.float32)
    ro, rg, rgh = ob.policy_loss("clip", lp, h, w, adv, old, ref, lo, hi, 0.0, kl, ent)
    rd = ob.logits_grad(xv, y, rg, rgh, s)
    pol = q.policy_struct(q.OBJ_CLIP, lo, hi, 0.0, kl, ent)
    out, glp, dx, _ = _policy_logits(x, V, dt, y, s, pol, w, adv, old, ref)
    tl, tz, th = _tols(xv, V, lp, z, s)
    assert np.all(np.abs(glp - lp) <= tl)
    tloss, tg, tk = _token_tol(dict(logp=lp, entropy=h, adv=adv, old=old, ref=ref), kl, ent, tl)
    gerr = w * tg + 2 * U * np.abs(rg)
    tol = _tol_grad(xv, y, rd, rg, rgh, s, gerr)
    p = np.exp(s * (xv - m[:, None]) - z[:, None])
    tol = tol + s * (np.abs(rg) + np.abs(rgh) * (1 + z))[:, None] * p * (tz + th)[:, None]
    tol = tol + _lost(xv, m, z, h, rg, rgh, s)
    if dt == "bf16":
        tol = tol + 2.0 ** -8 * (np.abs(rd) + tol)
    assert np.all(np.abs(out_to_f64(dx, dt).reshape(T, V) - rd) <= tol)
    absum = np.array([(w * (tloss + abs(ent) * th)).sum(), (w * tk).sum(), 0.0, (w * th).sum()])
    terms = w.sum() * (4 + np.abs(ro).max() / w.sum()) + (w * (np.abs(lp) + h)).sum()
    assert np.all(np.abs(out - ro) <= absum + 4 * U * terms)
    # in place: the same bits
    out2, lp2, dx2, _ = _policy_logits(x.clone(), V, dt, y, s, pol, w, adv, old, ref, inplace=True)
    assert np.array_equal(out, out2) and np.array_equal(glp, lp2)
    assert np.array_equal(out_to_f64(dx2, dt).reshape(T, V), out_to_f64(dx, dt).reshape(T, V))


@pytest.mark.parametrize("V", [13, 4100, 12001, 70001])
@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("kind,ent", [("clip", 0.02), ("clip", 0.0), ("nll", 0.02)])
def test_policy_of_special_rows(V, dt, kind, ent):
    """Rows with words at -inf, all at bf16's lowest value, and one possible
    word: scores, sums and gradient; beside them, in a call of their own, rows
    of NaN and +inf, which are NaN themselves and leave the others alone."""
    torch, dev = torch_dev()
    say(f"[policy special] V={V} {dt} {kind} ent={ent}")
    s, ent, kl, lo, hi = f32(1.5), f32(ent), f32(0.1), f32(0.2), f32(0.28)
    xs, y = _special(V)
    x = _dev(xs).to(torch.bfloat16 if dt == "bf16" else torch.float32)
    good, bad = [0, 2, 3, 8], [5, 6, 7]
    xv = out_to_f64(x, dt).reshape(xs.shape)[good]
    T, yg = len(good), y[good]
    lp, m, z, h = ob.token_logp(xv, yg, s)
    w, adv = np.full(T, 0.25, np.float32), np.array([1.0, -0.5, 0.25, 2.0], np.float32)
    old, ref = (lp + 0.05).astype(np.float32), (lp - 0.1).astype(np.float32)
    ro, rg, rgh = ob.policy_loss(kind, lp, h, w, adv, old, ref, lo, hi, 0.0, kl, ent)
    rd = ob.logits_grad(xv, yg, rg, rgh, s)
    pol = q.policy_struct(q.OBJ_CLIP if kind == "clip" else q.OBJ_NLL, lo, hi, 0.0, kl, ent)
    out, glp, dx, _ = _policy_logits(x[good].contiguous(), V, dt, yg, s, pol, w, adv, old, ref)
    tl, tz, th = _tol_rows(V, lp, z)
    assert np.all(np.abs(glp - lp) <= tl)
    tloss, tg, tk = _token_tol(dict(logp=lp, entropy=h, adv=adv, old=old, ref=ref), kl, ent, tl)
    tol = _tol_grad(xv, yg, rd, rg, rgh, s, w * tg + 2 * U * np.abs(rg))
    if dt == "bf16":
        tol = tol + 2.0 ** -8 * (np.abs(rd) + tol)
    got = out_to_f64(dx, dt).reshape(T, V)
    assert np.all(np.abs(got - rd) <= tol)
    absum = np.array([(w * (tloss + abs(ent) * th)).sum(), (w * tk).sum(), 0.0, (w * th).sum()])
    terms = w.sum() * (4 + np.abs(ro).max() / w.sum()) + (w * (np.abs(lp) + h)).sum()
    assert np.all(np.abs(out - ro) <= absum + 4 * U * terms)
    # with the others in the same call
    at = good + bad
    more = lambda v: np.concatenate([v, np.full(3, 0.25, np.float32)])  # noqa: E731
    out, glp2, dx, _ = _policy_logits(x[at].contiguous(), V, dt, y[at], s, pol, more(w), more(adv),
                                      more(old), more(ref))
    d = out_to_f64(dx, dt).reshape(len(at), V)
    assert np.array_equal(glp2[:T], glp) and np.array_equal(d[:T], got)
    assert np.isnan(glp2[T:]).all() and np.isnan(d[T:]).all() and np.isnan(out[[0, 3]]).all()
