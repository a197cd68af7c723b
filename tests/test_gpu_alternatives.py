"""The top alternatives of rows of logits, and the loss against a teacher's.

The words are compared exactly (value, then the lower index); log-probabilities,
entropies and gradients with the bounds of tests/test_gpu_objective.py.  A
teacher's q_j = e^(x - top) / c is within (|x - top| + 72) 2^-24 of itself (the
argument's rounding, expf, a sum of 64, a quotient), ln q_j within 4 (1 + |ln q_j|)
2^-24; a kl adds each product's and 8 additions' roundings."""

import numpy as np
import pytest

from oracle import objective as ob
from quantized_rank_fine_amd import qlora as q

from gpu_harness import out_to_f64, say, torch_dev
from test_gpu_objective import SHAPES, U, _dev, _fwd, _rows, _tol_rows, f32

pytestmark = pytest.mark.gpu


def _qd(dt):
    return q.BF16 if dt == "bf16" else q.F32


def _top(x, ld, dt, labels, s, k, logp=True, entropy=True):
    torch, dev = torch_dev()
    T, V = x.shape
    ids = torch.full((T * k + 8,), 77, dtype=torch.int32, device=dev)
    top = torch.full((T * k + 8,), 7.0, device=dev)
    lp = torch.full((T + 8,), 7.0, device=dev) if logp and labels is not None else None
    h = torch.full((T + 8,), 7.0, device=dev) if entropy else None
    n = q.qlora_token_top_workspace_bytes(T, V, _qd(dt), k)
    ws = torch.full((n + 256,), 255, dtype=torch.uint8, device=dev)
    q.qlora_token_top(x, ld, T, V, _qd(dt), labels, s, k, ids, top, lp, h, ws if n else None, n)
    torch.cuda.synchronize()
    assert (ws[n:] == 255).all() and (ids[T * k:] == 77).all() and (top[T * k:] == 7).all()
    assert all(v is None or (v[T:] == 7).all() for v in (lp, h))
    cut = lambda v: None if v is None else v[:T]  # noqa: E731
    return (ids[:T * k].view(T, k).cpu().numpy(), top[:T * k].view(T, k).cpu().numpy(), cut(lp),
            cut(h))


def _check_top(x, xv, ld, dt, s, k, labels=None):
    torch, _ = torch_dev()
    T, V = xv.shape
    ids, top, lp, h = _top(x, ld, dt, None if labels is None else _dev(labels), s, k)
    want, wlp = ob.token_top(xv, k, s)
    _, _, z, _ = ob.token_logp(xv, np.zeros(T, np.int64), s)
    ok = np.ones(T, bool) if labels is None else (labels >= 0) & (labels < V)
    bad = np.nonzero((ids[ok] != want[ok]).any(1))[0]
    assert not len(bad), (bad[:4], ids[ok][bad[:1]], want[ok][bad[:1]])
    with np.errstate(invalid="ignore"):
        tol = _tol_rows(V, 0.0, z)[0][:, None] + 3 * U * np.abs(np.where(wlp > -np.inf, wlp, 0.0))
        near = (top == wlp) | (np.abs(top - wlp) <= tol)
    assert near[ok].all(), np.abs(top - wlp)[ok].max()
    assert np.all(ids[~ok] == -1) and np.all(top[~ok] == 0)
    if labels is not None:
        # the same sums as the scoring's: the same bits
        l2, _, h2 = _fwd(x, ld, dt, _dev(labels), s)
        assert torch.equal(lp, l2) and torch.equal(h, h2)
        some = _top(x, ld, dt, _dev(labels), s, k, logp=False, entropy=False)
        assert np.array_equal(some[0], ids) and np.array_equal(some[1], top)
    return ids, top


@pytest.mark.parametrize("T,V,ld,dt,s,at", SHAPES + [
    (9, 8200, 8200, "bf16", 1.0, 1), (9, 12345, 12345, "f32", 1.0, 1),
    (5, 40000, 40001, "bf16", 1.0, 2), (65, 65537, 65537, "f32", 1.0, 0)])
@pytest.mark.parametrize("k", [1, 7, 20, 64])
def test_top(T, V, ld, dt, s, at, k):
    if k > V:
        return
    say(f"[top] T={T} V={V} ld={ld} {dt} s={s} at={at} k={k}")
    s = f32(s)
    x, xv = _rows(T, V, ld, dt, V + T, at)
    y = np.random.default_rng(V).integers(0, V, T)
    if T > 3:
        y[1], y[2] = -100, V
    _check_top(x, xv, ld, dt, s, k, y)
    _check_top(x, xv, ld, dt, s, k)


def _hard_rows(V, k, g):
    """Rows that a bound from lane maxima does not suit, by name."""
    r = lambda: g.standard_normal(V) * 2  # noqa: E731
    rows = {
        "equal": np.zeros(V), "equal negative": np.full(V, -3.5),
        "ascending": np.arange(V) / 16.0, "descending": -np.arange(V) / 16.0,
        "two values": (np.arange(V) % 3 == 1) * 1.0, "nothing": np.full(V, -np.inf),
        "lowest": np.full(V, -3.3895314e38), "zeros": np.where(np.arange(V) % 2, 0.0, -0.0),
        "coarse": np.round(r()), "constant tail": np.where(np.arange(V) < k // 2, 1.0, 0.5),
    }
    live = r()
    live[np.setdiff1d(np.arange(V), g.permutation(V)[:max(1, k // 2)])] = -np.inf
    rows["few live"] = live
    live = r()
    live[np.setdiff1d(np.arange(V), g.permutation(V)[:max(1, k // 2)])] = -1e9
    rows["few above a finite mask"] = live
    half = r()
    half[V // 2:] = -np.inf
    rows["half masked"] = half
    one = np.full(V, -np.inf)
    one[V - 1] = 3.0
    rows["one, the last"] = one
    lane = r() - 20
    lane[:min(V, 600)] += 60                       # the best all side by side
    rows["side by side"] = lane
    far = r()
    far[g.integers(0, V, 3)] = 3e38
    rows["far"] = far
    return rows


@pytest.mark.parametrize("V", [64, 100, 2047, 4096, 8191, 16000, 32000, 32003, 40007, 131072])
@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_top_of_hard_rows(V, dt):
    """Ties past every list, masks that leave fewer words than are asked for,
    sorted rows; cut rows among them."""
    torch, dev = torch_dev()
    for k in (1, 20, 64):
        rows = _hard_rows(V, k, np.random.default_rng(V + k))
        say(f"[top hard] V={V} {dt} k={k}")
        v = torch.from_numpy(np.stack(list(rows.values())).astype(np.float32)).to(dev)
        x = v.to(torch.bfloat16 if dt == "bf16" else torch.float32)
        xv = out_to_f64(x, dt).reshape(len(rows), V)
        ids, _, _, _ = _top(x, V, dt, None, 1.0, k)
        want, _ = ob.token_top(xv, k)
        for i, name in enumerate(rows):
            assert np.array_equal(ids[i], want[i]), (name, ids[i], want[i])
        many = x.repeat(9, 1)                      # and too many rows to be cut
        ids, _, _, _ = _top(many, V, dt, None, 1.0, k)
        assert np.array_equal(ids, np.tile(want, (9, 1)))


@pytest.mark.parametrize("V", [70, 5000, 131072])
def test_top_of_masked_rows_values(V):
    """log p of masked words and of rows of nothing else."""
    x = np.full((3, V), -np.inf, np.float32)
    x[0, 5], x[0, 9] = 1.0, 2.0
    x[2, 3] = -2.0
    xd = _dev(x)
    ids, top, _, h = _top(xd, V, "f32", None, 1.0, 4)
    assert ids.tolist() == [[9, 5, 0, 1], [0, 1, 2, 3], [3, 0, 1, 2]]
    lse = np.log(np.exp(1.0) + np.exp(2.0))
    assert np.allclose(top[0, :2], [2 - lse, 1 - lse], atol=1e-6)
    assert np.all(top[0, 2:] == -np.inf) and np.all(top[1] == -np.inf) and top[2, 0] == 0
    assert h[1] == 0 and h[2] == 0


@pytest.mark.parametrize("V", [300, 5000, 32000, 131072])
def test_top_of_rows_with_nan(V):
    g = np.random.default_rng(V)
    x = (g.standard_normal((4, V)) * 2).astype(np.float32)
    x[0, 7] = np.nan
    x[1] = np.nan
    x[2, :] = np.nan
    x[2, V // 2] = 1.0
    x[3, 11] = np.inf
    ids, top, _, h = _top(_dev(x), V, "f32", None, 1.0, 8)
    want, _ = ob.token_top(x, 8)
    assert np.array_equal(ids[0], want[0]) and np.array_equal(ids[3], want[3]) and ids[3, 0] == 11
    assert np.all(ids[1] == -1) and ids[2, 0] == V // 2 and np.all(ids[2, 1:] == -1)
    assert np.isnan(top).all() and np.isnan(h.cpu().numpy()).all()


@pytest.mark.parametrize("V", [64, 300, 2049, 8191, 16000, 32003, 40007, 131077])
@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_top_of_nan_beside_a_mask(V, dt):
    """NaN among the first words of rows that -inf leaves few others: as many
    words at -inf as are asked for, the lowest, wherever they lie."""
    torch, dev = torch_dev()
    at = np.arange(V)
    for k in (2, 20, 64):
        g = np.random.default_rng(V + k)
        masked = lambda: np.full(V, -np.inf)  # noqa: E731
        rows = {n: masked() for n in ("first", "all of the first", "every other", "few live",
                                      "long run", "few left", "last alone", "none", "an infinity")}
        rows["first"][0] = np.nan
        rows["all of the first"][:k] = np.nan
        rows["every other"][::2] = np.nan
        rows["few live"][g.permutation(V)[:k // 2]] = g.standard_normal(k // 2)
        rows["few live"][:k // 2] = np.nan
        rows["long run"][:V - 70] = np.nan
        rows["few left"][:] = np.nan
        rows["few left"][g.permutation(V)[:k // 2]] = -np.inf
        rows["few left"][V // 3] = 0.5
        rows["last alone"][:V - 1] = np.nan
        rows["an infinity"][at % 7 == 0] = np.nan
        rows["an infinity"][V - 2] = np.inf
        say(f"[top nan] V={V} {dt} k={k}")
        v = torch.from_numpy(np.stack(list(rows.values())).astype(np.float32)).to(dev)
        x = v.to(torch.bfloat16 if dt == "bf16" else torch.float32)
        want, _ = ob.token_top(out_to_f64(x, dt).reshape(len(rows), V), k)
        for many in (1, 9):                        # and too many rows to be cut
            ids, top, _, h = _top(x.repeat(many, 1), V, dt, None, 1.0, k)
            for i, name in enumerate(list(rows) * many):
                assert np.array_equal(ids[i], want[i % len(rows)]), (name, k, ids[i])
            sound = np.array([n == "none" for n in rows] * many)
            assert np.isnan(top[~sound]).all() and np.isnan(h.cpu().numpy()[~sound]).all()
            assert np.all(top[sound] == -np.inf)


@pytest.mark.parametrize("V", [64, 300, 2049, 8191, 32003, 40007, 131077])
@pytest.mark.parametrize("dt,bits", [("bf16", 0x7f81), ("bf16", 0xff81), ("bf16", 0xffc0),
                                     ("f32", 0x7f800001), ("f32", 0xff800001), ("f32", 0xffc00000)])
def test_top_of_every_kind_of_nan(V, dt, bits):
    """Signalling and quiet NaN of both signs, few and many of them, beside ordinary
    words and words at -inf: the other words of their groups are found."""
    torch, dev = torch_dev()
    g = np.random.default_rng(V)
    x = (g.standard_normal((4, V)) * 2).astype(np.float32)
    x[g.random(x.shape) < 0.3] = -np.inf
    nan = g.random(x.shape) < np.array([0.0, 0.01, 0.5, 0.98])[:, None]
    nan[:, g.integers(0, V)] = True
    u = np.uint16 if dt == "bf16" else np.uint32
    t = torch.from_numpy(x).to(torch.bfloat16 if dt == "bf16" else torch.float32)
    xv = np.where(nan, np.nan, t.double().numpy())
    raw = t.view(torch.int16 if dt == "bf16" else torch.int32).numpy().view(u).copy()
    raw[nan] = bits
    xd = torch.from_numpy(raw.view(np.int16 if dt == "bf16" else np.int32)).to(dev).view(t.dtype)
    for k in (1, 20, 64):
        say(f"[top nan] V={V} {dt} {bits:#x} k={k}")
        want, _ = ob.token_top(xv, k)
        for many in (1, 17):                       # and too many rows to be cut
            ids, top, _, h = _top(xd.repeat(many, 1), V, dt, None, 1.0, k)
            assert np.array_equal(ids, np.tile(want, (many, 1)))
            assert np.isnan(top).all() and np.isnan(h.cpu().numpy()).all()


def test_top_many_rows():
    """More rows than a grid's dimension holds, tiny vocabularies."""
    x, xv = _rows(40000, 9, 9, "bf16", 1, 1)
    _check_top(x, xv, 9, "bf16", 1.0, 9)


def test_top_and_distill_far_into_memory():
    """Rows past 2^32 bytes from the first."""
    torch, dev = torch_dev()
    V, ld = 501, (1 << 31) + 8
    buf = torch.zeros(ld + V, dtype=torch.bfloat16, device=dev)
    rows, xv = _rows(2, V, V, "bf16", 3)
    buf[:V], buf[ld:ld + V] = rows[0], rows[1]
    x = buf.as_strided((2, V), (ld, 1))
    ids, top = _check_top(x, xv, ld, "bf16", 1.0, 5)
    a = _distill(rows, V, "bf16", 1.0, _dev(ids), _dev(top), None, True)
    b = _distill(x, ld, "bf16", 1.0, _dev(ids), _dev(top), None, True, inplace=True)
    assert torch.equal(a[2], b[2]) and torch.equal(a[1], b[1])


# --------------------------------------------------------------- distillation

def _distill(x, ld, dt, s, ids, teacher, weight, normalize, inplace=False):
    torch, dev = torch_dev()
    T, V = x.shape
    k = ids.shape[1]
    loss = torch.full((5,), 7.0, device=dev)
    kl = torch.full((T + 8,), 7.0, device=dev)
    ldd = ld if inplace else V + 5
    buf = None if inplace else torch.full((T * ldd + 9,), 3.0, dtype=x.dtype, device=dev)
    dx = x if inplace else buf[1:]
    n = q.qlora_distill_workspace_bytes(T, V, _qd(dt), k)
    ws = torch.full((n + 256,), 255, dtype=torch.uint8, device=dev)
    q.qlora_distill_logits(x, ld, T, V, _qd(dt), s, weight, k, ids, teacher, normalize, loss, kl,
                           dx, ldd, ws if n else None, n)
    torch.cuda.synchronize()
    assert (ws[n:] == 255).all() and (loss[1:] == 7).all() and (kl[T:] == 7).all()
    if inplace:
        return loss[:1], kl[:T], x.clone()
    assert buf[0] == 3 and (buf[1 + T * ldd:] == 3).all()
    rows = buf[1:1 + T * ldd].view(T, ldd)
    assert (rows[:, V:] == 3).all()
    return loss[:1], kl[:T], rows[:, :V].contiguous()


def _teacher(xv, k, g, s):
    """A teacher near the student: its alternatives, with words twice, words
    outside the vocabulary, impossible ones, rows of none."""
    T, V = xv.shape
    ids, t = ob.token_top(xv + g.standard_normal(xv.shape), min(k, V), s)
    ids = np.concatenate([ids, np.full((T, k - ids.shape[1]), -1)], 1)
    t = np.concatenate([t, np.zeros((T, k - t.shape[1]))], 1).astype(np.float32)
    ids = ids.astype(np.int32)
    for r in range(T):
        if k > 3 and r % 3 == 1:
            ids[r, 2] = ids[r, 0]                  # twice
            ids[r, 3] = (-1, V, -7, 2 ** 31 - 1)[r % 4]
        if k > 5 and r % 3 == 2:
            t[r, 1] = -np.inf
            ids[r, 4] = V - 1
            ids[r, 5] = 0
    if T > 5:
        ids[4] = -1
        t[5] = -np.inf
    return ids, t


def _check_distill(got, xv, ids, t, w, s, normalize, dt):
    loss, kl, dx = got
    T, V = xv.shape
    rl, rk, rd = ob.distill(xv, ids, t, w, s, normalize)
    lp, m, z, _ = ob.token_logp(xv, np.zeros(T, np.int64), s)
    on = (ids >= 0) & (ids < V) & (t != -np.inf) & (w != 0)[:, None]
    tt = np.where(on, t.astype(np.float64), -np.inf)
    top = np.where(on.any(1), tt.max(1), 0.0)[:, None]
    e = np.where(on, np.exp(tt - top), 0.0)
    c = np.maximum(e.sum(1, keepdims=True), 1e-300)
    q_ = e / c if normalize else np.where(on, np.exp(tt), 0.0)
    lq = np.where(on, tt - top - np.log(c) if normalize else tt, 0.0)
    zt = _tol_rows(V, lp, z)[1][:, None]
    l = s * (xv - m[:, None]) - z[:, None]
    word = np.where(on, ids, 0)
    lw = np.take_along_axis(l, word, 1)
    qrel = (np.abs(np.where(on, tt - (top if normalize else 0.0), 0.0)) + 72) * U
    with np.errstate(invalid="ignore"):
        ktol = (q_ * (zt + 3 * U * np.abs(lw) + 4 * U * (1 + np.abs(lq))
                      + (qrel + 12 * U) * np.abs(lq - lw))).sum(1) + 1e-37
    gk = kl.cpu().numpy()
    assert np.all(np.abs(gk - rk) <= ktol), np.abs(gk - rk).max()
    assert abs(float(loss) - rl) <= (np.abs(w) * ktol).sum() + U * (abs(rl) + 1e-30)
    p = np.exp(l)
    C = q_.sum(1, keepdims=True)
    Q, Qt = np.zeros_like(p), np.zeros_like(p)
    for r in range(T):
        np.add.at(Q[r], word[r], q_[r])
        np.add.at(Qt[r], word[r], q_[r] * (qrel[r] + 4 * U))
    crel = 0.0 if normalize else (q_ * qrel).sum(1, keepdims=True) / np.maximum(C, 1e-300) + 8 * U
    tol = C * p * (zt + (3 * np.abs(l) + 8) * U + crel) + Qt + 4 * U * (Q + C * p)
    tol = np.abs(s * w)[:, None] * tol + 2 * U * np.abs(rd) + 1e-36
    gd = out_to_f64(dx, dt).reshape(T, V)
    if dt == "bf16":
        tol = tol + 2.0 ** -8 * (np.abs(rd) + tol)
    assert np.all(np.abs(gd - rd) <= tol), (np.abs(gd - rd) - tol).max()
    assert not gd[~on.any(1)].any() and not gk[~on.any(1)].any()


@pytest.mark.parametrize("T,V,ld,dt,s,at", [
    (1, 1, 1, "f32", 1.0, 0), (7, 7, 7, "bf16", 1.0, 1), (6, 8, 8, "bf16", 0.7, 0),
    (7, 63, 65, "f32", 1.25, 3), (7, 2047, 2047, "bf16", 1.0, 5), (6, 2049, 2056, "f32", 2.0, 0),
    (70, 1000, 1000, "bf16", 1.0, 0), (6, 4097, 4097, "bf16", 1.0, 0),
    (7, 9000, 9000, "f32", 1.0, 1), (7, 16001, 16001, "bf16", 1.0, 0),
    (7, 32000, 32000, "bf16", 1.0, 0), (6, 50001, 50016, "f32", 1.25, 1),
    (6, 65537, 65537, "bf16", 0.5, 1), (6, 131077, 131077, "f32", 1.0, 0),
    (66, 70003, 70003, "bf16", 1.0, 0)])
@pytest.mark.parametrize("k,normalize", [(1, True), (6, False), (20, True), (64, True)])
def test_distill(T, V, ld, dt, s, at, k, normalize):
    say(f"[distill] T={T} V={V} ld={ld} {dt} s={s} at={at} k={k} normalize={normalize}")
    torch, _ = torch_dev()
    s = f32(s)
    g = np.random.default_rng(V + k)
    x, xv = _rows(T, V, ld, dt, V + T, at)
    ids, t = _teacher(xv, k, g, s)
    w = (g.standard_normal(T) / T).astype(np.float32)
    if T > 3:
        w[3] = 0.0
    got = _distill(x, ld, dt, s, _dev(ids), _dev(t), _dev(w), normalize)
    _check_distill(got, xv, ids, t, w.astype(np.float64), s, normalize, dt)
    # without weights: all 1
    one = _distill(x, ld, dt, s, _dev(ids), _dev(t), None, normalize)
    _check_distill(one, xv, ids, t, np.ones(T), s, normalize, dt)
    # in place
    again = _distill(x, ld, dt, s, _dev(ids), _dev(t), _dev(w), normalize, inplace=True)
    assert all(torch.equal(a, b) for a, b in zip(got, again))


@pytest.mark.parametrize("V", [300, 32000, 70000])
def test_distill_special_rows(V):
    """Skipped tokens hold anything; a word that the student cannot give; rows
    of nothing; NaN."""
    g = np.random.default_rng(V)
    x = (g.standard_normal((8, V)) * 2).astype(np.float32)
    ids = np.tile(np.array([[3, 5, 9]], np.int32), (8, 1))
    t = np.tile(np.log(np.array([[0.5, 0.3, 0.2]], np.float32)), (8, 1))
    w = np.ones(8, np.float32)
    x[0], t[0], w[0] = np.nan, np.nan, 0.0             # skipped
    x[1, 5] = -np.inf                                  # cannot be given, but is wanted
    x[2] = -np.inf                                     # nothing can
    x[3, 100] = np.nan
    t[4, 1] = np.nan
    x[5, V // 2:] = -np.inf                            # masked words
    x[6], ids[6] = np.nan, -1                          # no alternatives: not read for a value
    x[7, 20:] = -1e9                                   # masked by a finite value
    loss, kl, dx = _distill(_dev(x), V, "f32", 1.0, _dev(ids), _dev(t), _dev(w), True)
    kl, dx = kl.cpu().numpy(), dx.cpu().numpy()
    assert kl[0] == 0 and not dx[0].any() and kl[6] == 0 and not dx[6].any()
    assert kl[1] == np.inf and kl[2] == np.inf and not dx[2].any()
    p = np.exp(x[1].astype(float) - x[1].max())
    p /= p.sum()
    p[[3, 5, 9]] -= [0.5, 0.3, 0.2]
    assert np.abs(dx[1] - p).max() < 1e-6
    assert np.isnan(kl[3]) and np.isnan(dx[3]).all() and np.isnan(kl[4]) and np.isnan(dx[4]).all()
    assert np.isnan(float(loss))
    for r in (5, 7):
        rl, rk, rd = ob.distill(x[r:r + 1], ids[r:r + 1], t[r:r + 1], [1.0])
        assert abs(kl[r] - rk[0]) < 1e-5 and np.abs(dx[r] - rd).max() < 1e-6
    only = np.zeros(8, np.float32)
    only[5] = 1.0
    loss, _, _ = _distill(_dev(x), V, "f32", 1.0, _dev(ids), _dev(t), _dev(only), True)
    assert abs(float(loss) - kl[5]) < 1e-6             # infinities and NaN of weight 0 add nothing


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_distill_many_rows(dt):
    """More rows than a grid's dimension, the loss in two launches."""
    g = np.random.default_rng(2)
    T, V, k = 40000, 21, 5
    x, xv = _rows(T, V, V, dt, 4, 1)
    ids = np.argsort(g.random((T, V)), 1)[:, :k].astype(np.int32)
    t = -np.abs(g.standard_normal((T, k))).astype(np.float32)
    w = (g.random(T) / T).astype(np.float32)
    _check_distill(_distill(x, V, dt, 1.0, _dev(ids), _dev(t), _dev(w), True), xv, ids, t,
                   w.astype(float), 1.0, True, dt)


def test_distill_gradient_is_the_difference_quotient():
    g = np.random.default_rng(0)
    T, V, k = 3, 40, 6
    x = g.standard_normal((T, V))
    ids = g.integers(0, V, (T, k)).astype(np.int32)
    t = -np.abs(g.standard_normal((T, k))).astype(np.float32)
    w = g.random(T)
    for normalize in (True, False):
        _, _, d = ob.distill(x, ids, t, w, 0.8, normalize)
        for r, v in ((0, int(ids[0, 0])), (1, 7), (2, int(ids[2, 3]))):
            up, down = x.copy(), x.copy()
            up[r, v] += 1e-5
            down[r, v] -= 1e-5
            diff = (ob.distill(up, ids, t, w, 0.8, normalize)[0]
                    - ob.distill(down, ids, t, w, 0.8, normalize)[0]) / 2e-5
            assert abs(diff - d[r, v]) < 1e-8
        got = _distill(_dev(x.astype(np.float32)), V, "f32", f32(0.8), _dev(ids), _dev(t),
                       _dev(w.astype(np.float32)), normalize)[2].cpu().numpy()
        assert np.abs(got - d).max() < 1e-6


def test_no_tokens():
    torch, dev = torch_dev()
    loss = torch.full((1,), 3.0, device=dev)
    q.qlora_distill_logits(None, 9, 0, 9, q.F32, 1.0, None, 2, None, None, True, loss, None, None,
                           9, None, 0)
    assert float(loss) == 0
    q.qlora_token_top(None, 9, 0, 9, q.F32, None, 1.0, 2, None, None, None, None, None, 0)


@pytest.mark.parametrize("T,V,dt", [(20, 5000, "bf16"), (3, 140001, "bf16"), (90, 70001, "f32")])
def test_teacher_to_student_captured(T, V, dt):
    """What a distillation step runs: the teacher's alternatives, the student's
    loss on them in place; as a graph, replayed with other work between, and on
    another stream."""
    torch, dev = torch_dev()
    k = 24
    xt, _ = _rows(T, V, V, dt, 1)
    xs, xv = _rows(T, V, V, dt, 2)
    xs = xs.contiguous()
    keep = xs.clone()
    y = _dev(np.where(np.arange(T) % 4 == 1, -100, np.arange(T)))
    ids = torch.empty(T, k, dtype=torch.int32, device=dev)
    top, lp, kl, loss = (torch.empty(*n, device=dev) for n in ((T, k), (T,), (T,), (1,)))
    n = q.qlora_token_top_workspace_bytes(T, V, _qd(dt), k)
    m = q.qlora_distill_workspace_bytes(T, V, _qd(dt), k)
    ws = torch.empty(max(n, m, 16), dtype=torch.uint8, device=dev)
    xtc = xt.contiguous()

    def step():
        q.qlora_token_top(xtc, V, T, V, _qd(dt), y, 1.0, k, ids, top, lp, None, ws, n)
        xs.copy_(keep)
        q.qlora_distill_logits(xs, V, T, V, _qd(dt), 1.0, None, k, ids, top, True, loss, kl, xs, V,
                               ws, m)

    step()
    torch.cuda.synchronize()
    outs = (ids, top, lp, kl, loss, xs)
    want = [t.clone() for t in outs]
    _check_distill((loss, kl, xs), xv, ids.cpu().numpy(), top.cpu().numpy(), np.ones(T), 1.0, True,
                   dt)
    assert not xs[1].any() and kl[1] == 0              # the teacher did not score it
    cg = torch.cuda.CUDAGraph()
    with torch.cuda.graph(cg):
        step()
    for _ in range(3):
        for t in outs:
            t.fill_(5)
        ws.fill_(255)
        torch.cuda.synchronize()
        cg.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(outs, want))
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()
    s.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(outs, want))
