"""Objectives of an adapter's training step and counter-based dropout, in
float64 (oracle).

TEST INFRASTRUCTURE ONLY -- see ``oracle/__init__.py``.

Written from the definitions: log-softmax and entropy of a row of logits and
their derivatives; the preference losses over pairs of answers; the clipped
policy objective with a KL estimate; the Philox4x32-10 generator of Salmon et
al. ("Parallel random numbers: as easy as 1, 2, 3"), in Python integers.
"""

import math

import numpy as np


def token_logp(x, labels, s=1.0):
    """(logp, m, z, entropy) by row of logits x [T, V]; zeros where the label
    is outside [0, V); a row of -inf alone: logp = -inf, the rest (-inf, 0, 0)."""
    T, V = x.shape
    out = np.zeros((4, T))
    with np.errstate(all="ignore"):
        for t in range(T):
            y = int(labels[t])
            if not 0 <= y < V:
                continue
            row = np.asarray(x[t], np.float64)
            if np.isnan(row).any() or (row == np.inf).any():
                out[:, t] = np.nan
                continue
            m = row.max()
            if m == -np.inf:
                out[:, t] = -np.inf, -np.inf, 0.0, 0.0
                continue
            u = s * (row - m)
            e = np.exp(u)
            z = math.log(e.sum())
            live = e > 0
            out[:, t] = u[y] - z, m, z, z - (u[live] * e[live]).sum() / e.sum()
    return out


def logits_grad(x, labels, g, gh, s=1.0):
    """s (g (1[v = y] - p_v) - gh p_v (log p_v + H)) by row."""
    T, V = x.shape
    _, m, z, h = token_logp(x, labels, s)
    d = np.zeros((T, V))
    with np.errstate(all="ignore"):
        for t in range(T):
            y = int(labels[t])
            if not 0 <= y < V or m[t] == -np.inf:
                continue
            lp = s * (np.asarray(x[t], np.float64) - m[t]) - z[t]
            p = np.exp(lp)
            ent = np.where(p > 0, p * (lp + h[t]), p)
            d[t] = -g[t] * p - (gh[t] * ent if gh[t] != 0 else 0.0)
            d[t, y] += g[t]
    return s * d


def pair_loss(kind, h, beta, margin=0.0, smoothing=0.0):
    """(l, dl/dh) of one pair."""
    if kind == "squared":
        return (h - 0.5 / beta) ** 2, 2.0 * (h - 0.5 / beta)
    u = beta * h - margin
    if kind == "hinge":
        return max(0.0, 1.0 - u), -beta if u < 1.0 else 0.0
    a, b = np.logaddexp(0.0, -u), np.logaddexp(0.0, u)
    sig, neg = math.exp(-a), math.exp(-b)
    return ((1.0 - smoothing) * a + smoothing * b,
            beta * (smoothing * sig - (1.0 - smoothing) * neg))


def pref_loss(kind, logp, ref, mask, cu, beta, margin=0.0, smoothing=0.0, average=False):
    """(loss, rewards [2P], dlogp [T]) of pairs (k, P + k) of the answers
    cu[i] .. cu[i + 1] - 1."""
    T = len(logp)
    n = len(cu) - 1
    P = n // 2
    total, where = np.zeros(n), []
    for i in range(n):
        a = min(max(int(cu[i]), 0), T)
        b = max(a, min(int(cu[i + 1]), T))
        at = np.array([t for t in range(a, b) if mask is None or mask[t]], dtype=np.int64)
        d = np.asarray(logp, np.float64)[at]
        if ref is not None:
            d = d - np.asarray(ref, np.float64)[at]
        total[i] = d.sum()
        if average:
            total[i] /= max(1, len(at))
        where.append(at)
    loss, grad = 0.0, np.zeros(T)
    for k in range(P):
        l, dh = pair_loss(kind, total[k] - total[P + k], beta, margin, smoothing)
        loss += l / P
        for i, sign in ((k, 1.0), (P + k, -1.0)):
            grad[where[i]] += sign * dh / P / (max(1, len(where[i])) if average else 1)
    return loss, beta * total, grad


def policy_loss(kind, logp, entropy, weight, adv, old, ref, clip_lo=0.2, clip_hi=0.2, clip_dual=0.0,
                kl_coef=0.0, ent_coef=0.0):
    """(out [4], dlogp, dentropy) of the token objective; tokens of weight 0
    are left out whatever they hold."""
    T = len(logp)
    out, g, gh = np.zeros(4), np.zeros(T), np.zeros(T)
    for t in range(T):
        w = 1.0 if weight is None else float(weight[t])
        if w == 0.0:
            continue
        lp, a = float(logp[t]), 1.0 if adv is None else float(adv[t])
        bound = 0.0
        if kind == "nll":
            f, df = a * lp, a
        else:
            d = 0.0 if old is None else lp - float(old[t])
            r = math.exp(d)
            f = min(r * a, min(max(r, 1.0 - clip_lo), 1.0 + clip_hi) * a)
            if clip_dual and a < 0:
                f = max(f, clip_dual * a)
            bound = float(f != r * a)
            df = 0.0 if bound else r * a
        k = dk = 0.0
        if ref is not None:
            q = float(ref[t]) - lp
            k, dk = math.expm1(q) - q, -math.expm1(q)
        h = 0.0 if entropy is None else float(entropy[t])
        out += w * np.array([-f + kl_coef * k - ent_coef * h, k, bound, h])
        g[t] = w * (-df + kl_coef * dk)
        gh[t] = -w * ent_coef
    return out, g, gh


def philox4x32(counter, key, rounds=10):
    """One block: counter (4 words), key (2 words) -> 4 words."""
    a, b, c, d = counter
    k0, k1 = key
    for _ in range(rounds):
        u, v = a * 0xD2511F53, c * 0xCD9E8D57
        a, b, c, d = (v >> 32) ^ b ^ k0, v % 2 ** 32, (u >> 32) ^ d ^ k1, u % 2 ** 32
        k0, k1 = (k0 + 0x9E3779B9) % 2 ** 32, (k1 + 0xBB67AE85) % 2 ** 32
    return a, b, c, d


def dropout_keep(rows, cols, p, seed, counter, only=None):
    """Boolean mask [rows, cols] (or of the rows `only`): 16 bits an element
    from block row * ceil(cols / 8) + col / 8, kept from p16 up."""
    groups = -(-cols // 8)
    p16 = min(int(math.floor(65536 * p + 0.5)), 65535)
    split = lambda v: (v % 2 ** 32, v >> 32)  # noqa: E731
    picked = range(rows) if only is None else only
    keep = np.zeros((len(picked), cols), bool)
    for i, row in enumerate(picked):
        for j in range(groups):
            w = philox4x32(split(row * groups + j) + split(counter), split(seed))
            half = [(w[k // 2] >> (16 * (k % 2))) % 65536 for k in range(8)]
            n = min(8, cols - 8 * j)
            keep[i, 8 * j:8 * j + n] = np.array(half[:n]) >= p16
    return keep, p16


def token_top(x, k, scale=1.0):
    """The k largest logits of each row, ties to the lower index: (ids, log p).
    A NaN is no word: behind all others, with the id -1."""
    x = np.asarray(x, np.float64)
    order = np.lexsort((-x, np.isnan(x)), axis=1)[:, :k]
    m = x.max(1, keepdims=True)
    m = np.where(np.isfinite(m), m, 0.0)
    with np.errstate(divide="ignore"):
        lp = scale * (x - m) - np.log(np.exp(scale * (x - m)).sum(1, keepdims=True))
    lp = np.where(x == -np.inf, -np.inf, lp)
    some = ~np.isnan(np.take_along_axis(x, order, 1))
    return np.where(some, order, -1), np.take_along_axis(lp, order, 1)


def distill(x, ids, teacher, weight, scale=1.0, normalize=True):
    """(loss, kl [T], dx [T, V]) of rows x against the teacher's alternatives."""
    x = np.asarray(x, np.float64)
    T, V = x.shape
    kl, dx = np.zeros(T), np.zeros((T, V))
    for t in range(T):
        if weight[t] == 0:
            continue
        on = (ids[t] >= 0) & (ids[t] < V) & (teacher[t] != -np.inf)
        if not on.any():
            continue
        word, lq = ids[t][on], teacher[t][on].astype(np.float64)
        if normalize:
            lq = lq - (lq.max() + np.log(np.exp(lq - lq.max()).sum()))
        q = np.exp(lq)
        m = x[t].max()
        if m == -np.inf:
            kl[t] = np.inf
            continue
        u = scale * (x[t] - m)
        lp = u - np.log(np.exp(u).sum())
        kl[t] = np.where(q > 0, q * (lq - lp[word]), 0.0).sum()
        dx[t] = q.sum() * np.exp(lp)
        np.subtract.at(dx[t], word, q)
        dx[t] *= scale * weight[t]
    return (weight * kl)[weight != 0].sum(), kl, dx
