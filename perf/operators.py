"""The operators of an adapter's training step beside the adapted linear,
as measured cases: token log-probabilities, preference loss, policy loss and
dropout without a stored mask.

``listed()`` names the cases, ``draw()`` gives more of the same ranges,
``prepare()`` makes a case's inputs on the GPU from a seed, ``run()`` is one
call and ``work()`` what that call has to move and compute.  With ``own``
false, ``run()`` computes the operators in plain 32-bit torch operations;
with ``own`` true it calls the library.  ``exact()`` gives the results in 64
bits from the definitions.

Notation: x logits, s the inverse temperature, y a token's label (a label
outside [0, V) is not scored), m = max x over the row,
z = log sum exp(s (x - m)), log p_v = s (x_v - m) - z, H = -sum p log p.
"""

import math

import numpy as np
import torch

own = False

IGNORE = -100
BLOCK = 64          # prompts are laid out in runs of this many tokens
PAD = 32            # masked vocabulary entries at the end of a row


# ------------------------------------------------------------------- cases

def listed():
    return [
        # one decoded token scored against the 32000-word head
        dict(name="logp-one-token", op="logp_fwd", T=1, V=32000, ld=32000, dt="bf16", scale=1.0,
             prompt=0.0, masked=False, entropy=False),
        # a batch of completions scored for a preference or policy step, a
        # quarter of the tokens being prompt
        dict(name="logp-batch", op="logp_fwd", T=4096, V=32000, ld=32000, dt="bf16", scale=1.0,
             prompt=0.25, masked=False, entropy=True),
        # the gradient of the same batch
        dict(name="logp-batch-grad", op="logp_bwd", T=4096, V=32000, ld=32000, dt="bf16",
             scale=1.0, prompt=0.25, masked=False, entropy=False),
        # fp32 logits of an odd vocabulary in padded rows, sampled at a
        # temperature, with an entropy bonus's gradient and masked words
        dict(name="logp-odd-f32-grad", op="logp_bwd", T=509, V=50001, ld=50016, dt="f32",
             scale=1.25, prompt=0.0, masked=True, entropy=True),
        # four pairs of short answers
        dict(name="pref-short", op="pref", P=4, longest=300, kind="sigmoid", ref=True,
             average=False),
        # a large batch of pairs, length-averaged log-probabilities
        dict(name="pref-batch", op="pref", P=256, longest=4096, kind="squared", ref=True,
             average=True),
        # few pairs of very long answers
        dict(name="pref-long", op="pref", P=2, longest=131072, kind="sigmoid", ref=True,
             average=False),
        # the tokens of a short answer
        dict(name="policy-short", op="policy", T=1000, kind="clip", dual=0.0, entropy=False),
        # 512 answers of 4096 tokens
        dict(name="policy-batch", op="policy", T=2097152, kind="clip", dual=3.0, entropy=True),
        # the whole loss of a policy step from the head's logits
        dict(name="policy-logits", op="policy_logits", T=8192, V=32000, ld=32000, dt="bf16",
             scale=1.0, prompt=0.25, masked=False, kind="clip"),
        # hidden states of one decoded batch
        dict(name="dropout-16-tokens", op="dropout", rows=16, cols=4096, dt="bf16", p=0.1,
             residual=False),
        # a block's output dropped and added to the residual stream
        dict(name="dropout-residual", op="dropout", rows=16384, cols=4096, dt="bf16", p=0.05,
             residual=True),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["logp_fwd", "logp_bwd", "policy_logits", "pref", "policy", "dropout"])
    if op in ("logp_fwd", "logp_bwd", "policy_logits"):
        dt = rng.choice(["bf16", "bf16", "f32"])
        V = _log_int(rng, 1000, 200000)
        T = _log_int(rng, 1, 8192)
        T = max(1, min(T, 200_000_000 // (V * (2 if dt == "f32" else 1))))
        ld = V + rng.choice([0, 0, 1, 7, 64])
        c = dict(op=op, T=T, V=V, ld=ld, dt=dt, scale=rng.choice([1.0, 1.0, 1.25, 0.7]),
                 prompt=rng.choice([0.0, 0.25, 0.5]), masked=rng.random() < 0.3)
        if op == "policy_logits":
            c["kind"] = rng.choice(["clip", "nll"])
        else:
            c["entropy"] = rng.random() < 0.5
        return c
    if op == "pref":
        longest = _log_int(rng, 16, 131072)
        P = max(1, min(_log_int(rng, 1, 512), (1 << 21) // longest))
        return dict(op=op, P=P, longest=longest, kind=rng.choice(["sigmoid", "squared"]),
                    ref=rng.random() < 0.8, average=rng.random() < 0.4)
    if op == "policy":
        return dict(op=op, T=_log_int(rng, 1, 1 << 21), kind=rng.choice(["clip", "clip", "nll"]),
                    dual=rng.choice([0.0, 3.0]), entropy=rng.random() < 0.5)
    cols = _log_int(rng, 64, 16384)
    rows = max(1, min(_log_int(rng, 1, 32768), (1 << 26) // cols))
    return dict(op=op, rows=rows, cols=cols, dt=rng.choice(["bf16", "f32"]),
                p=rng.choice([0.05, 0.1, 0.3]), residual=rng.random() < 0.5)


# ------------------------------------------------------------------- inputs

BETA = {"sigmoid": 0.1, "squared": 0.1}
SMOOTHING, MARGIN = 0.0, 0.25
CLIP_LO, CLIP_HI, KL, ENT = 0.2, 0.28, 0.04, 0.01


def _lengths(c):
    """Tokens of the 2 P answers, spread evenly over [longest / 8, longest]."""
    n = 2 * c["P"]
    return np.round(np.linspace(max(1, c["longest"] // 8), c["longest"], n)).astype(np.int64)


def _dtype(c):
    return torch.bfloat16 if c["dt"] == "bf16" else torch.float32


def _unscored(T, prompt):
    """Which of T tokens are prompt (by their place in runs of BLOCK)."""
    return (np.arange(T) % BLOCK) < round(prompt * BLOCK) if T >= BLOCK else np.zeros(T, bool)


def _ratios(n, g, dual=0.0):
    """Log-ratios of the new policy to the old, a few of them large, moved
    off the places where the clipped surrogate's branch changes, so that a
    rounding does not choose the branch."""
    f = dict(generator=g, device=g.device)
    d = torch.randn(n, **f) * torch.where(torch.rand(n, **f) < 0.03, 1.0, 0.15)
    edges = [math.log1p(-CLIP_LO), math.log1p(CLIP_HI)] + ([math.log(dual)] if dual else [])
    for e in edges:
        d = torch.where((d - e).abs() < 2e-3, d + 4e-3, d)
    return d


def _logits(c, g, dev):
    T, V, ld = c["T"], c["V"], c["ld"]
    x = torch.empty(T, ld, dtype=_dtype(c), device=dev)
    for r in range(0, T, 2048):
        n = min(2048, T - r)
        x[r:r + n] = torch.randn(n, ld, generator=g, device=dev) * 2.5
    live = V - PAD if c["masked"] else V
    labels = torch.randint(0, live, (T,), generator=g, device=dev)
    at = torch.arange(T, device=dev)
    lift = 8.0 * (torch.rand(T, generator=g, device=dev) < 0.5)
    x[at, labels] = (x[at, labels].float() + lift).to(x.dtype)
    if c["masked"]:
        x[:, live:V] = -math.inf
    labels[torch.from_numpy(_unscored(T, c["prompt"])).to(dev)] = IGNORE
    return x[:, :V], labels


def _stats(x, labels, s):
    """(logp, m, z, H) in 32 bits, in slices of rows."""
    parts = []
    for r in range(0, x.shape[0], 2048):
        xf = x[r:r + 2048].float()
        m = xf.amax(1)
        u = (xf - m[:, None]) * s
        e = u.exp()
        t = e.sum(1)
        z = t.log()
        h = z - torch.where(e > 0, u * e, 0.0).sum(1) / t
        y = labels[r:r + 2048]
        ok = (y >= 0) & (y < x.shape[1])
        lp = u.gather(1, torch.where(ok, y, 0)[:, None])[:, 0] - z
        parts.append([torch.where(ok, v, 0.0) for v in (lp, m, z, h)])
    return [torch.cat(v) for v in zip(*parts)]


def prepare(case, seed):
    c = dict(case)
    dev = torch.device("cuda:0")
    g = torch.Generator(dev)
    g.manual_seed(seed)
    f32 = dict(dtype=torch.float32, device=dev)
    rand = lambda n: torch.randn(n, generator=g, **f32)  # noqa: E731
    op = c["op"]
    if op in ("logp_fwd", "logp_bwd", "policy_logits"):
        x, labels = _logits(c, g, dev)
        T, V = c["T"], c["V"]
        c |= dict(x=x, labels=labels)
        if op == "logp_fwd":
            c |= dict(logp=torch.empty(T, **f32), stats=torch.empty(T, 2, **f32),
                      ent=torch.empty(T, **f32) if c["entropy"] else None)
            return c
        lp, m, z, h = _stats(x, labels, c["scale"])
        c["dx"] = torch.empty(T, V, dtype=x.dtype, device=dev)
        if op == "logp_bwd":
            c |= dict(stats=torch.stack([m, z], 1).contiguous(), glogp=rand(T) / T,
                      ent=h if c["entropy"] else None,
                      gent=rand(T) / T if c["entropy"] else None)
            return c
        live = labels >= 0
        c |= dict(weight=live / live.sum().float(), adv=rand(T) + 0.2, ent_coef=ENT,
                  old=lp - _ratios(T, g), ref=lp + rand(T) * 0.2,
                  out=torch.empty(4, **f32), logp=torch.empty(T, **f32))
        if c["kind"] == "nll":                      # a supervised step: no advantages, no KL
            c |= dict(adv=None, old=None, ref=None, ent_coef=0.0)
        return c
    if op == "pref":
        n = 2 * c["P"]
        length = np.random.RandomState(seed % (1 << 32)).permutation(_lengths(c))
        cu = np.concatenate([[0], np.cumsum(length)]).astype(np.int64)
        T = int(cu[-1])
        prompt = np.concatenate([np.arange(k) < k // 4 for k in length])
        lp = -(rand(T).abs() * 1.5)
        chosen = torch.arange(T, device=dev) < int(cu[c["P"]])
        c |= dict(T=T, cu=torch.from_numpy(cu).to(dev),
                  mask=torch.from_numpy((~prompt).astype(np.uint8)).to(dev), logp=lp,
                  reflp=lp + rand(T) * 0.05 - 0.0005 * chosen if c["ref"] else None,
                  loss=torch.empty(1, **f32), rewards=torch.empty(n, **f32),
                  dlogp=torch.empty(T, **f32))
        return c
    if op == "policy":
        T = c["T"]
        w = torch.from_numpy(~_unscored(T, 0.125)).to(dev)
        lp = -(rand(T).abs() * 1.5)
        c |= dict(logp=lp, weight=w / w.sum().float(), out=torch.empty(4, **f32),
                  adv=rand(-(-T // BLOCK)).repeat_interleave(BLOCK)[:T].contiguous() + 0.2,
                  old=lp - _ratios(T, g, c["dual"]), ref=lp + rand(T) * 0.2,
                  dlogp=torch.empty(T, **f32), ent_coef=ENT if c["entropy"] else 0.0,
                  ent=rand(T).abs() + 1.0 if c["entropy"] else None,
                  dent=torch.empty(T, **f32) if c["entropy"] else None)
        if c["kind"] == "nll":
            c |= dict(old=None)
        return c
    x = rand(c["rows"] * c["cols"]).view(c["rows"], c["cols"]).to(_dtype(c))
    res = rand(x.numel()).view_as(x).to(x.dtype) if c["residual"] else None
    c |= dict(x=x, res=res, y=torch.empty_like(x), seed=1234567890123 + seed, counter=seed % 1000)
    return c


# -------------------------------------------------------------- plain forms

def _plain_logp_fwd(c):
    x, y, s = c["x"].float(), c["labels"], c["scale"]
    ok = (y >= 0) & (y < c["V"])
    m = x.amax(1)
    u = (x - m[:, None]) * s
    e = u.exp()
    t = e.sum(1)
    z = t.log()
    lp = u.gather(1, torch.where(ok, y, 0)[:, None])[:, 0] - z
    out = dict(logp=torch.where(ok, lp, 0.0),
               stats=torch.where(ok[:, None], torch.stack([m, z], 1), 0.0))
    if c["entropy"]:
        h = z - torch.where(e > 0, u * e, 0.0).sum(1) / t
        out["entropy"] = torch.where(ok, h, 0.0)
    return out


def _plain_dlogits(x, y, s, m, z, h, g, ge, dt):
    """s (g (1[y] - p) - ge p (log p + H)), zero rows where y is not scored."""
    V = x.shape[1]
    ok = (y >= 0) & (y < V)
    lp = (x.float() - m[:, None]) * s - z[:, None]
    p = lp.exp()
    d = -g[:, None] * p
    d[torch.arange(len(y), device=y.device), torch.where(ok, y, 0)] += g
    if ge is not None:
        d = d - ge[:, None] * torch.where(p > 0, p * (lp + h[:, None]), 0.0)
    return torch.where(ok[:, None], d * s, 0.0).to(dt)


def _plain_policy(logp, h, w, adv, old, ref, kind, dual, ent_coef):
    """(out[4], dlogp, dentropy) of the token objective."""
    one = torch.ones_like(logp)
    a = one if adv is None else adv
    if kind == "nll":
        surr, dsurr, clipped = a * logp, a, 0.0 * one
    else:
        d = torch.zeros_like(logp) if old is None else logp - old
        lo, hi = (float(np.float32(math.log1p(float(np.float32(v))))) for v in (-CLIP_LO, CLIP_HI))
        r = d.exp()
        above, below = (d > hi) & (a > 0), (d < lo) & (a < 0)
        surr = torch.where(above, (1 + CLIP_HI) * a, torch.where(below, (1 - CLIP_LO) * a, r * a))
        off = above | below
        if dual:
            far = (d > float(np.float32(math.log(dual)))) & (a < 0)
            surr = torch.where(far, dual * a, surr)
            off = off | far
        dsurr = torch.where(off, 0.0, r * a)
        clipped = off.float()
    loss, dlp = -surr, -dsurr
    kl = 0.0 * one
    if ref is not None:
        k = ref - logp
        kl = k.exp() - k - 1
        loss = loss + KL * kl
        dlp = dlp + KL * (1 - k.exp())
    hh = 0.0 * one if h is None else h
    loss = loss - ent_coef * hh
    on = w != 0
    terms = torch.stack([loss, kl, clipped, hh])
    out = torch.where(on, w * terms, 0.0).sum(1)
    return out, torch.where(on, w * dlp, 0.0), torch.where(on, -ent_coef * w, 0.0)


def _plain_pref(c):
    cu, lp, P, T = c["cu"], c["logp"], c["P"], c["T"]
    on = c["mask"] != 0
    d = torch.where(on, lp if c["reflp"] is None else lp - c["reflp"], 0.0)
    at = cu[:-1, None] + torch.arange(c["longest"], device=cu.device)[None]
    inside = at < cu[1:, None]
    at = torch.where(inside, at, 0)
    total = torch.where(inside, d[at], 0.0).sum(1)
    count = (inside & on[at]).sum(1).clamp(min=1).float()
    if c["average"]:
        total = total / count
    h = total[:P] - total[P:]
    beta = BETA[c["kind"]]
    if c["kind"] == "sigmoid":
        zz = beta * h - MARGIN
        soft = lambda v: v.clamp(min=0) + (-v.abs()).exp().log1p()  # noqa: E731
        loss = (1 - SMOOTHING) * soft(-zz) + SMOOTHING * soft(zz)
        dh = beta * (SMOOTHING - 1 / (1 + zz.exp()))
    else:
        e = h - 1 / (2 * beta)
        loss, dh = e * e, 2 * e
    coef = torch.cat([dh, -dh]) / P
    if c["average"]:
        coef = coef / count
    seq = torch.bucketize(torch.arange(T, device=cu.device), cu[1:], right=True)
    return dict(loss=loss.sum()[None] / P, rewards=beta * total,
                dlogp=torch.where(on, coef[seq], 0.0))


def _plain_keep(rows, cols, p, seed, counter, dev):
    """Philox4x32-10 in 64-bit integers: 8 elements of a row to a block, 16
    bits each; kept where they reach round(65536 p)."""
    groups = (cols + 7) // 8
    n = torch.arange(rows * groups, dtype=torch.int64, device=dev)
    low = 0xFFFFFFFF
    a, b = n & low, n >> 32
    cc = torch.full_like(n, counter & low)
    d = torch.full_like(n, (counter >> 32) & low)
    k0, k1 = seed & low, (seed >> 32) & low
    for _ in range(10):
        u, v = a * 0xD2511F53, cc * 0xCD9E8D57
        a, b, cc, d = ((v >> 32) & low) ^ b ^ k0, v & low, ((u >> 32) & low) ^ d ^ k1, u & low
        k0, k1 = (k0 + 0x9E3779B9) & low, (k1 + 0xBB67AE85) & low
    w = torch.stack([a, b, cc, d], 1)
    h = torch.stack([w & 0xFFFF, w >> 16], 2).view(rows, groups * 8)[:, :cols]
    return h >= math.floor(p * 65536 + 0.5)


def _plain_dropout(c):
    keep = _plain_keep(c["rows"], c["cols"], c["p"], c["seed"], c["counter"], c["x"].device)
    drop = math.floor(c["p"] * 65536 + 0.5)
    y = torch.where(keep, c["x"].float() * (65536 / (65536 - drop)), 0.0)
    return (y if c["res"] is None else c["res"].float() + y).to(c["x"].dtype)


def _plain(c):
    op = c["op"]
    if op == "logp_fwd":
        return _plain_logp_fwd(c)
    if op == "logp_bwd":
        m, z = c["stats"].unbind(1)
        return _plain_dlogits(c["x"], c["labels"], c["scale"], m, z, c["ent"], c["glogp"],
                              c["gent"], c["x"].dtype)
    if op == "policy_logits":
        x, y, s = c["x"], c["labels"], c["scale"]
        f = _plain_logp_fwd(dict(c, entropy=True))
        w = torch.where((y >= 0) & (y < c["V"]), c["weight"], 0.0)
        out, g, ge = _plain_policy(f["logp"], f["entropy"], w, c["adv"], c["old"], c["ref"],
                                   c["kind"], 0.0, c["ent_coef"])
        m, z = f["stats"].unbind(1)
        dx = _plain_dlogits(x, y, s, m, z, f["entropy"], g, ge, x.dtype)
        return dict(out=out, logp=f["logp"], dlogits=dx)
    if op == "policy":
        out, g, ge = _plain_policy(c["logp"], c["ent"], c["weight"], c["adv"], c["old"], c["ref"],
                                   c["kind"], c["dual"], c["ent_coef"])
        return dict(out=out, dlogp=g, **(dict(dentropy=ge) if c["entropy"] else {}))
    if op == "pref":
        return _plain_pref(c)
    return _plain_dropout(c)


# ------------------------------------------------------------ the library's

def _ws(c, nbytes):
    """The workspace a training program keeps beside its buffers."""
    if "ws" not in c:
        c["ws"] = torch.empty(max(nbytes, 16), dtype=torch.uint8, device="cuda:0")
        c["ws_bytes"] = nbytes
    return c["ws"], c["ws_bytes"]


def _library(c):
    from quantized_rank_fine_amd import qlora as q
    op = c["op"]
    if op in ("logp_fwd", "logp_bwd", "policy_logits"):
        x, T, V = c["x"], c["T"], c["V"]
        dt = q.BF16 if c["dt"] == "bf16" else q.F32
    if op == "logp_fwd":
        ws = _ws(c, q.qlora_token_logp_workspace_bytes(T, V, dt))
        q.qlora_token_logp_fwd(x, c["ld"], T, V, dt, c["labels"], c["scale"], c["logp"],
                               c["stats"], c["ent"], *ws)
        out = dict(logp=c["logp"], stats=c["stats"])
        if c["entropy"]:
            out["entropy"] = c["ent"]
        return out
    if op == "logp_bwd":
        q.qlora_token_logp_bwd(x, c["ld"], T, V, dt, c["labels"], c["scale"], c["stats"],
                               c["ent"], c["glogp"], c["gent"], c["dx"], V)
        return c["dx"]
    if op == "policy_logits":
        ws = _ws(c, q.qlora_policy_logits_workspace_bytes(T, V, dt))
        pol = q.policy_struct(q.OBJ_NLL if c["kind"] == "nll" else q.OBJ_CLIP, CLIP_LO, CLIP_HI,
                              0.0, KL, c["ent_coef"])
        q.qlora_policy_logits(x, c["ld"], T, V, dt, c["labels"], c["scale"], c["weight"],
                              c["adv"], c["old"], c["ref"], pol, c["out"], c["logp"], c["dx"], V,
                              *ws)
        return dict(out=c["out"], logp=c["logp"], dlogits=c["dx"])
    if op == "policy":
        ws = _ws(c, q.qlora_policy_workspace_bytes(c["T"]))
        pol = q.policy_struct(q.OBJ_NLL if c["kind"] == "nll" else q.OBJ_CLIP, CLIP_LO, CLIP_HI,
                              c["dual"], KL, c["ent_coef"])
        q.qlora_policy_loss(c["logp"], c["ent"], c["T"], c["weight"], c["adv"], c["old"],
                            c["ref"], pol, c["out"], c["dlogp"], c["dent"], *ws)
        return dict(out=c["out"], dlogp=c["dlogp"],
                    **(dict(dentropy=c["dent"]) if c["entropy"] else {}))
    if op == "pref":
        ws = _ws(c, q.qlora_pref_workspace_bytes(c["P"], c["T"]))
        kind = q.PREF_SIGMOID if c["kind"] == "sigmoid" else q.PREF_SQUARED
        pref = q.pref_struct(kind, BETA[c["kind"]], MARGIN, SMOOTHING, c["average"])
        q.qlora_pref_loss(c["logp"], c["reflp"], c["mask"], c["cu"], c["P"], c["T"], pref,
                          c["loss"], c["rewards"], c["dlogp"], *ws)
        return dict(loss=c["loss"], rewards=c["rewards"], dlogp=c["dlogp"])
    dt = q.BF16 if c["dt"] == "bf16" else q.F32
    cols = c["cols"]
    q.qlora_dropout(c["x"], cols, c["res"], cols, c["rows"], cols, dt, c["p"], c["seed"],
                    c["counter"], c["y"], cols)
    return c["y"]


def run(state):
    return _library(state) if own else _plain(state)


# --------------------------------------------------------------------- work

def work(case):
    c, op = case, case["op"]
    if op in ("logp_fwd", "logp_bwd", "policy_logits"):
        T, V, size = c["T"], c["V"], 2 if c["dt"] == "bf16" else 4
        live = T - int(_unscored(T, c["prompt"]).sum())
        ent = c.get("entropy", True)
        read = live * V * size + 8 * T
        if op == "logp_fwd":
            return dict(bytes=read + T * (12 + 4 * ent), flops=live * V * (4 + 2 * ent))
        wrote = T * V * size
        if op == "logp_bwd":
            return dict(bytes=read + wrote + T * (12 + 8 * ent), flops=live * V * (5 + 3 * ent))
        rows = 4 + 4 * (1 if c["kind"] == "nll" else 4)     # logp; weight, adv, old, ref
        return dict(bytes=read + wrote + T * rows + 16, flops=live * V * 12)
    if op == "pref":
        T = int(_lengths(c).sum())
        return dict(bytes=T * (4 + 4 * c["ref"] + 1 + 4), flops=3 * T)
    if op == "policy":
        arrays = 5 + (c["kind"] == "clip") + 2 * c["entropy"]
        return dict(bytes=4 * arrays * c["T"] + 16, flops=20 * c["T"])
    n, size = c["rows"] * c["cols"], 2 if c["dt"] == "bf16" else 4
    return dict(bytes=n * size * (2 + c["residual"]), flops=n * (2 + c["residual"]))


# -------------------------------------------------------------------- exact

def _exact_policy(lp, h, w, adv, old, ref, kind, dual, ent_coef):
    a = torch.ones_like(lp) if adv is None else adv.double()
    if kind == "nll":
        obj, slope, off = a * lp, a, torch.zeros_like(lp)
    else:
        r = torch.exp(lp - old.double())
        bound = torch.clamp(r, 1 - CLIP_LO, 1 + CLIP_HI) * a
        obj = torch.minimum(r * a, bound)
        free = r * a <= bound
        if dual:
            free = free & ~((a < 0) & (obj < dual * a))
            obj = torch.where(a < 0, torch.maximum(obj, dual * a), obj)
        slope, off = torch.where(free, r * a, 0.0), (~free).double()
    kl, dkl = torch.zeros_like(lp), torch.zeros_like(lp)
    if ref is not None:
        q = ref.double() - lp
        kl, dkl = torch.expm1(q) - q, -torch.expm1(q)
    hh = torch.zeros_like(lp) if h is None else h
    w = w.double()
    out = torch.stack([(w * (-obj + KL * kl - ent_coef * hh)).sum(), (w * kl).sum(),
                       (w * off).sum(), (w * hh).sum()])
    return out, w * (-slope + KL * dkl), -ent_coef * w


def exact(case, seed):
    c = prepare(case, seed)
    op = c["op"]
    if op in ("logp_fwd", "logp_bwd", "policy_logits"):
        T, V, s = c["T"], c["V"], c["scale"]
        y, live = c["labels"], c["labels"] >= 0
        want, lp, m, z, h = [], [], [], [], []
        step = 1024
        for r in range(0, T, step):
            x = c["x"][r:r + step].double()
            logs = torch.log_softmax(x * s, 1)
            ent = -torch.special.xlogy(logs.exp(), logs.exp()).sum(1)
            top = x.amax(1)
            yy = y[r:r + step].clamp(min=0)
            on = live[r:r + step].double()
            lp.append(logs.gather(1, yy[:, None])[:, 0] * on)
            m.append(top * on)
            z.append((torch.logsumexp(x * s, 1) - s * top) * on)
            h.append(ent * on)
        lp, m, z, h = (torch.cat(v) for v in (lp, m, z, h))
        if op == "logp_fwd":
            out = dict(logp=lp, stats=torch.stack([m, z], 1))
            if c["entropy"]:
                out["entropy"] = h
            return out
        if op == "logp_bwd":
            g, ge = c["glogp"].double(), c["gent"]
            ge = None if ge is None else ge.double()
        else:
            out, g, ge = _exact_policy(lp, h, c["weight"] * live, c["adv"], c["old"], c["ref"],
                                       c["kind"], 0.0, c["ent_coef"])
        dx = torch.empty(T, V, dtype=torch.float64, device=y.device)
        for r in range(0, T, step):
            logs = torch.log_softmax(c["x"][r:r + step].double() * s, 1)
            p = logs.exp()
            hot = torch.zeros_like(p).scatter_(1, y[r:r + step].clamp(min=0)[:, None], 1.0)
            v = g[r:r + step, None] * (hot - p)
            if ge is not None:
                v -= ge[r:r + step, None] * (torch.special.xlogy(p, p) + p * h[r:r + step, None])
            dx[r:r + step] = v * s * live[r:r + step, None]
        return dx if op == "logp_bwd" else dict(out=out, logp=lp, dlogits=dx)
    if op == "policy":
        ent = None if c["ent"] is None else c["ent"].double()
        out, g, ge = _exact_policy(c["logp"].double(), ent, c["weight"], c["adv"], c["old"],
                                   c["ref"], c["kind"], c["dual"], c["ent_coef"])
        return dict(out=out, dlogp=g, **(dict(dentropy=ge) if c["entropy"] else {}))
    if op == "pref":
        cu = c["cu"].cpu().numpy()
        lp = c["logp"].cpu().numpy().astype(np.float64)
        if c["reflp"] is not None:
            lp = lp - c["reflp"].cpu().numpy()
        on = c["mask"].cpu().numpy() != 0
        P, beta = c["P"], BETA[c["kind"]]
        span = [slice(int(a), int(b)) for a, b in zip(cu[:-1], cu[1:])]
        count = np.array([on[k].sum() for k in span])
        total = np.array([lp[k][on[k]].sum() for k in span])
        if c["average"]:
            total = total / np.maximum(count, 1)
        h = total[:P] - total[P:]
        if c["kind"] == "sigmoid":
            v = beta * h - MARGIN
            loss = (1 - SMOOTHING) * np.logaddexp(0, -v) + SMOOTHING * np.logaddexp(0, v)
            dh = beta * (1 / (1 + np.exp(-v)) - (1 - SMOOTHING))
        else:
            loss, dh = (h - 0.5 / beta) ** 2, 2 * h - 1 / beta
        coef = np.concatenate([dh, -dh]) / P
        if c["average"]:
            coef = coef / np.maximum(count, 1)
        grad = np.zeros(c["T"])
        for i, k in enumerate(span):
            grad[k] = coef[i] * on[k]
        return dict(loss=np.array([loss.mean()]), rewards=beta * total, dlogp=grad)
    rows, cols, drop = c["rows"], c["cols"], int(c["p"] * 65536 + 0.5)
    groups = -(-cols // 8)
    u = np.uint64
    n = np.arange(rows * groups, dtype=np.uint64)
    word = [n & u(0xFFFFFFFF), n >> u(32), np.full_like(n, c["counter"]), np.zeros_like(n)]
    key = [c["seed"] % (1 << 32), c["seed"] >> 32]
    for _ in range(10):
        lo, hi = word[0] * u(0xD2511F53), word[2] * u(0xCD9E8D57)
        word = [(hi >> u(32)) ^ word[1] ^ u(key[0]), hi & u(0xFFFFFFFF),
                (lo >> u(32)) ^ word[3] ^ u(key[1]), lo & u(0xFFFFFFFF)]
        key = [(key[0] + 0x9E3779B9) % (1 << 32), (key[1] + 0xBB67AE85) % (1 << 32)]
    bits = np.stack(word, 1).astype("<u4").view("<u2").reshape(rows, groups * 8)[:, :cols]
    y = c["x"].double() * torch.from_numpy((bits >= drop) / (1 - drop / 65536)).to(c["x"].device)
    return y if c["res"] is None else y + c["res"].double()
