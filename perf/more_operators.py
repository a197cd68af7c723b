"""The operators of a step that distils a model into an adapted 4-bit one, as
measured cases: the linear with bias, activation, factor and residual in its
epilogue and that epilogue's gradient; log-probabilities with the top
alternatives; the loss against a teacher's stored alternatives; and the
orthogonalised update of the adapters.

``listed()`` names the cases, ``draw()`` gives more of the same ranges,
``prepare()`` makes a case's inputs on the GPU from a seed, ``run()`` is one
call and ``work()`` what that call has to move and compute.  With ``own``
false, ``run()`` computes the operators in plain 32-bit torch operations;
with ``own`` true it calls the library.  ``exact()`` gives the results in 64
bits from the definitions.

Definitions (deq is the 4-bit weight's value in bf16, as the library expands
it for its products; s the inverse temperature, log p the log-softmax of s x):

  linear   z = X deq(Wq) + c (X A) B + bias,  y = residual + act(z) mul
  its end  dZ = dY mul act'(Z),  dmul = dY act(Z),  dbias = column sums of dZ
  top      the k largest logits of a row, ties to the lower index, their
           log p, the label's log p and the entropy
  distill  q_j = exp(t_j) / sum exp(t),  kl = sum q_j (ln q_j - log p_j),
           loss = sum w kl,  dx_v = w s (p_v - sum_{j: i_j = v} q_j)
  muon     m <- mu m + g,  u = g + mu m,  X = u / (|u| + eps),  five times
           X <- a X + b X (X^T X) + c X (X^T X)^2 on the smaller side,
           theta <- theta - lr (scale X + wd theta)
"""

import math

import numpy as np
import torch

own = False

IGNORE = -100
BLOCK = 64          # prompts are laid out in runs of this many tokens
PAD = 32            # masked vocabulary entries at the end of a row
LORA_SCALE = 2.0    # alpha / r
MU, LR, WD, EPS = 0.95, 0.02, 0.01, 1e-7
NS = (3.4445, -4.7750, 2.0315)


# ------------------------------------------------------------------- cases

def listed():
    return [
        # one decoded token through a block's last projection, back into the
        # residual stream
        dict(name="down-one-token", op="linear", M=1, n_in=11008, n_out=4096, r=16, act="none",
             bias=False, mul=False, res=True, z=False),
        # a training batch through the gate projection: act(gate) up in one
        # call, with what the backward needs
        dict(name="gate-batch", op="linear", M=2048, n_in=4096, n_out=11008, r=16, act="silu",
             bias=False, mul=True, res=False, z=True),
        # an odd number of tokens through a biased layer with GELU
        dict(name="gelu-odd", op="linear", M=777, n_in=1600, n_out=6400, r=64, act="gelu_tanh",
             bias=True, mul=False, res=False, z=True),
        # the gradient of the gate's epilogue
        dict(name="gate-batch-grad", op="end", M=2048, n_out=11008, act="silu", mul=True,
             bias=False, dt="bf16"),
        # an odd batch in fp32: exact GELU and the bias's gradient
        dict(name="gelu-odd-f32-grad", op="end", M=509, n_out=4096, act="gelu", mul=False,
             bias=True, dt="f32"),
        # one adapter's update
        dict(name="muon-one", op="muon", L=1, n_in=4096, n_out=4096, r=16, copy=True,
             update=False),
        # the adapters of one projection in 32 layers
        dict(name="muon-layers", op="muon", L=32, n_in=4096, n_out=4096, r=64, copy=True,
             update=False),
        # two adapters of an odd high rank; the orthogonalised updates are
        # asked for too
        dict(name="muon-rank-200", op="muon", L=2, n_in=11008, n_out=4096, r=200, copy=False,
             update=True),
        # one decoded token's alternatives
        dict(name="top-one-token", op="top", T=1, V=32000, ld=32000, dt="bf16", k=20, scale=1.0,
             prompt=0.0, masked=False),
        # a teacher scoring a batch of completions
        dict(name="top-batch", op="top", T=4096, V=32000, ld=32000, dt="bf16", k=32, scale=1.0,
             prompt=0.25, masked=False),
        # fp32 logits of an odd vocabulary in padded rows, masked words, a
        # temperature
        dict(name="distill-odd-f32", op="distill", T=61, V=50001, ld=50016, dt="f32", k=16,
             scale=0.5, prompt=0.0, masked=True),
        # the student's loss and gradient on a batch
        dict(name="distill-batch", op="distill", T=4096, V=32000, ld=32000, dt="bf16", k=32,
             scale=1.0, prompt=0.25, masked=False),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _log_64(rng, lo, hi):
    return max(1, round(_log_int(rng, lo, hi) / 64)) * 64


def draw(rng):
    op = rng.choice(["linear", "linear", "end", "muon", "muon", "top", "distill"])
    if op == "linear":
        M = _log_int(rng, 1, 4096)
        n_in, n_out = _log_64(rng, 256, 11008), _log_64(rng, 256, 11008)
        M = max(1, min(M, 90_000_000_000 // (n_in * n_out)))
        # few tokens: the projections back into the residual stream
        few = M <= 16
        return dict(op=op, M=M, n_in=n_in, n_out=n_out, r=rng.choice([8, 16, 20, 64]),
                    act="none" if few else rng.choice(["none", "relu", "gelu", "gelu_tanh",
                                                       "silu"]),
                    bias=rng.random() < 0.5, mul=not few and rng.random() < 0.4,
                    res=few or rng.random() < 0.3, z=not few and rng.random() < 0.5)
    if op == "end":
        n_out = _log_64(rng, 64, 11008)
        M = max(1, min(_log_int(rng, 1, 8192), 22_000_000 // n_out))
        act = rng.choice(["relu", "gelu", "gelu_tanh", "silu"])
        return dict(op=op, M=M, n_out=n_out, act=act, mul=rng.random() < 0.5,
                    bias=rng.random() < 0.5, dt=rng.choice(["bf16", "bf16", "f32"]))
    if op == "muon":
        r = _log_int(rng, 1, 256)
        n_in, n_out = (max(r, _log_int(rng, 64, 11008)) for _ in range(2))
        L = max(1, min(_log_int(rng, 1, 32), 16_000_000 // ((n_in + n_out) * r),
                       32_000_000 // r ** 3))
        return dict(op=op, L=L, n_in=n_in, n_out=n_out, r=r, copy=rng.random() < 0.5,
                    update=rng.random() < 0.3)
    dt = rng.choice(["bf16", "bf16", "f32"])
    V = _log_int(rng, 1000, 200000)
    T = max(1, min(_log_int(rng, 1, 4096), 130_000_000 // (V * (2 if dt == "f32" else 1))))
    return dict(op=op, T=T, V=V, ld=V + rng.choice([0, 0, 1, 7, 64]), dt=dt,
                k=_log_int(rng, 1, 64), scale=rng.choice([1.0, 1.0, 0.5, 1.25]),
                prompt=rng.choice([0.0, 0.25, 0.5]), masked=rng.random() < 0.3)


# ------------------------------------------------------------------- inputs

def _dtype(c):
    return torch.bfloat16 if c["dt"] == "bf16" else torch.float32


def _unscored(T, prompt):
    """Which of T tokens are prompt (by their place in runs of BLOCK)."""
    return (np.arange(T) % BLOCK) < round(prompt * BLOCK) if T >= BLOCK else np.zeros(T, bool)


def _levels(dev):
    """The 16 levels: normal quantiles at 16 evenly spaced probabilities in
    [0.02, 0.98] over the largest magnitude, in fp32."""
    q = torch.special.ndtri(torch.linspace(0.02, 0.98, 16, dtype=torch.float64))
    return (q / q.abs().max()).float().to(dev)


def _logits(c, g, dev):
    """Logits [T, V] in rows of ld, and labels (IGNORE in prompts)."""
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


def prepare(case, seed):
    c = dict(case)
    dev = torch.device("cuda:0")
    g = torch.Generator(dev)
    g.manual_seed(seed)
    f32 = dict(dtype=torch.float32, device=dev)
    rand = lambda *n: torch.randn(*n, generator=g, **f32)  # noqa: E731
    op = c["op"]
    if op == "linear":
        M, n_in, n_out, r = c["M"], c["n_in"], c["n_out"], c["r"]
        n, bf = n_in * n_out, torch.bfloat16
        c |= dict(codes=torch.randint(0, 256, (n // 2,), generator=g, device=dev,
                                      dtype=torch.uint8),
                  qscale=torch.randint(40, 128, (n // 64,), generator=g, device=dev,
                                       dtype=torch.int8),
                  gscale=0.04 / 84 * (1 + 0.1 * torch.rand((n // 64 + 255) // 256, generator=g,
                                                           **f32)),
                  X=(rand(M, n_in) * 0.5).to(bf), A=(rand(n_in, r) / n_in ** 0.5).to(bf),
                  B=(rand(r, n_out) * 0.02).to(bf), Y=torch.empty(M, n_out, dtype=bf, device=dev),
                  XA=torch.empty(M, r, **f32) if c["z"] else None,
                  Z=torch.empty(M, n_out, dtype=bf, device=dev) if c["z"] else None,
                  b=(rand(n_out) * 0.5).to(bf) if c["bias"] else None,
                  mulv=rand(M, n_out).to(bf) if c["mul"] else None,
                  resv=(rand(M, n_out) * 4).to(bf) if c["res"] else None)
        return c
    if op == "end":
        shape, dt = (c["M"], c["n_out"]), _dtype(c)
        c |= dict(Z=(rand(*shape) * 1.5).to(dt), dY=rand(*shape).to(dt),
                  mulv=rand(*shape).to(dt) if c["mul"] else None,
                  dZ=torch.empty(shape, dtype=dt, device=dev),
                  dmul=torch.empty(shape, dtype=dt, device=dev) if c["mul"] else None,
                  db=torch.empty(c["n_out"], **f32) if c["bias"] else None)
        return c
    if op == "muon":
        L, n_in, n_out, r = c["L"], c["n_in"], c["n_out"], c["r"]
        # few strong directions over a floor, as an adapter's gradients have
        strong = lambda n, m: (rand(L, n, 4) @ rand(L, 4, m) + rand(L, n, m)) * 1e-3  # noqa: E731
        c |= dict(A=rand(L, n_in, r) / n_in ** 0.5, B=rand(L, r, n_out) * 0.02,
                  gA=strong(n_in, r), gB=strong(r, n_out), mA=strong(n_in, r) * 4,
                  mB=strong(r, n_out) * 4)
        for w in "AB":
            like = lambda dt: torch.empty_like(c[w], dtype=dt)  # noqa: E731
            c |= {w + "16": like(torch.bfloat16) if c["copy"] else None,
                  "O" + w: like(torch.float32) if c["update"] else None}
        c |= dict(scaleA=max(1.0, n_in / r) ** 0.5, scaleB=max(1.0, r / n_out) ** 0.5)
        return c
    x, labels = _logits(c, g, dev)
    T, V, k = c["T"], c["V"], c["k"]
    c |= dict(x=x)
    if op == "top":
        c |= dict(labels=labels, ids=torch.empty(T, k, dtype=torch.int32, device=dev),
                  top=torch.empty(T, k, **f32), logp=torch.empty(T, **f32),
                  ent=torch.empty(T, **f32))
        return c
    # a teacher that mostly agrees; a few rows have two alternatives less
    ids, logt = [], []
    for r in range(0, T, 1024):
        y = x[r:r + 1024].float()
        y = y + torch.randn(y.shape, generator=g, device=dev)
        lp = torch.log_softmax(y, 1)
        v, i = torch.topk(lp, k, 1)
        ids.append(i)
        logt.append(v)
    ids, logt = torch.cat(ids).int(), torch.cat(logt)
    if k > 4:
        ids[::8, k - 2:] = -1
    live = (labels >= 0).float()
    c |= dict(ids=ids.contiguous(), logt=logt.contiguous(), weight=live / live.sum().clamp(min=1),
              loss=torch.empty(1, **f32), kl=torch.empty(T, **f32),
              dx=torch.empty(T, V, dtype=x.dtype, device=dev))
    return c


# -------------------------------------------------------------- plain forms

def _plain_weight(c):
    """deq(Wq) [in, out] as the products take it: L[code] (q s2) in fp32,
    rounded to bf16."""
    both = torch.stack([c["codes"] & 15, c["codes"] >> 4], 1).view(-1, 64)
    q = c["qscale"].float()
    s = q * c["gscale"].repeat_interleave(256)[:len(q)]
    w = _levels(q.device)[both.long()] * s[:, None]
    return w.view(c["n_in"], c["n_out"]).to(torch.bfloat16).float()


def _plain_act(z, act):
    """act(z) and act'(z)."""
    if act == "none":
        return z, torch.ones_like(z)
    if act == "relu":
        return z.clamp(min=0), (z > 0).to(z.dtype)
    if act == "silu":
        s = 1 / (1 + (-z).exp())
        return z * s, s * (1 + z * (1 - s))
    if act == "gelu":
        cdf = 0.5 * (1 + torch.erf(z * 0.5 ** 0.5))
        return z * cdf, cdf + z * (-0.5 * z * z).exp() * (0.5 / math.pi) ** 0.5
    k = (2 / math.pi) ** 0.5
    t = torch.tanh(k * (z + 0.044715 * z * z * z))
    return (0.5 * z * (1 + t),
            0.5 * (1 + t) + 0.5 * z * (1 - t * t) * k * (1 + 3 * 0.044715 * z * z))


def _plain_linear(c):
    x = c["X"].float()
    xa = x @ c["A"].float()
    z = x @ _plain_weight(c) + LORA_SCALE * (xa @ c["B"].float())
    if c["bias"]:
        z = z + c["b"].float()
    y = _plain_act(z, c["act"])[0]
    if c["mul"]:
        y = y * c["mulv"].float()
    if c["res"]:
        y = c["resv"].float() + y
    out = dict(Y=y.to(torch.bfloat16))
    if c["z"]:                                      # kept for the backward
        out |= dict(XA=xa, Z=z.to(torch.bfloat16))
    return out


def _plain_end(c):
    f, df = _plain_act(c["Z"].float(), c["act"])
    dy = c["dY"].float()
    dz = dy * df
    out = {}
    if c["mul"]:
        dz = dz * c["mulv"].float()
        out["dmul"] = (dy * f).to(_dtype(c))
    if c["bias"]:
        out["dbias"] = dz.sum(0)
    return dict(out, dZ=dz.to(_dtype(c)))


def _plain_products(X):
    """One Newton-Schulz step of a stack of tall matrices."""
    G = X.transpose(1, 2).contiguous() @ X
    return NS[0] * X + X @ (NS[1] * G + NS[2] * (G @ G))


def _plain_update(c, w):
    """One stack's step; theta and momentum are updated in place."""
    p, g, m = c[w], c["g" + w], c["m" + w]
    m.mul_(MU).add_(g)
    u = g + MU * m
    X = u / (u.square().sum((1, 2), keepdim=True).sqrt() + EPS)
    wide = X.shape[1] < X.shape[2]
    X = X.transpose(1, 2).contiguous() if wide else X
    X = _plain_products(_plain_products(_plain_products(_plain_products(_plain_products(X)))))
    X = X.transpose(1, 2).contiguous() if wide else X
    p.copy_(p - LR * (c["scale" + w] * X + WD * p))
    out = {w: p, "m" + w: m}
    if c["copy"]:
        out[w + "16"] = p.to(torch.bfloat16)
    if c["update"]:
        out["O" + w] = X
    return out


def _plain_logp(x, s):
    """log p [T, V] in 32 bits."""
    u = (x.float() - x.float().amax(1, keepdim=True)) * s
    return u - u.exp().sum(1, keepdim=True).log()


def _plain_top(c):
    x, y, k = c["x"], c["labels"], c["k"]
    on = (y >= 0) & (y < c["V"])
    lp = _plain_logp(x, c["scale"])
    # fp32 bits in the order of the values, then the lower index first
    bits = (x.float() + 0.0).view(torch.int32).long()
    key = torch.where(bits >= 0, bits, bits ^ 0x7FFFFFFF) * (1 << 25)
    key = key + ((1 << 24) - torch.arange(c["V"], device=x.device))
    ids = torch.topk(key, k, 1).indices
    p = lp.exp()
    out = dict(top=lp.gather(1, ids), logp=lp.gather(1, torch.where(on, y, 0)[:, None])[:, 0],
               entropy=-torch.where(p > 0, p * lp, 0.0).sum(1))
    out = {n: torch.where(on[:, None] if v.dim() == 2 else on, v, 0.0) for n, v in out.items()}
    return dict(out, ids=torch.where(on[:, None], ids, -1).int())


def _plain_distill(c):
    x, ids, w, s = c["x"], c["ids"].long(), c["weight"], c["scale"]
    on = (ids >= 0) & (ids < c["V"])
    t = torch.where(on, c["logt"], -math.inf)
    t = t - t.amax(1, keepdim=True)
    t = t - t.exp().sum(1, keepdim=True).log()
    q = t.exp()
    lp = _plain_logp(x, s)
    at = torch.where(on, ids, 0)
    kl = torch.where(q > 0, q * (t - lp.gather(1, at)), 0.0).sum(1)
    kl = torch.where(w != 0, kl, 0.0)
    d = lp.exp().scatter_add_(1, at, -q)
    dx = (d * (s * w)[:, None]).to(x.dtype)
    return dict(loss=(w * kl).sum()[None], kl=kl, dlogits=dx)


def _plain(c):
    op = c["op"]
    if op == "linear":
        return _plain_linear(c)
    if op == "end":
        return _plain_end(c)
    if op == "muon":
        return {**_plain_update(c, "A"), **_plain_update(c, "B")}
    return _plain_top(c) if op == "top" else _plain_distill(c)


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
    acts = dict(none=q.EP_NONE, relu=q.EP_RELU, gelu=q.EP_GELU, gelu_tanh=q.EP_GELU_TANH,
                silu=q.EP_SILU)
    if op == "linear":
        M, r = c["M"], c["r"]
        if "wq" not in c:
            c["wq"] = q.nf4_struct(c["n_in"], c["n_out"], c["codes"], c["qscale"], c["gscale"])
        ws = _ws(c, q.qlora_fwd_workspace_bytes(M, c["n_in"], c["n_out"], r, q.BF16))
        ep = q.epilogue_struct(acts[c["act"]], c["b"], c["mulv"], c["resv"], c["Z"])
        q.qlora_linear_fwd_ep(c["wq"], c["X"], M, q.BF16, c["A"], c["B"], r, q.BF16, LORA_SCALE,
                              0.0, None, ep, c["Y"], c["XA"], *ws)
        out = dict(Y=c["Y"])
        return dict(out, XA=c["XA"], Z=c["Z"]) if c["z"] else out
    if op == "muon":
        if "mats" not in c:
            c["mats"] = q.muon_mats(
                [q.muon_mat(*c[w][i].shape, c["g" + w][i], c["m" + w][i], c[w][i],
                            c[w + "16"][i] if c["copy"] else None,
                            c["O" + w][i] if c["update"] else None, c["scale" + w])
                 for w in "AB" for i in range(c["L"])])
        ws = _ws(c, q.qlora_muon_workspace_bytes(c["mats"]))
        q.qlora_muon_step(c["mats"], LR, *ws, momentum=MU, nesterov=True, weight_decay=WD,
                          eps=EPS, steps=5, coef=NS)
        names = ["A", "B", "mA", "mB"] + (["A16", "B16"] if c["copy"] else [])
        return {n: c[n] for n in names + (["OA", "OB"] if c["update"] else [])}
    dt = q.BF16 if c["dt"] == "bf16" else q.F32
    if op == "end":
        M, n = c["M"], c["n_out"]
        ws = _ws(c, q.qlora_ep_bwd_workspace_bytes(M, n, dt))
        q.qlora_ep_bwd(c["Z"], c["mulv"], c["dY"], M, n, dt, acts[c["act"]], c["dZ"], c["dmul"],
                       c["db"], *ws)
        out = dict(dZ=c["dZ"])
        if c["mul"]:
            out["dmul"] = c["dmul"]
        return dict(out, dbias=c["db"]) if c["bias"] else out
    T, V, k = c["T"], c["V"], c["k"]
    if op == "top":
        ws = _ws(c, q.qlora_token_top_workspace_bytes(T, V, dt, k))
        q.qlora_token_top(c["x"], c["ld"], T, V, dt, c["labels"], c["scale"], k, c["ids"],
                          c["top"], c["logp"], c["ent"], *ws)
        return dict(ids=c["ids"], top=c["top"], logp=c["logp"], entropy=c["ent"])
    ws = _ws(c, q.qlora_distill_workspace_bytes(T, V, dt, k))
    q.qlora_distill_logits(c["x"], c["ld"], T, V, dt, c["scale"], c["weight"], k, c["ids"],
                           c["logt"], True, c["loss"], c["kl"], c["dx"], V, *ws)
    return dict(loss=c["loss"], kl=c["kl"], dlogits=c["dx"])


def run(state):
    return _library(state) if own else _plain(state)


# --------------------------------------------------------------------- work

def work(case):
    c, op = case, case["op"]
    if op == "linear":
        M, n, m, r = c["M"], c["n_in"], c["n_out"], c["r"]
        weight = n * m // 2 + n * m // 64 + 4 * ((n * m // 64 + 255) // 256)
        acts = M * n + M * m * (1 + c["mul"] + c["res"] + c["z"]) + r * (n + m) + m * c["bias"]
        return dict(bytes=weight + 2 * acts + 4 * M * r * c["z"],
                    flops=2 * M * (n * m + r * (n + m)))
    if op == "end":
        size = 2 if c["dt"] == "bf16" else 4
        n = c["M"] * c["n_out"]
        return dict(bytes=n * size * (3 + 2 * c["mul"]) + 4 * c["n_out"] * c["bias"],
                    flops=n * (10 + 2 * c["mul"] + c["bias"]))
    if op == "muon":
        r, L = c["r"], c["L"]
        n = L * r * (c["n_in"] + c["n_out"])
        # the Gram matrix and the last product of each matrix (the iterations
        # act on the r x r matrix: five squares, and with the next Gram
        # matrix 12 products more)
        return dict(bytes=n * (20 + 2 * c["copy"] + 4 * c["update"]),
                    flops=n * (3 * r + 8) + 2 * L * 17 * r * r * r)
    T, V, k, size = c["T"], c["V"], c["k"], 2 if c["dt"] == "bf16" else 4
    live = T - int(_unscored(T, c["prompt"]).sum())
    if op == "top":
        return dict(bytes=live * V * size + T * (8 + 8 + 8 * k), flops=live * V * 7)
    return dict(bytes=live * V * size + T * V * size + T * 8 + live * 8 * k + 4,
                flops=live * V * 9)


# -------------------------------------------------------------------- exact

def _exact_linear(c):
    dev = c["X"].device
    codes = c["codes"].cpu().numpy()
    lv = torch.special.ndtri(torch.linspace(0.02, 0.98, 16, dtype=torch.float64)).numpy()
    lv = (lv / abs(lv).max()).astype(np.float32)
    w = np.empty(2 * len(codes), np.float32)
    w[0::2], w[1::2] = lv[codes % 16], lv[codes // 16]
    q = c["qscale"].cpu().numpy().astype(np.float32)
    s = q * np.repeat(c["gscale"].cpu().numpy(), 256)[:len(q)]
    w *= np.repeat(s, 64)                           # one rounding to fp32, then one to bf16
    W = torch.from_numpy(w).to(dev).view(c["n_in"], c["n_out"]).bfloat16().double()
    X = c["X"].double()
    xa = X @ c["A"].double()
    z = torch.addmm(LORA_SCALE * xa @ c["B"].double(), X, W)
    if c["bias"]:
        z += c["b"].double()
    y = _exact_act(z, c["act"])[0]
    if c["mul"]:
        y = y * c["mulv"].double()
    if c["res"]:
        y = y + c["resv"].double()
    return dict(Y=y, **(dict(XA=xa, Z=z) if c["z"] else {}))


def _exact_act(z, act):
    """The published definitions and their derivatives, the tails without
    cancellation."""
    if act == "none":
        return z, torch.ones_like(z)
    if act == "relu":
        return torch.relu(z), (z > 0).double()
    if act == "silu":
        s = torch.sigmoid(z)
        return z * s, s + z * s * torch.sigmoid(-z)
    if act == "gelu":
        cdf = torch.special.ndtr(z)
        return z * cdf, cdf + z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)
    k = math.sqrt(8 / math.pi)                      # (1 + tanh v) / 2 = sigmoid(2 v)
    s = torch.sigmoid(k * (z + 0.044715 * z ** 3))
    return z * s, s + z * s * (1 - s) * k * (1 + 0.134145 * z * z)


def _exact_update(c, w):
    """f(X) through the eigenvectors of the small Gram matrix: each singular
    value v goes five times through a v + b v^3 + c v^5."""
    g, m, p = c["g" + w].double(), c["m" + w].double(), c[w].double()
    m = MU * m + g
    u = g + MU * m
    tall = u if u.shape[1] >= u.shape[2] else u.mT
    norm = torch.linalg.matrix_norm(u) + EPS
    e, vec = np.linalg.eigh((tall.mT.contiguous() @ tall).cpu().numpy())
    lam = np.maximum(e, 0) / norm.cpu().numpy()[:, None] ** 2
    factor = np.ones_like(lam)
    for _ in range(5):
        step = NS[0] + NS[1] * lam + NS[2] * lam ** 2
        factor, lam = factor * step, lam * step ** 2
    mid = torch.from_numpy((vec * factor[:, None, :]) @ vec.transpose(0, 2, 1)).to(u.device)
    X = tall @ mid / norm[:, None, None]
    X = X if u.shape[1] >= u.shape[2] else X.mT.contiguous()
    p = p * (1 - LR * WD) - LR * c["scale" + w] * X
    out = {w: p, "m" + w: m}
    if c["copy"]:
        out[w + "16"] = p
    if c["update"]:
        out["O" + w] = X
    return out


def exact(case, seed):
    c = prepare(case, seed)
    op = c["op"]
    if op == "linear":
        return _exact_linear(c)
    if op == "end":
        f, df = _exact_act(c["Z"].double(), c["act"])
        dz = df * c["dY"].double()
        out = {}
        if c["mul"]:
            dz = dz * c["mulv"].double()
            out["dmul"] = f * c["dY"].double()
        if c["bias"]:
            out["dbias"] = dz.sum(0)
        return dict(out, dZ=dz)
    if op == "muon":
        return {**_exact_update(c, "A"), **_exact_update(c, "B")}
    T, s, step, parts = c["T"], c["scale"], 512, []
    dx = torch.empty(T, c["V"], dtype=torch.float64, device="cuda:0") if op == "distill" else None
    for r in range(0, T, step):
        x = c["x"][r:r + step].double()
        logs = torch.log_softmax(x * s, 1)
        if op == "top":
            y = c["labels"][r:r + step]
            live = (y >= 0).double()
            ids = torch.sort(x, dim=1, descending=True, stable=True).indices[:, :c["k"]]
            ent = -torch.special.xlogy(logs.exp(), logs.exp()).sum(1)
            parts.append((torch.where(live[:, None] > 0, ids, -1),
                          torch.where(live[:, None] > 0, logs.gather(1, ids), 0.0),
                          logs.gather(1, y.clamp(min=0)[:, None])[:, 0] * live, ent * live))
            continue
        ids, w = c["ids"][r:r + step].long(), c["weight"][r:r + step].double()
        t = c["logt"][r:r + step].double().masked_fill(ids < 0, -math.inf)
        q = torch.softmax(t, 1)
        at = ids.clamp(min=0)
        cross = torch.where(q > 0, q * logs.gather(1, at), 0.0).sum(1)
        kl = (torch.special.xlogy(q, q).sum(1) - cross) * (w > 0)
        hot = torch.zeros_like(logs).scatter_add_(1, at, q)
        dx[r:r + step] = s * w[:, None] * (logs.exp() - hot)
        parts.append((kl, kl * w))
    cat = [torch.cat(v) for v in zip(*parts)]
    if op == "top":
        return dict(ids=cat[0], top=cat[1], logp=cat[2], entropy=cat[3])
    return dict(loss=cat[1].sum()[None], kl=cat[0], dlogits=dx)
