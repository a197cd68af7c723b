"""The objectives at the sizes where another kernel takes over, or a loop runs
a second time: widths that exactly fill a workgroup's registers and those
beside them, more rows than the sum of terms takes at once, more tokens than
the policy loss's grid."""

import numpy as np
import pytest

from oracle import objective as ob
from quantized_rank_fine_amd import qlora as q

import test_gpu_objective as o
from gpu_harness import out_to_f64, say, torch_dev
from test_gpu_objective import U, _dev, _policy_inputs, _policy_logits, _rows, _token_tol, f32

pytestmark = pytest.mark.gpu

WIDTHS = [  # T, V, ld, dt, s, elements before the first row
    (2, 2048, 2048, "bf16", 1.0, 0), (3, 2048, 2050, "f32", 1.25, 1),
    (2, 4096, 4096, "f32", 1.0, 0), (3, 4097, 4097, "bf16", 0.7, 2),
    (3, 6001, 6001, "bf16", 1.0, 1), (2, 6000, 6000, "f32", 1.0, 0),
    (2, 8192, 8192, "bf16", 1.0, 0), (2, 8192, 8192, "f32", 1.0, 3),
    (5, 8193, 8195, "bf16", 1.25, 0), (3, 8193, 8193, "f32", 1.0, 1),
    (5, 12001, 12001, "bf16", 1.0, 3), (2, 12000, 12000, "f32", 1.25, 0),
    (2, 16384, 16384, "bf16", 1.0, 0), (2, 16384, 16384, "f32", 1.0, 0),
    (3, 16385, 16385, "bf16", 1.0, 5), (2, 32768, 32768, "bf16", 1.0, 0),
    (2, 32768, 32768, "f32", 1.0, 1), (3, 32769, 32769, "bf16", 1.0, 0),
    (2, 32769, 32776, "f32", 1.0, 0), (2, 65536, 65536, "bf16", 1.0, 0),
    (2, 65536, 65536, "f32", 1.0, 0), (2, 65536, 65536, "bf16", 1.0, 1),
    (2, 65537, 65537, "bf16", 1.0, 0), (66, 65537, 65537, "bf16", 1.0, 1),
    (65, 65537, 65544, "f32", 1.0, 0),
]


@pytest.mark.parametrize("T,V,ld,dt,s,at", WIDTHS)
@pytest.mark.parametrize("ent", [True, False])
def test_logp_at_the_edges(T, V, ld, dt, s, at, ent):
    o.test_logp_forward_and_gradient(T, V, ld, dt, s, at, ent)


@pytest.mark.parametrize("T,V,ld,dt,s,at", WIDTHS)
@pytest.mark.parametrize("kind,ent", [("clip", 0.02), ("clip", 0.0), ("nll", 0.0)])
def test_policy_logits_at_the_edges(T, V, ld, dt, s, at, kind, ent):
    o.test_policy_logits(T, V, ld, dt, s, at, kind, ent)


def _clip(c, lo, hi, dual, kl, ent):
    """(out, dlogp, dentropy) of all tokens at once, in float64."""
    a, w = c["adv"].astype(float), c["weight"].astype(float)
    r = np.exp(c["logp"].astype(float) - c["old"])
    f = np.minimum(r * a, np.clip(r, 1 - lo, 1 + hi) * a)
    if dual:
        f = np.where(a < 0, np.maximum(f, dual * a), f)
    bound = f != r * a
    v = c["ref"].astype(float) - c["logp"]
    k, h = np.expm1(v) - v, c["entropy"].astype(float)
    out = np.array([(w * (-f + kl * k - ent * h)).sum(), (w * k).sum(), (w * bound).sum(),
                    (w * h).sum()])
    return out, w * (-np.where(bound, 0.0, r * a) - kl * np.expm1(v)), -w * ent


@pytest.mark.parametrize("T", [8192, 8193, 2097152, 2097153, 2100003, 4194311])
def test_policy_loss_of_more_tokens_than_the_grid(T):
    """2048 workgroups take 1024 tokens each at a time."""
    torch, dev = torch_dev()
    say(f"[policy long] T={T}")
    lo, hi, dual, kl, ent = f32(0.2), f32(0.28), 3.0, f32(0.04), f32(0.01)
    c = _policy_inputs(T, T, dual)
    some = {k: v[-300:] for k, v in c.items()}           # the oracle's own, of the last tokens
    ref = ob.policy_loss("clip", *[some[k] for k in ("logp", "entropy", "weight", "adv", "old",
                                                     "ref")], lo, hi, dual, kl, ent)
    for got, want in zip(_clip(some, lo, hi, dual, kl, ent), ref):
        assert np.allclose(got, want, rtol=1e-12, atol=1e-18)
    ro, rg, rh = _clip(c, lo, hi, dual, kl, ent)
    t = {k: _dev(v) for k, v in c.items()}
    out = torch.full((4,), 9.0, device=dev)
    d, dh = torch.full((T + 1,), 9.0, device=dev), torch.full((T + 1,), 9.0, device=dev)
    n = q.qlora_policy_workspace_bytes(T)
    ws = torch.empty(n, dtype=torch.uint8, device=dev) if n else None
    q.qlora_policy_loss(t["logp"], t["entropy"], T, t["weight"], t["adv"], t["old"], t["ref"],
                        q.policy_struct(q.OBJ_CLIP, lo, hi, dual, kl, ent), out, d, dh, ws, n)
    gd, gh = d.cpu().numpy().astype(float), dh.cpu().numpy().astype(float)
    assert gd[-1] == 9.0 and gh[-1] == 9.0
    w = c["weight"].astype(float)
    tl, tg, tk = _token_tol(c, kl, ent)
    assert np.all(np.abs(gd[:-1] - rg) <= w * tg + 2 * U * np.abs(rg))
    assert np.all(np.abs(gh[:-1] - rh) <= 2 * U * np.abs(rh))
    absum = np.array([(w * tl).sum(), (w * tk).sum(), 0.0, 0.0])
    assert np.all(np.abs(out.cpu().numpy() - ro) <= absum + 2 * U * (np.abs(ro) + w.sum()))


@pytest.mark.parametrize("T", [8192, 8193, 1048577, 1100001])
def test_policy_logits_of_more_rows_than_terms_at_once(T):
    """Cross-entropy of rows of three words; 1024 workgroups add 1024 rows'
    terms each at a time."""
    V = 3
    say(f"[policy rows] T={T}")
    x, xv = _rows(T, V, V, "f32", 12)
    g = np.random.default_rng(13)
    y, c = g.integers(0, V, T), (g.random(T) / T).astype(np.float32)
    e = np.exp(xv - xv.max(1, keepdims=True))
    z = np.log(e.sum(1))
    rl, p = xv[np.arange(T), y] - xv.max(1) - z, e / e.sum(1, keepdims=True)
    ref = c[:, None] * (p - np.eye(V)[y])
    out, lp, dx, _ = _policy_logits(x, V, "f32", y, 1.0, q.policy_struct(q.OBJ_NLL), c)
    tl = o._tol_rows(V, rl, z)[0]
    assert np.all(np.abs(lp - rl) <= tl)
    tol = c[:, None] * (p * 120 * U + 4 * U)
    assert np.all(np.abs(out_to_f64(dx, "f32").reshape(T, V) - ref) <= tol)
    h = (z - (p * (xv - xv.max(1, keepdims=True))).sum(1))
    # a term errs by its logp (entropy) and the roundings of product and sum
    th = o._tol_rows(V, rl, z)[2]
    assert abs(out[0] + (c * rl).sum()) <= (c * (tl + 4 * U * np.abs(rl))).sum()
    assert abs(out[3] - (c * h).sum()) <= (c * (th + 4 * U * h)).sum()
    assert out[1] == 0 and out[2] == 0
