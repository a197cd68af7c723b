"""The linear's elementwise end and its gradient.

The end is checked from its own z: Z is the plain forward's result (the same
accumulators, so the same bits where there is no bias, and in fp32 one rounded
addition where there is), and y against float64 from z.  Of an fp32 y:
sigma(v) is within 0.28 * 4 2^-24 (its argument's error) + 3 2^-24 (exp2,
addition, reciprocal) < 5 2^-24, Phi within half of 1.5e-7 (its formula's) and 3
2^-24 < 5 2^-24, then three products and sums: 8 2^-24 of |act| and 12 2^-24 of the parts (the derivatives' of
(1 + |z|)).  A bf16 z is known to half a step, 2^-8 |z| (act' <= 1.13), and a
bf16 result adds 2^-8 of itself."""

import math

import numpy as np
import pytest
from scipy import special

from quantized_rank_fine_amd import qlora as q

from gpu_harness import Layer, out_to_f64, rel_err, say, torch_dev

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
ACTS = {"none": q.EP_NONE, "relu": q.EP_RELU, "gelu": q.EP_GELU, "gelu_tanh": q.EP_GELU_TANH,
        "silu": q.EP_SILU}


def act(z, kind):
    """act(z) and act'(z) in float64."""
    if kind == "none":
        return z, np.ones_like(z)
    if kind == "relu":
        return np.maximum(z, 0), (z > 0).astype(float)
    if kind == "silu":
        s = special.expit(z)
        return z * s, s + z * s * special.expit(-z)
    if kind == "gelu":
        c = special.ndtr(z)
        return z * c, c + z * np.exp(-z * z / 2) / math.sqrt(2 * math.pi)
    k = math.sqrt(8 / math.pi)
    v = np.clip(z, -1e5, 1e5)
    s = special.expit(k * (v + 0.044715 * v ** 3))
    return z * s, s + v * s * special.expit(-k * (v + 0.044715 * v ** 3)) * k * (1 + 0.134145 * v * v)


def test_oracle_derivatives_against_differences():
    z = np.linspace(-6, 6, 2401) + 1e-4
    for kind in ACTS:
        d = (act(z + 1e-6, kind)[0] - act(z - 1e-6, kind)[0]) / 2e-6
        assert np.abs(d - act(z, kind)[1]).max() < 1e-8, kind


class Case:
    def __init__(self, M, n_in, n_out, r, dt="bf16", block=64, adt="bf16"):
        torch, dev = torch_dev()
        self.L = Layer(77, M, n_in, n_out, r, dt, adt, block=block)
        self.dt, self.shape = dt, (M, n_out)
        g = torch.Generator(dev)
        g.manual_seed(M + n_out)
        rand = lambda *s: (torch.randn(*s, generator=g, device=dev)).to(self.L.tdt)  # noqa: E731
        self.bias, self.mul, self.res = rand(n_out), rand(M, n_out), rand(M, n_out)

    def run(self, kind, bias, mul, res, z=True, lora=(1.0, 0.0, None), alias=None):
        torch, dev = torch_dev()
        L = self.L
        M, n_out = self.shape
        pad = 64
        Y = torch.full((M * n_out + pad,), 9.0, dtype=L.tdt, device=dev)
        Z = torch.full((M * n_out + pad,), 9.0, dtype=L.tdt, device=dev) if z else None
        XA = torch.empty(M, max(L.r, 1), device=dev)
        n = q.qlora_fwd_workspace_bytes(M, L.n_in, n_out, L.r, L.qact)
        ws = torch.full((n + 256,), 255, dtype=torch.uint8, device=dev)
        mt, rt = self.mul, self.res
        if alias == "mul":
            Y[:M * n_out] = mt.reshape(-1)
            mt = Y
        if alias == "res":
            Y[:M * n_out] = rt.reshape(-1)
            rt = Y
        ep = q.epilogue_struct(ACTS[kind], self.bias if bias else None, mt if mul else None,
                               rt if res else None, Z)
        q.qlora_linear_fwd_ep(L.wq, L.tX, M, L.qact, L.tA, L.tB, L.r, L.qadt, *lora, ep, Y,
                              XA if L.r else None, ws, n)
        torch.cuda.synchronize()
        assert (ws[n:] == 255).all() and (Y[M * n_out:] == 9).all()
        if z:
            assert (Z[M * n_out:] == 9).all()
            Z = Z[:M * n_out].view(M, n_out)
        return Y[:M * n_out].view(M, n_out), Z, XA

    def check(self, kind, bias, mul, res, alias=None):
        torch, _ = torch_dev()
        plain, xa = self.L.fwd(lora=(1.0, 0.0, None))
        Y, Z, XA = self.run(kind, bias, mul, res, alias=alias)
        if self.L.r:
            assert torch.equal(XA[:, :self.L.r], xa)
        f64 = lambda t: out_to_f64(t, self.dt)  # noqa: E731
        if not bias:
            assert torch.equal(Z, plain)
        elif self.dt == "f32":
            assert torch.equal(Z, plain + self.bias)
        else:
            want = f64(plain) + f64(self.bias)
            assert np.all(np.abs(f64(Z) - want) <= 2.0 ** -8 * (np.abs(f64(plain)) + np.abs(want)) + U)
        z = f64(Z)
        m = f64(self.mul) if mul else 1.0
        f, _ = act(z, kind)
        want = f * m + (f64(self.res) if res else 0.0)
        tol = 12 * U * (np.abs(f * m) + np.abs(want)) + 8 * U * np.abs(z * m)
        if self.dt == "bf16":
            tol = tol + 2.0 ** -8 * (np.abs(want) + 1.13 * np.abs(z * m) * (1 + 2.0 ** -8))
            tol = tol + 2.0 ** -16 * np.abs(z * m)
        bad = np.abs(f64(Y) - want) > tol
        assert not bad.any(), (kind, np.abs(f64(Y) - want)[bad].max())
        Y2, none, _ = self.run(kind, bias, mul, res, z=False, alias=alias)
        assert none is None and torch.equal(Y, Y2)


SHAPES = [(1, 256, 256, 8), (5, 576, 448, 16), (16, 320, 192, 0), (16, 256, 320, 64),
          (17, 256, 192, 16), (3, 256, 192, 100), (256, 192, 128, 8), (300, 320, 448, 24),
          (1030, 256, 320, 16), (777, 128, 64, 0)]


@pytest.mark.parametrize("M,n_in,n_out,r", SHAPES)
@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_every_activation(M, n_in, n_out, r, dt):
    c = Case(M, n_in, n_out, r, dt)
    for kind in ACTS:
        say(f"[ep] {M}x{n_in}x{n_out} r={r} {dt} {kind}")
        c.check(kind, True, True, True)
        c.check(kind, False, False, False)


@pytest.mark.parametrize("M,n_in,n_out,r", [(5, 256, 448, 16), (300, 256, 448, 16)])
@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("bias,mul,res", [(1, 0, 0), (0, 1, 0), (0, 0, 1), (1, 1, 0), (0, 1, 1)])
def test_parts(M, n_in, n_out, r, dt, bias, mul, res):
    say(f"[ep parts] {M} {dt} {bias}{mul}{res}")
    c = Case(M, n_in, n_out, r, dt)
    c.check("silu", bias, mul, res)
    c.check("none", bias, mul, res)
    if mul:
        c.check("gelu", bias, mul, res, alias="mul")
    if res:
        c.check("gelu_tanh", bias, mul, res, alias="res")


@pytest.mark.parametrize("M", [4, 200])
def test_sixteen_entry_weight_and_fp32_adapters(M):
    c = Case(M, 256, 320, 12, "bf16", block=16, adt="f32")
    c.check("silu", True, True, True)
    c = Case(M, 256, 320, 12, "f32", block=16, adt="f32")
    c.check("gelu", True, True, True)


@pytest.mark.parametrize("M", [7, 130])
@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_against_the_oracle_with_adapter_options(M, dt):
    """Scale and dropout on U: the parity bound of the forward, 1e-2."""
    torch, dev = torch_dev()
    c = Case(M, 320, 192, 16, dt)
    keep = torch.randint(0, 2, (M, 16), device=dev, dtype=torch.uint8)
    Y, Z, _ = c.run("silu", True, True, True, lora=(2.0, 0.5, keep))
    L = c.L
    f64 = lambda t: out_to_f64(t, dt)  # noqa: E731
    xa = L.X.values.astype(float) @ L.A.values.astype(float)
    z = (L.X.values.astype(float) @ L.w_hat() +
         4.0 * keep.cpu().numpy() * xa @ L.B.values.astype(float) + f64(c.bias))
    y = act(z, "silu")[0] * f64(c.mul) + f64(c.res)
    assert rel_err(f64(Z), z) < 1e-2 and rel_err(f64(Y), y) < 1e-2
    plain, _ = L.fwd(lora=(2.0, 0.5, keep))
    assert torch.equal(c.run("none", False, False, False, lora=(2.0, 0.5, keep))[1], plain)


@pytest.mark.parametrize("M", [3, 140])
@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_a_nan_stays_one(M, dt):
    """A NaN before the end, or in one of its operands, is a NaN in Y there and
    nowhere else, whatever the activation."""
    torch, _ = torch_dev()
    c = Case(M, 256, 192, 8, dt)
    want = torch.zeros(M, 192, dtype=torch.bool)
    c.bias[5] = c.mul[1, 70] = c.res[M - 1, 191] = float("nan")
    want[:, 5] = want[1, 70] = want[M - 1, 191] = True
    for kind in ACTS:
        Y, Z, _ = c.run(kind, True, True, True)
        assert torch.equal(Y.isnan().cpu(), want), kind
        assert Z[:, 5].isnan().all() and Z.isnan().sum() == M
        # and the gradient's: what the loss has of it must not look sound
        dZ, dm, db = _bwd(Z, c.mul, c.res, kind, dt)
        assert dm[:, 5].isnan().all(), kind
        assert dZ[1, 70].isnan() and dZ[M - 1, 191].isnan() and db[191].isnan()


def test_no_tokens():
    c = Case(4, 256, 192, 8)
    L = c.L
    q.qlora_linear_fwd_ep(L.wq, None, 0, q.BF16, None, None, 8, q.BF16, 1.0, 0.0, None,
                          q.epilogue_struct(q.EP_SILU), None, None, None, 0)


# ------------------------------------------------------------------ gradient

def _bwd(Z, mul, dY, kind, dt, want_dz=True, want_dmul=True, want_db=True, alias=False):
    torch, dev = torch_dev()
    M, n = dY.shape
    t = torch.bfloat16 if dt == "bf16" else torch.float32
    out = lambda: torch.full((M * n + 64,), 9.0, dtype=t, device=dev)  # noqa: E731
    dZ, dm = out() if want_dz else None, out() if want_dmul and mul is not None else None
    if alias:
        dZ[:M * n] = dY.reshape(-1)
        dY = dZ
        if dm is not None:
            dm[:M * n] = mul.reshape(-1)
            mul = dm
    db = torch.full((n + 64,), 9.0, device=dev) if want_db else None
    need = q.qlora_ep_bwd_workspace_bytes(M, n, q.BF16 if dt == "bf16" else q.F32)
    ws = torch.full((need + 256,), 255, dtype=torch.uint8, device=dev)
    q.qlora_ep_bwd(Z, mul, dY, M, n, q.BF16 if dt == "bf16" else q.F32, ACTS[kind], dZ, dm, db,
                   ws if need else None, need)
    torch.cuda.synchronize()
    assert (ws[need:] == 255).all()
    for o, size in ((dZ, M * n), (dm, M * n), (db, n)):
        assert o is None or (o[size:] == 9).all()
    cut = lambda o: None if o is None else o[:M * n].view(M, n)  # noqa: E731
    return cut(dZ), cut(dm), None if db is None else db[:n]


def _inputs(M, n, dt, seed=0):
    torch, dev = torch_dev()
    t = torch.bfloat16 if dt == "bf16" else torch.float32
    g = torch.Generator(dev)
    g.manual_seed(seed + M)
    Z = torch.randn(M, n, generator=g, device=dev) * 3
    # tails, zeros and sizes whose squares and cubes leave fp32
    far = torch.tensor([0.0, -0.0, 12.0, -12.0, 40.0, -40.0, 100.0, -100.0, 1e10, -1e10, 1e25,
                        -1e25, 3e38, -3e38], device=dev)
    Z.view(-1)[:min(14, M * n)] = far[:M * n]
    rand = lambda: torch.randn(M, n, generator=g, device=dev).to(t)  # noqa: E731
    return Z.to(t), rand(), rand()


@pytest.mark.parametrize("M,n", [(1, 64), (3, 128), (64, 64), (65, 192), (129, 448), (300, 1088),
                                 (2000, 320), (17000, 64), (40, 11008)])
@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("with_mul", [True, False])
def test_gradient(M, n, dt, with_mul):
    torch, _ = torch_dev()
    Z, mul, dY = _inputs(M, n, dt)
    f64 = lambda t: out_to_f64(t, dt)  # noqa: E731
    z, m, d = f64(Z), f64(mul) if with_mul else 1.0, f64(dY)
    for kind in ACTS:
        say(f"[ep bwd] {M}x{n} {dt} {kind} mul={with_mul}")
        dZ, dm, db = _bwd(Z, mul if with_mul else None, dY, kind, dt)
        f, df = act(z, kind)
        half = 2.0 ** -8 if dt == "bf16" else U
        part = 16 * U * np.abs(d * m) * (1 + np.minimum(np.abs(z), 30))
        want = d * m * df
        assert np.all(np.abs(f64(dZ) - want) <= half * np.abs(want) + part), kind
        if with_mul:
            w = d * f
            with np.errstate(over="ignore"):
                top = torch.finfo(torch.float32).max
                fine = np.abs(w) < top / 2
                assert np.all((np.abs(f64(dm) - w) <= half * np.abs(w) + 16 * U * np.abs(d * z))[fine])
        # a lane adds the rows of its share of a slab, fp64 from there on
        adds = max(64, (M + 255) // 256 + 64)
        total = np.abs(want).sum(0)
        tol = (adds * U) * total + part.sum(0) + U * np.abs(want.sum(0))
        assert np.all(np.abs(db.cpu().numpy() - want.sum(0)) <= tol), kind
        again = _bwd(Z, mul if with_mul else None, dY, kind, dt, alias=True)
        for a, b in zip((dZ, dm, db), again):
            assert a is b is None or torch.equal(a, b)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_outputs_left_out(dt):
    torch, _ = torch_dev()
    Z, mul, dY = _inputs(150, 320, dt, 3)
    full = _bwd(Z, mul, dY, "silu", dt)
    for keep in range(8):
        part = _bwd(Z, mul, dY, "silu", dt, *(bool(keep & b) for b in (1, 2, 4)))
        for i, (a, b) in enumerate(zip(full, part)):
            assert (b is None) == (not keep >> i & 1) and (b is None or torch.equal(a, b))
    # without an activation Z is not read unless dmul is wanted
    dZ, _, db = _bwd(None, None, dY, "none", dt)
    assert torch.equal(dZ, dY)
    a = _bwd(None, mul, dY, "none", dt, want_dmul=False)
    b = _bwd(Z, mul, dY, "none", dt)
    assert torch.equal(a[0], b[0]) and torch.equal(a[2], b[2])


@pytest.mark.parametrize("M,n", [(1 << 24, 64), (2500, 1 << 19)])
def test_gradient_far_into_memory(M, n):
    """Arrays past 2^32 bytes; the ReLU's gradient has one rounding at most."""
    torch, dev = torch_dev()
    say(f"[ep bwd] {M}x{n}")
    g = torch.Generator(dev)
    g.manual_seed(1)
    Z, mul, dY = (torch.randn(M, n, generator=g, device=dev) for _ in range(3))
    dZ, dm, db = _bwd(Z, mul, dY, "relu", "f32")
    assert torch.equal(dm, dY * Z.clamp(min=0))
    dY *= Z > 0
    dY *= mul                                          # now dZ
    assert torch.equal(dZ, dY)
    # fp32 over a lane's rows of a slab (1/8 or more of 65536 or 32), fp64 from there on
    for c in range(0, n, 1 << 19):
        want = dZ[:, c:c + (1 << 19)].double()
        tol = 8192 * U * want.abs().sum(0) + U * want.sum(0).abs()
        assert ((db[c:c + (1 << 19)].double() - want.sum(0)).abs() <= tol).all()


def _tail_bounds(z, kind, half):
    """Bounds of act(z) and act'(z) relative to the size of their terms, U = 2^-24.

    GELU: e^(-z^2/2) or erfc take an argument of up to 1.3 U (constant, product), which
    moves them by (1 + z^2) 1.3 U, or twice that where z^2 has two roundings; exp2
    or erfcf, a reciprocal, a polynomial and three products give 16 U at most.  SiLU:
    1.3 U of v = z moves e^-v by 1.3 |v| U; exp2, addition, reciprocal, product 8 U.
    GELU_TANH: v = 2 sqrt(2 / pi) (z + 0.044715 z^3) is within 5 U, its product with
    log2 e 1.3 U more.  The derivatives have two products and a sum more each.  A
    result's rounding is `half` of it."""
    if kind == "gelu":
        rel, phi = (2.6 * z * z + 18) * U, np.exp(-z * z / 2) / math.sqrt(2 * math.pi)
        terms = special.ndtr(z) + np.abs(z) * phi
    else:
        v = z if kind == "silu" else math.sqrt(8 / math.pi) * (z + 0.044715 * z ** 3)
        rel = (1.5 * np.abs(v) + 12) * U if kind == "silu" else (6.5 * np.abs(v) + 16) * U
        slope = 1.0 if kind == "silu" else math.sqrt(8 / math.pi) * (1 + 0.134145 * z * z)
        terms = special.expit(v) * (1 + np.abs(z) * slope * special.expit(-v))
    f, df = act(z, kind)
    return (rel + half) * np.abs(f), rel * terms + half * np.abs(df)


@pytest.mark.parametrize("kind,low", [("gelu", -12.5), ("gelu_tanh", -9.5), ("silu", -80.0)])
@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_digits_of_the_tails(kind, low, dt):
    """act and act' keep the digits of their type where they are small: of the forward
    z = bias (no input, no adapter), of the gradient dY = mul = 1."""
    torch, dev = torch_dev()
    n, half = 1024, 2.0 ** -8 if dt == "bf16" else U
    t = torch.bfloat16 if dt == "bf16" else torch.float32
    z = torch.linspace(low, 12.0, n, device=dev).to(t)
    z[:8] = torch.tensor([-3.0, -4.0, -5.0, -6.2, -8.0, -0.75, 1e-3, -1e-3], device=dev)
    zv = out_to_f64(z, dt)
    tol, dtol = _tail_bounds(zv, kind, half)
    f, df = act(zv, kind)
    one = torch.ones(1, n, dtype=t, device=dev)
    dZ, dm, _ = _bwd(z[None], one, one, kind, dt)
    for name, got, want, bound in (("act", dm, f, tol), ("act'", dZ, df, dtol)):
        err = np.abs(out_to_f64(got, dt).reshape(-1) - want)
        bad = np.nonzero(err > bound)[0]
        assert bad.size == 0, (name, bad.size, zv[bad[:5]], (err / np.abs(want))[bad[:5]])
    for M in (3, 140):
        say(f"[ep tails] {kind} {dt} M={M}")
        c = Case(M, 256, n, 0, dt)
        c.L.tX.zero_()
        c.bias = z
        Y, Z, _ = c.run(kind, True, False, False)
        assert torch.equal(Z, z.expand(M, n))
        assert (np.abs(out_to_f64(Y, dt).reshape(M, n) - f) <= tol).all(), (kind, M)


@pytest.mark.parametrize("M,n", [(1 << 20, 64), (300001, 64), (100003, 320), (1 << 19, 256)])
@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_bias_gradient_of_many_rows(M, n, dt):
    """The sums of equal values (a mean's gradient), whose roundings all go one way.
    A lane adds at most 16 rows in fp32: (1 + ... + 16) / 16 half units < 9 2^-24 of the
    sum, fp64 from there, one rounding."""
    torch, dev = torch_dev()
    t = torch.bfloat16 if dt == "bf16" else torch.float32
    row = (torch.arange(1, n + 1, device=dev) / (3.0 * M)).to(t)
    scale = torch.full((n,), 1 / 7, device=dev).to(t)
    dY, mul = row.expand(M, n).contiguous(), scale.expand(M, n).contiguous()
    _, _, db = _bwd(None, mul, dY, "none", dt, want_dmul=False)
    want = M * (row * scale if dt == "f32" else row.float() * scale.float()).double()
    err = ((db.double() - want).abs() / want).max()
    assert float(err) <= 10 * U, float(err) / U


def test_no_tokens_gradient():
    torch, dev = torch_dev()
    db = torch.full((128,), 3.0, device=dev)
    q.qlora_ep_bwd(None, None, None, 0, 128, q.F32, q.EP_SILU, None, None, db, None, 0)
    assert not db.any()


@pytest.mark.parametrize("M", [6, 200])
def test_step_through_a_block_captured(M):
    """Gate and up projections, gated product, down projection into the
    residual stream, and back: every gradient against float64, and a graph's
    replays give the eager bits."""
    torch, dev = torch_dev()
    n, h, r = 256, 448, 16
    up, gate, down = (Layer(78, M, *s, r, linear=i) for i, s in enumerate(((n, h), (n, h), (h, n))))
    b16 = lambda *s: torch.empty(*s, dtype=torch.bfloat16, device=dev)  # noqa: E731
    u, zg, y, out = b16(M, h), b16(M, h), b16(M, h), b16(M, n)
    dy, dz, du, dx, dx2 = b16(M, h), b16(M, h), b16(M, h), b16(M, n), b16(M, n)
    ad = {x: (torch.empty(x.n_in, r, device=dev), torch.empty(r, x.n_out, device=dev))
          for x in (up, gate, down)}
    X, dO = up.tX, down.tdY
    nf = max(q.qlora_fwd_workspace_bytes(M, *s, r) for s in ((n, h), (h, n)))
    nb = max(max(q.qlora_bwd_workspace_bytes(M, *s, r) for s in ((n, h), (h, n))),
             q.qlora_ep_bwd_workspace_bytes(M, h))
    ws = torch.empty(max(nf, nb), dtype=torch.uint8, device=dev)

    def fwd(L, x, ep, yy):
        q.qlora_linear_fwd_ep(L.wq, x, M, q.BF16, L.tA, L.tB, r, q.BF16, 2.0, 0.0, None, ep, yy,
                              None, ws, nf)

    def bwd(L, x, dyy, dxx):
        q.qlora_linear_bwd_lora(L.wq, x, dyy, M, q.BF16, L.tA, L.tB, r, q.BF16, 2.0, 0.0, None,
                                None, dxx, *ad[L], ws, nb)

    def step():
        fwd(up, X, q.epilogue_struct(), u)
        fwd(gate, X, q.epilogue_struct(q.EP_SILU, mul=u, Z=zg), y)
        fwd(down, y, q.epilogue_struct(residual=X), out)
        bwd(down, y, dO, dy)
        q.qlora_ep_bwd(zg, u, dy, M, h, q.BF16, q.EP_SILU, dz, du, None, ws, nb)
        bwd(gate, X, dz, dx)
        bwd(up, X, du, dx2)

    outs = [out, dx, dx2] + [t for v in ad.values() for t in v]
    step()
    torch.cuda.synchronize()
    want = [t.clone() for t in outs]
    f64 = lambda t: out_to_f64(t, "bf16")  # noqa: E731
    W = {x: x.w_hat() + 2.0 * x.A.values.astype(float) @ x.B.values.astype(float)
         for x in (up, gate, down)}
    x, do = f64(X), f64(dO)
    ru, rz = x @ W[up], x @ W[gate]
    f, df = act(rz, "silu")
    assert rel_err(f64(out), x + (f * ru) @ W[down]) < 1e-2
    rdy = do @ W[down].T
    rdz, rdu = rdy * ru * df, rdy * f
    assert rel_err(f64(dx), rdz @ W[gate].T) < 2e-2      # two forward and two backward roundings
    assert rel_err(f64(dx2), rdu @ W[up].T) < 2e-2
    for L, xx, g in ((gate, x, rdz), (up, x, rdu), (down, f * ru, do)):
        A, B = L.A.values.astype(float), L.B.values.astype(float)
        assert rel_err(ad[L][0].cpu().numpy(), 2 * xx.T @ (g @ B.T)) < 2e-2
        assert rel_err(ad[L][1].cpu().numpy(), 2 * (xx @ A).T @ g) < 2e-2
    cg = torch.cuda.CUDAGraph()
    with torch.cuda.graph(cg):
        step()
    for _ in range(3):
        for t in outs + [u, zg, y, dy, dz, du]:
            t.fill_(float("nan"))
        ws.fill_(255)
        torch.cuda.synchronize()
        cg.replay()
        torch.cuda.synchronize()
        for t, w in zip(outs, want):
            assert torch.equal(t, w)
