"""The orthogonalised update against float64.

m, theta and theta_bf16 are fp32 operations rounded one by one, so they are
compared bit by bit with NumPy's fp32 (theta from the update the call itself
returned).  The update X is compared with the oracle's, from the singular
values of the same fp32 direction u: it is rounded to fp32 once (half a step,
2^-24 |X|), and before that held in fp64, where an error e of an eigenvalue of
the Gram matrix (at most 4 k 2^-53 after sums of k products) moves X by
s q'(s^2) e, s q' below 1.2e5 for five steps of the usual polynomial (its peak,
at s = 0.002, scanned below): 4 * 256 * 1.1e-16 * 1.2e5 = 1.4e-8."""

import numpy as np
import pytest

import oracle
from quantized_rank_fine_amd import qlora as q

from gpu_harness import bf16_to_f64, say, torch_dev

pytestmark = pytest.mark.gpu

F = np.float32
TOL = 1.4e-8


def _gradient(g, rows, cols, kind="plain"):
    x = g.standard_normal((rows, cols))
    if kind == "strong":                     # four directions over a weak floor
        x = 20 * g.standard_normal((rows, 4)) @ g.standard_normal((4, cols)) + x
    if kind == "rank1":
        x = np.outer(g.standard_normal(rows), g.standard_normal(cols))
    if kind == "zero":
        x = 0 * x
    return (x * 1e-3).astype(F)


class Mat:
    """One matrix's host and device state; `off`: elements its buffers start
    past a 16-byte boundary."""

    def __init__(self, rows, cols, seed=0, kind="plain", m=True, theta=True, copy=True, off=0,
                 scale=1.0, size=1.0):
        torch, dev = torch_dev()
        g = np.random.default_rng([seed, rows, cols])
        self.rows, self.cols, self.scale = rows, cols, scale
        self.g = _gradient(g, rows, cols, kind) * F(size)
        self.m = _gradient(g, rows, cols, kind) * F(4 * size) if m else None
        self.th = g.standard_normal((rows, cols)).astype(F) if theta else None

        def put(a, dtype=torch.float32):
            n = rows * cols
            t = torch.full((n + off + 64,), 7.0, dtype=dtype, device=dev)
            if a is not None:
                t[off:off + n] = torch.from_numpy(a.reshape(-1)).to(dev)
            return t

        self.off = off
        self.tg = put(self.g)
        self.tm = put(self.m) if m else None
        self.tt = put(self.th) if theta else None
        self.tc = put(None, torch.bfloat16) if theta and copy else None
        self.tu = put(None)

    def _at(self, t):
        return None if t is None else t.data_ptr() + self.off * t.element_size()

    def desc(self, update=True):
        return q.muon_mat(self.rows, self.cols, self._at(self.tg), self._at(self.tm),
                          self._at(self.tt), self._at(self.tc),
                          self._at(self.tu) if update else None, self.scale)

    def read(self, t):
        n = self.rows * self.cols
        assert (t[:self.off] == 7).all() and (t[self.off + n:] == 7).all()
        t = t[self.off:self.off + n]
        v = t.cpu().numpy() if t.element_size() == 4 else bf16_to_f64(t.contiguous())
        return v.reshape(self.rows, self.cols)

    def check(self, lr, momentum, nesterov, wd, eps, steps, coef, tol=TOL):
        mu = F(momentum)
        u = self.g
        if self.m is not None:
            self.m = mu * self.m + self.g
            assert np.array_equal(self.read(self.tm), self.m)
            u = self.g + mu * self.m if nesterov else self.m
        want = oracle.orthogonalize(u, coef, steps, eps)
        got = self.read(self.tu).astype(np.float64)
        assert np.all(np.abs(got - want) <= 2.0 ** -24 * np.abs(want) + tol), \
            np.abs(got - want).max()
        if self.th is not None:
            x = got.astype(F)
            self.th = self.th - F(lr) * (F(self.scale) * x + F(wd) * self.th)
            assert np.array_equal(self.read(self.tt), self.th)
            if self.tc is not None:
                torch, _ = torch_dev()
                bf = torch.from_numpy(self.th).to(torch.bfloat16)
                assert np.array_equal(self.read(self.tc), bf16_to_f64(bf))
        assert np.array_equal(self.read(self.tg), self.g)


def run(mats, lr=0.02, momentum=0.95, nesterov=True, wd=0.01, eps=1e-7, steps=5,
        coef=q.MUON_COEF, check=True, tol=TOL, **kw):
    torch, dev = torch_dev()
    arr = q.muon_mats([m.desc() for m in mats])
    n = q.qlora_muon_workspace_bytes(arr)
    ws = torch.full((n + 256,), 255, dtype=torch.uint8, device=dev)
    q.qlora_muon_step(arr, lr, ws, n, momentum, nesterov, wd, eps, steps, coef, **kw)
    torch.cuda.synchronize()
    assert (ws[n:] == 255).all()
    if check:
        for m in mats:
            m.check(lr, momentum, nesterov, wd, eps, steps, coef, tol)


def test_slope_of_the_tolerance():
    """s |q'(s^2)| of five steps stays below 1.2e5 (q = f(s) / s)."""
    lam = np.logspace(-12, 0, 200001)
    p, dp, x, dx = np.ones_like(lam), np.zeros_like(lam), lam.copy(), np.ones_like(lam)
    a, b, c = q.MUON_COEF
    for _ in range(5):
        s, ds = a + b * x + c * x * x, (b + 2 * c * x) * dx
        p, dp = p * s, dp * s + p * ds
        x, dx = x * s * s, dx * s * s + 2 * x * s * ds
    assert (np.sqrt(lam) * np.abs(dp)).max() < 1.2e5


SHAPES = [(1, 1), (1, 5), (5, 1), (1, 4096), (4096, 1), (7, 3), (3, 8), (16, 16), (17, 16),
          (100, 16), (16, 1000), (257, 17), (33, 300), (48, 640), (1001, 48), (64, 64), (63, 64),
          (65, 64), (64, 65), (65, 65), (500, 64), (64, 4100), (130, 128), (96, 200), (129, 200),
          (200, 201), (2050, 192), (193, 700), (256, 256), (1111, 255), (256, 1500)]


@pytest.mark.parametrize("rows,cols", SHAPES)
@pytest.mark.parametrize("kind,off", [("plain", 0), ("strong", 1)])
def test_shapes(rows, cols, kind, off):
    say(f"[muon] {rows}x{cols} {kind} off={off}")
    run([Mat(rows, cols, kind=kind, off=off)])


@pytest.mark.parametrize("rows,cols", [(300, 16), (24, 200), (300, 130)])
@pytest.mark.parametrize("kind", ["rank1", "zero"])
def test_deficient_gradients(rows, cols, kind):
    say(f"[muon] {rows}x{cols} {kind}")
    m = Mat(rows, cols, kind=kind)
    run([m])
    if kind == "zero":
        assert not m.read(m.tu).any()


def test_zero_gradient_without_eps():
    m = Mat(40, 8, kind="zero")
    run([m], eps=0.0)
    assert not m.read(m.tu).any()


@pytest.mark.parametrize("size", [1e-33, 1e30])
@pytest.mark.parametrize("rows,cols", [(200, 16), (16, 200), (300, 64), (300, 100)])
def test_far_sizes(rows, cols, size):
    """Gradients near the ends of fp32 (m x 4 stays finite)."""
    say(f"[muon] {rows}x{cols} size {size}")
    run([Mat(rows, cols, size=size)], eps=0.0)


@pytest.mark.parametrize("kw", [
    dict(nesterov=False), dict(momentum=0.0), dict(steps=1), dict(steps=2), dict(steps=3),
    dict(coef=(1.5, -0.5, 0.0), steps=12), dict(coef=(2.0, -1.5, 0.5), steps=6), dict(eps=0.1),
    dict(wd=0.0, lr=-0.5), dict(lr=0.0)])
@pytest.mark.parametrize("rows,cols", [(150, 16), (40, 300), (200, 90)])
def test_options(rows, cols, kw):
    """(the milder polynomials' slopes are below the usual one's: a^(3 steps)
    is 2.2e6 and 2.6e5 at most, with s below 1 over their a^steps)"""
    say(f"[muon] {rows}x{cols} {kw}")
    run([Mat(rows, cols)], **kw)


def _slope(steps):
    """The peak of s |q'(s^2)|, as scanned above, for more steps."""
    lam = np.logspace(-14, 0, 200001)
    p, dp, x, dx = np.ones_like(lam), np.zeros_like(lam), lam.copy(), np.ones_like(lam)
    a, b, c = q.MUON_COEF
    for _ in range(steps):
        s, ds = a + b * x + c * x * x, (b + 2 * c * x) * dx
        p, dp = p * s, dp * s + p * ds
        x, dx = x * s * s, dx * s * s + 2 * x * s * ds
    return (np.sqrt(lam) * np.abs(dp)).max()


@pytest.mark.parametrize("steps", [6, 7, 8])
@pytest.mark.parametrize("rows,cols", [(300, 16), (64, 500), (400, 200), (700, 256)])
def test_more_steps_of_the_usual_polynomial(rows, cols, steps):
    """Up to the most that is allowed; the slope is 0.15 a^(2 steps), as the header
    says, and 10% more than its scan is left for what lies between its points."""
    slope = _slope(steps)
    assert 0.14 < slope / q.MUON_COEF[0] ** (2 * steps) < 0.16
    for kind in ("plain", "strong"):
        say(f"[muon] {rows}x{cols} {kind} {steps} steps")
        run([Mat(rows, cols, kind=kind)], steps=steps,
            tol=1.1 * slope * 4 * min(rows, cols) * 2.0 ** -53)


def test_parts_left_out():
    """No momentum, no theta, no copy, no update: each alone."""
    mats = [Mat(90, 12, m=False), Mat(12, 90, theta=False), Mat(90, 100, copy=False),
            Mat(90, 100, m=False, theta=False)]
    run(mats)
    torch, dev = torch_dev()
    a, b = Mat(90, 12, seed=3), Mat(90, 12, seed=3)
    arr = q.muon_mats([a.desc(update=False)])
    n = q.qlora_muon_workspace_bytes(arr)
    ws = torch.empty(n, dtype=torch.uint8, device=dev)
    q.qlora_muon_step(arr, 0.02, ws, n, weight_decay=0.01)
    run([b])
    assert np.array_equal(a.read(a.tt), b.th) and (a.tu == 7).all()


def test_many_matrices_of_all_sizes():
    """More than one launch describes, short sides of every kind mixed."""
    g = np.random.default_rng(5)
    mats = [Mat(*((n, k) if i % 2 else (k, n)), seed=i, off=i % 3, scale=0.5 + i % 4,
                kind="strong" if i % 5 == 0 else "plain")
            for i, (n, k) in enumerate(zip(g.integers(20, 700, 75), g.integers(1, 257, 75)))]
    say(f"[muon] {len(mats)} matrices")
    run(mats)


@pytest.mark.parametrize("sizes", [
    [(82, 3), (3, 1248), (16, 16)], [(40, 500), (501, 40), (33, 70)], [(200, 90), (90, 201)],
    [(60, 400), (401, 60), (300, 130), (131, 300), (7, 7)], [(40000, 50), (48, 4000)],
    [(100, 16)] * 16, [(101, 15), (100, 16)] * 8, [(100, 16), (101, 15), (30, 100)] * 6])
def test_calls_of_matrices_of_both_kinds_of_access(sizes):
    """Short calls, whose matrices travel with the launch, and the first longer one;
    aligned and not; small and large."""
    say(f"[muon] {sizes[:5]} x {len(sizes)}")
    run([Mat(r, c, seed=i, off=i % 2) for i, (r, c) in enumerate(sizes)])


def test_the_most_matrices_of_a_call():
    """A full table, single values and small matrices."""
    g = np.random.default_rng(6)
    mats = [Mat(*map(int, g.integers(1, 20, 2)), seed=i) for i in range(q.MUON_MAX_MATS)]
    say(f"[muon] {len(mats)} matrices")
    run(mats, check=False)
    for m in mats[:40] + mats[2000:2040] + mats[-40:]:
        m.check(0.02, 0.95, True, 0.01, 1e-7, 5, q.MUON_COEF)


@pytest.mark.parametrize("value", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("rows,cols", [(1, 1), (90, 12), (12, 500), (300, 40), (60, 300), (300, 130)])
def test_a_value_that_is_not_finite(rows, cols, value):
    """It has no norm: the whole update is NaN, and no other matrix's."""
    torch, _ = torch_dev()
    m, other = Mat(rows, cols), Mat(rows, cols, seed=2)
    m.tg[rows * cols // 2] = value
    run([m, other], check=False)
    n = rows * cols
    assert m.tu[:n].isnan().all() and m.tt[:n].isnan().all()
    other.check(0.02, 0.95, True, 0.01, 1e-7, 5, q.MUON_COEF)


@pytest.mark.parametrize("rows,cols", [(256, 1 << 24), (1 << 24, 256), (64, (1 << 24) - 1),
                                       ((1 << 24) - 3, 90)])
def test_the_longest_matrices(rows, cols):
    """The longest long sides, past 2^32 values: zero but for 120 long rows (the
    ends among them), which are a small matrix's, and so is the step of them."""
    torch, dev = torch_dev()
    say(f"[muon] {rows}x{cols}")
    k, n, wide = min(rows, cols), max(rows, cols), rows < cols
    g = np.random.default_rng(7)
    at = np.unique(np.concatenate([[0, 1, n - 2, n - 1], g.integers(0, n, 116)]))
    small = Mat(*((k, len(at)) if wide else (len(at), k)), scale=1.0)
    at = torch.from_numpy(at).to(dev)
    t = [torch.zeros(rows, cols, device=dev) for _ in range(3)]
    part = lambda x: x[:, at] if wide else x[at]  # noqa: E731
    for x, v in zip(t, (small.g, small.m, small.th)):
        v = torch.from_numpy(v).to(dev)
        if wide:
            x[:, at] = v
        else:
            x[at] = v
    update = torch.full((rows, cols), 7.0, device=dev)
    arr = q.muon_mats([q.muon_mat(rows, cols, *t, None, update)])
    need = q.qlora_muon_workspace_bytes(arr)
    ws = torch.empty(need, dtype=torch.uint8, device=dev)
    q.qlora_muon_step(arr, 0.02, ws, need, weight_decay=0.01)
    torch.cuda.synchronize()
    for x, name in zip((t[0], t[1], t[2], update), ("tg", "tm", "tt", "tu")):
        a = getattr(small, name)
        a[:small.rows * small.cols] = part(x).reshape(-1)
        # nothing elsewhere (0 in, 0 out)
        if wide:
            x[:, at] = 0
        else:
            x[at] = 0
        for r in range(0, rows, max(1, rows // 16)):
            assert not x[r:r + max(1, rows // 16)].any(), name
    small.tc = None
    small.check(0.02, 0.95, True, 0.01, 1e-7, 5, q.MUON_COEF)


def test_steps_follow_each_other():
    """Five steps in place, momentum and theta carried on."""
    mats = [Mat(300, 16), Mat(16, 200), Mat(200, 72)]
    for _ in range(5):
        run(mats)


def test_no_matrices():
    q.qlora_muon_step(q.muon_mats([]), 0.1, None, 0)


def test_captured_and_on_another_stream():
    """Graph replays, with other work between, and a call on a side stream
    give the eager bits."""
    torch, dev = torch_dev()
    make = lambda: [Mat(300, 16, seed=1), Mat(24, 500, seed=2), Mat(300, 90, seed=3)]  # noqa: E731
    eager, graph, side = make(), make(), make()
    for _ in range(4):
        run(eager, check=False)
    arr = q.muon_mats([m.desc() for m in graph])
    n = q.qlora_muon_workspace_bytes(arr)
    ws = torch.empty(n, dtype=torch.uint8, device=dev)
    go = lambda: q.qlora_muon_step(arr, 0.02, ws, n, weight_decay=0.01)  # noqa: E731
    go()                                                  # step 1, eagerly
    torch.cuda.synchronize()
    cg = torch.cuda.CUDAGraph()
    with torch.cuda.graph(cg):
        go()
    del arr                                               # the array is read by the call alone
    for _ in range(3):
        ws.fill_(255)
        torch.cuda.synchronize()
        cg.replay()
        torch.cuda.synchronize()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        for _ in range(4):
            run(side, check=False)
    torch.cuda.synchronize()
    for a, b, c in zip(eager, graph, side):
        for name in ("tm", "tt", "tc", "tu"):
            want = getattr(a, name)
            assert torch.equal(getattr(b, name), want) and torch.equal(getattr(c, name), want), name
