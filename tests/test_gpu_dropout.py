"""GPU parity of the counter-based dropout: the mask bit by bit against the
oracle's generator, the kept values to a rounding."""

import numpy as np
import pytest

from oracle import objective as ob
from quantized_rank_fine_amd import qlora as q

from gpu_harness import out_to_f64, say, torch_dev

pytestmark = pytest.mark.gpu

U = 2.0 ** -24


def _run(x, ldx, res, ldr, rows, cols, dt, p, seed, ctr, y, ldy):
    q.qlora_dropout(x, ldx, res, ldr, rows, cols, q.BF16 if dt == "bf16" else q.F32, p, seed, ctr,
                    y, ldy)


@pytest.mark.parametrize("rows,cols,pad,at", [
    (1, 1, 0, 0), (3, 7, 0, 1), (2, 8, 0, 0), (5, 9, 2, 3), (17, 64, 0, 0), (4, 1000, 24, 0),
    (33, 257, 0, 0), (2, 4096, 1, 0), (300, 40, 0, 0), (9, 64, 3, 2), (40, 65, 0, 7), (5, 505, 0, 1),
    (8, 511, 1, 0), (17, 1002, 0, 5),
])
@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("p,residual", [(0.1, True), (0.5, False), (0.0, True)])
def test_dropout(rows, cols, pad, at, dt, p, residual):
    torch, dev = torch_dev()
    say(f"[dropout] {rows}x{cols} pad={pad} at={at} {dt} p={p} residual={residual}")
    g = np.random.default_rng(rows * cols)
    tdt = torch.bfloat16 if dt == "bf16" else torch.float32
    ld = cols + pad
    seed, ctr = 0xFEDCBA9876543210 + rows, (1 << 40) + cols

    def rows_of():
        v = g.standard_normal(at + rows * ld).astype(np.float32)
        buf = torch.from_numpy(v).to(tdt).to(dev)
        view = buf[at:].view(rows, ld)[:, :cols]
        return view, out_to_f64(view.contiguous(), dt).reshape(rows, cols)

    x, xv = rows_of()
    r, rv = rows_of() if residual else (None, 0.0)
    keep, p16 = ob.dropout_keep(rows, cols, float(np.float32(p)), seed, ctr)
    # a dropped element may hold anything
    nanx = x.clone()
    nanx[torch.from_numpy(~keep).to(dev)] = float("nan")
    ldy = cols + 3
    buf = torch.full((rows * ldy + 2,), 5.0, dtype=tdt, device=dev)
    _run(nanx.contiguous(), cols, r, ld, rows, cols, dt, p, seed, ctr, buf[1:], ldy)
    got = out_to_f64(buf, dt)
    body = got[1:1 + rows * ldy].reshape(rows, ldy)
    assert got[0] == 5.0 and got[-1] == 5.0 and np.all(body[:, cols:] == 5.0)
    ref = np.where(keep, xv * (65536 / (65536 - p16)), 0.0) + rv
    tol = 4 * U * (np.abs(xv) * 2 + np.abs(rv)) + (2.0 ** -8 * np.abs(ref) if dt == "bf16" else 0)
    assert np.all(np.abs(body[:, :cols] - ref) <= tol)
    if not residual:
        assert np.array_equal(body[:, :cols] != 0, keep & (xv != 0))
        # the gradient through the same call: the mask and factor of the forward
        ones = torch.ones(rows, cols, dtype=tdt, device=dev)
        d = torch.empty_like(ones)
        _run(ones, cols, None, 0, rows, cols, dt, p, seed, ctr, d, cols)
        f = out_to_f64(d, dt).reshape(rows, cols)
        c = 65536 / (65536 - p16)
        assert np.all(np.abs(f - keep * c) <= c * (2.0 ** -8 if dt == "bf16" else 2 * U))
    # in place over x, and over the residual
    want = body[:, :cols].copy()
    y = x.clone().contiguous()
    _run(y, cols, r, ld, rows, cols, dt, p, seed, ctr, y, cols)
    assert np.array_equal(out_to_f64(y, dt).reshape(rows, cols), want)
    if residual:
        y = r.clone().contiguous()
        _run(x, ld, y, cols, rows, cols, dt, p, seed, ctr, y, cols)
        assert np.array_equal(out_to_f64(y, dt).reshape(rows, cols), want)


def test_dropout_seed_and_counter_words():
    """Each of the four 32-bit words of seed and counter changes the mask;
    negative or oversized Python integers are taken modulo 2^64."""
    torch, dev = torch_dev()
    x = torch.ones(4, 64, device=dev)
    seen = set()
    for seed, ctr in ((1, 1), (2, 1), (1 + (1 << 32), 1), (1, 2), (1, 1 + (1 << 32))):
        y = torch.empty_like(x)
        _run(x, 64, None, 0, 4, 64, "f32", 0.5, seed, ctr, y, 64)
        keep, _ = ob.dropout_keep(4, 64, 0.5, seed, ctr)
        assert np.array_equal((y != 0).cpu().numpy(), keep)
        seen.add(keep.tobytes())
    assert len(seen) == 5


def test_dropout_nearly_everything():
    """p so near 1 that it rounds to 1 keeps one value of 65536."""
    torch, dev = torch_dev()
    x = torch.ones(64, 4096, device=dev)
    y = torch.empty_like(x)
    _run(x, 4096, None, 0, 64, 4096, "f32", 0.9999999, 3, 4, y, 4096)
    v = y.cpu().numpy()
    assert set(np.unique(v)) <= {0.0, 65536.0} and (v != 0).sum() < 40


def test_dropout_far_into_memory():
    """Row offsets past 2^32 elements, in place."""
    torch, dev = torch_dev()
    rows, cols, ld = 66000, 24, 65600
    say(f"[dropout far] {rows}x{cols} ld={ld}")
    x = torch.ones(rows * ld, dtype=torch.bfloat16, device=dev).view(rows, ld)
    _run(x, ld, None, 0, rows, cols, "bf16", 0.25, 9, 9, x, ld)
    some = [0, 1, 40000, 65471, rows - 1]
    keep, p16 = ob.dropout_keep(rows, cols, 0.25, 9, 9, only=some)
    got = np.stack([out_to_f64(x[r, :cols].contiguous(), "bf16") for r in some])
    assert np.array_equal(got != 0, keep)
    assert bool((x[rows - 1, cols:] == 1).all()) and bool((x[0, cols:] == 1).all())


def test_dropout_of_more_groups_than_a_launch_counts():
    """2^31 groups to a launch: rows on both sides of the second one's start."""
    torch, dev = torch_dev()
    rows, cols = (1 << 30) + 1000, 9                     # two groups a row
    say(f"[dropout many] {rows}x{cols}")
    x = torch.ones(rows, cols, dtype=torch.bfloat16, device=dev)
    _run(x, cols, None, 0, rows, cols, "bf16", 0.5, 11, 12, x, cols)
    some = [0, (1 << 30) - 1, 1 << 30, (1 << 30) + 1, rows - 1]
    keep, p16 = ob.dropout_keep(rows, cols, 0.5, 11, 12, only=some)
    got = np.stack([out_to_f64(x[r].contiguous(), "bf16") for r in some])
    assert np.array_equal(got, keep * 2.0)


def test_dropout_in_a_graph():
    torch, dev = torch_dev()
    x = torch.randn(40, 300, device=dev).to(torch.bfloat16)
    y = torch.empty_like(x)
    _run(x, 300, None, 0, 40, 300, "bf16", 0.3, 5, 6, y, 300)
    torch.cuda.synchronize()
    want = y.float().cpu().numpy()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        _run(x, 300, None, 0, 40, 300, "bf16", 0.3, 5, 6, y, 300)
    for _ in range(3):
        y.fill_(float("nan"))
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert np.array_equal(y.float().cpu().numpy(), want)
