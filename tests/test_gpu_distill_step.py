"""The example's distillation step: the linears with their epilogues, the
teacher's alternatives, the loss and its gradient, the way back and the update
together."""

import os
import sys

import numpy as np
import pytest

import oracle
from oracle import objective as ob
from quantized_rank_fine_amd import qlora as q

from gpu_harness import bf16_to_f64, rel_err, torch_dev

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                                "examples"))

pytestmark = pytest.mark.gpu


def _deq(x):
    return oracle.dequantize(x.wq.codes.cpu().numpy(), x.wq.qscale.cpu().numpy(),
                             x.wq.gscale.cpu().numpy(), x.n_in, x.n_out)


@pytest.mark.parametrize("tokens", [9, 150])
def test_gradients_and_updates_of_a_step(tokens):
    """Every adapter's gradient of the second step (B is 0 in the first) against
    the chain in float64 from the dequantized weights, and the update against
    the oracle's from the gradient that the step used."""
    import distill_step as ex
    torch, dev = torch_dev()
    hidden, inner, vocab, k = 192, 320, 640, 8
    h, teacher = ex.batch(tokens, hidden, vocab, 3, dev)
    ids, top = ex.alternatives(teacher, k)
    want, lp = ob.token_top(bf16_to_f64(teacher).reshape(tokens, vocab), k)
    assert np.array_equal(ids.cpu().numpy(), want) and np.abs(top.cpu().numpy() - lp).max() < 1e-5
    s = ex.Student(hidden, inner, vocab, 8, tokens, dev)
    weight = torch.full((tokens,), 1.0 / tokens, device=dev)
    first = ex.distill_steps(s, h, ids, top, weight, 1)
    before = [[t.cpu().numpy().copy() for t in v] for x in s.linears for v in (x.theta, x.m)]
    low = [[bf16_to_f64(c).reshape(c.shape) for c in x.copy] for x in s.linears]
    second = ex.distill_steps(s, h, ids, top, weight, 1)
    assert all(np.isfinite(first + second))
    # the forward in float64, from the weights and the adapters' bf16 copies
    W = [_deq(x) + ex.SCALE * a @ b for x, (a, b) in zip(s.linears, low)]
    x = bf16_to_f64(h).reshape(tokens, hidden)
    u, z = x @ W[0], x @ W[1]
    sig = 1 / (1 + np.exp(-z))
    y = z * sig * u
    out = x + y @ W[2]
    loss, _, dl = ob.distill(out @ W[3], ids.cpu().numpy(), top.cpu().numpy(), np.full(tokens, 1 / tokens))
    assert abs(second[0] - loss) < 1e-2 * abs(loss)
    # and the way back; roundings to bf16 of five results one behind the other,
    # each within the parity bound of a linear, 1e-2 of the largest
    dout = dl @ W[3].T
    dy = dout @ W[2].T
    dz, du = dy * u * (sig + z * sig * (1 - sig)), dy * z * sig
    for lin, (a, b), xx, g in zip(s.linears, low, (x, x, y, out), (du, dz, dout, dl)):
        assert rel_err(lin.grad[0].cpu().numpy(), ex.SCALE * xx.T @ (g @ b.T)) < 5e-2
        assert rel_err(lin.grad[1].cpu().numpy(), ex.SCALE * (xx @ a).T @ g) < 5e-2
    for i, lin in enumerate(s.linears):
        for j in range(2):
            th, m = before[2 * i][j], before[2 * i + 1][j]
            scale = max(1.0, th.shape[0] / th.shape[1]) ** 0.5
            rt, rm, _ = oracle.muon_step(th, lin.grad[j].cpu().numpy(), m, 0.02, 0.9, scale=scale)
            assert np.abs(lin.m[j].cpu().numpy() - rm).max() <= 2.0 ** -22 * np.abs(rm).max()
            got = lin.theta[j].cpu().numpy()
            # m's rounding turns weak directions: 2^-22 of m by the slope of f, 485
            assert np.abs(got - rt).max() <= 0.02 * scale * 485 * 2.0 ** -22 + 2.0 ** -23 * np.abs(rt).max()
            bf = torch.from_numpy(got).to(torch.bfloat16)
            assert torch.equal(lin.copy[j].cpu(), bf)


def test_a_captured_step_is_the_eager_one():
    import distill_step as ex
    torch, dev = torch_dev()
    hidden, inner, vocab, tokens = 128, 192, 448, 40
    h, teacher = ex.batch(tokens, hidden, vocab, 5, dev)
    ids, top = ex.alternatives(teacher, 16)
    weight = torch.full((tokens,), 1.0 / tokens, device=dev)
    a, b = (ex.Student(hidden, inner, vocab, 8, tokens, dev) for _ in range(2))
    ex.distill_steps(a, h, ids, top, weight, 4)
    ex.distill_steps(b, h, ids, top, weight, 1)
    loss, kl = torch.empty(1, device=dev), torch.empty(tokens, device=dev)
    g = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        logits = b.forward(h)
        q.qlora_distill_logits(logits, vocab, tokens, vocab, q.BF16, 1.0, weight, 16, ids, top,
                               True, loss, kl, logits, vocab, None, 0)
        b.backward(h, logits)
        b.update(0.02)
    for _ in range(3):
        b.ws.fill_(255)
        b.muon_ws.fill_(255)
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
    for x, y in zip(a.linears, b.linears):
        for s, t in zip(x.theta + x.m + x.copy, y.theta + y.m + y.copy):
            assert torch.equal(s, t)


def test_the_example_runs(capsys, monkeypatch):
    import distill_step as ex
    monkeypatch.setattr(sys, "argv", ["distill_step.py", "--tokens", "64", "--steps", "2",
                                      "--hidden", "256", "--inner", "320", "--vocab", "1024",
                                      "--alternatives", "8"])
    ex.main()
    assert "divergence" in capsys.readouterr().out
