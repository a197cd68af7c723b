"""An adapted 4-bit feed-forward block and head learn a teacher's alternatives.

    python examples/distill_step.py [--tokens 512] [--steps 20]

One process, one GPU, every step on it.  The teacher's logits are read once:
its top words and their log-probabilities are what is kept of it.  A step of the
student: up and gate projections, the gated product in the gate's epilogue, the
down projection back into the residual stream in its own, the head, the loss
against the stored alternatives with the logits' gradient in the logits' own
memory, the way back through both epilogues, and one orthogonalised update of
all eight adapter matrices in one call.  Hidden states and the teacher are
random: what it shows is how the calls fit together.
"""

import argparse
import os
import sys

import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)

from quantized_rank_fine_amd import qlora as q  # noqa: E402

SCALE = 2.0          # alpha / r


class Linear:
    """A frozen 4-bit weight [in, out] with adapters of rank r: fp32 masters,
    gradients, momenta, and the bf16 copies that the products read."""

    def __init__(self, W0, rank, seed):
        self.n_in, self.n_out = W0.shape
        self.rank = rank
        self.wq = q.NF4Weight(self.n_in, self.n_out, W0.device)
        q.qlora_quantize(W0, self.wq)
        g = torch.Generator(W0.device)
        g.manual_seed(seed)
        A = torch.randn(self.n_in, rank, generator=g, device=W0.device) / self.n_in ** 0.5
        B = torch.zeros(rank, self.n_out, device=W0.device)
        self.theta, self.grad, self.m, self.copy = [A, B], [], [], []
        for p in self.theta:
            self.grad.append(torch.zeros_like(p))
            self.m.append(torch.zeros_like(p))
            self.copy.append(p.to(torch.bfloat16))

    def workspace(self, tokens):
        shape = (tokens, self.n_in, self.n_out, self.rank)
        return max(q.qlora_fwd_workspace_bytes(*shape), q.qlora_bwd_workspace_bytes(*shape))

    def forward(self, x, end, y, ws):
        q.qlora_linear_fwd_ep(self.wq, x, x.shape[0], q.BF16, *self.copy, self.rank, q.BF16, SCALE,
                              0.0, None, end, y, None, ws, ws.numel())

    def backward(self, x, dy, dx, ws):
        q.qlora_linear_bwd_lora(self.wq, x, dy, x.shape[0], q.BF16, *self.copy, self.rank, q.BF16,
                                SCALE, 0.0, None, None, dx, *self.grad, ws, ws.numel())

    def matrices(self):
        """What the update takes; each step's size is that of its matrix."""
        return [q.muon_mat(*p.shape, g, m, p, c, None, max(1.0, p.shape[0] / p.shape[1]) ** 0.5)
                for p, g, m, c in zip(self.theta, self.grad, self.m, self.copy)]


class Student:
    def __init__(self, hidden, inner, vocab, rank, tokens, device):
        g = torch.Generator(device)
        g.manual_seed(11)
        w = lambda *s: torch.randn(*s, generator=g, device=device) / s[0] ** 0.5  # noqa: E731
        self.up, self.gate, self.down, self.head = self.linears = [
            Linear(w(*s), rank, i) for i, s in enumerate(((hidden, inner), (hidden, inner),
                                                          (inner, hidden), (hidden, vocab)))]
        b = lambda n: torch.empty(tokens, n, dtype=torch.bfloat16, device=device)  # noqa: E731
        self.u, self.z, self.y, self.dy = b(inner), b(inner), b(inner), b(inner)
        self.out, self.dout, self.dx = b(hidden), b(hidden), b(hidden)
        self.logits = b(vocab)
        n = max([x.workspace(tokens) for x in self.linears]
                + [q.qlora_ep_bwd_workspace_bytes(tokens, inner)])
        self.ws = torch.empty(n, dtype=torch.uint8, device=device)
        self.mats = q.muon_mats([m for x in self.linears for m in x.matrices()])
        n = q.qlora_muon_workspace_bytes(self.mats)
        self.muon_ws = torch.empty(n, dtype=torch.uint8, device=device)

    def forward(self, h):
        self.up.forward(h, q.epilogue_struct(), self.u, self.ws)
        self.gate.forward(h, q.epilogue_struct(q.EP_SILU, mul=self.u, Z=self.z), self.y, self.ws)
        self.down.forward(self.y, q.epilogue_struct(residual=h), self.out, self.ws)
        self.head.forward(self.out, q.epilogue_struct(), self.logits, self.ws)
        return self.logits

    def backward(self, h, dlogits):
        """The adapters' gradients."""
        self.head.backward(self.out, dlogits, self.dout, self.ws)
        self.down.backward(self.y, self.dout, self.dy, self.ws)
        # dz takes dy's place, du that of u
        q.qlora_ep_bwd(self.z, self.u, self.dy, h.shape[0], self.z.shape[1], q.BF16, q.EP_SILU,
                       self.dy, self.u, None, self.ws, self.ws.numel())
        self.gate.backward(h, self.dy, None, self.ws)
        self.up.backward(h, self.u, None, self.ws)

    def update(self, lr):
        q.qlora_muon_step(self.mats, lr, self.muon_ws, self.muon_ws.numel(), momentum=0.9)


def alternatives(logits, k):
    """The teacher's k most likely words of each row and their log p."""
    T, V = logits.shape
    ids = torch.empty(T, k, dtype=torch.int32, device=logits.device)
    top = torch.empty(T, k, device=logits.device)
    n = q.qlora_token_top_workspace_bytes(T, V, q.BF16, k)
    ws = torch.empty(max(n, 1), dtype=torch.uint8, device=logits.device)
    q.qlora_token_top(logits, V, T, V, q.BF16, None, 1.0, k, ids, top, None, None, ws, n)
    return ids, top


def distill_steps(student, h, ids, top, weight, steps, lr=0.02):
    """Losses of `steps` steps."""
    T, V = student.logits.shape
    loss, kl = torch.empty(1, device=h.device), torch.empty(T, device=h.device)
    n = q.qlora_distill_workspace_bytes(T, V, q.BF16, ids.shape[1])
    ws = torch.empty(max(n, 1), dtype=torch.uint8, device=h.device)
    losses = []
    for _ in range(steps):
        logits = student.forward(h)
        q.qlora_distill_logits(logits, V, T, V, q.BF16, 1.0, weight, ids.shape[1], ids, top, True,
                               loss, kl, logits, V, ws, n)
        student.backward(h, logits)
        student.update(lr)
        losses.append(loss.clone())
    return torch.cat(losses).tolist() if losses else []


def batch(tokens, hidden, vocab, seed, device):
    """Random hidden states and a teacher that is a linear map of them."""
    g = torch.Generator(device)
    g.manual_seed(seed)
    h = torch.randn(tokens, hidden, generator=g, device=device)
    W = torch.randn(hidden, vocab, generator=g, device=device) * (3.0 / hidden ** 0.5)
    return h.to(torch.bfloat16), (h @ W).to(torch.bfloat16)


def main():
    ap = argparse.ArgumentParser()
    ap.add_argument("--tokens", type=int, default=512)
    ap.add_argument("--steps", type=int, default=20)
    ap.add_argument("--hidden", type=int, default=1024)
    ap.add_argument("--inner", type=int, default=2752)
    ap.add_argument("--vocab", type=int, default=32000)
    ap.add_argument("--rank", type=int, default=16)
    ap.add_argument("--alternatives", type=int, default=32)
    args = ap.parse_args()
    dev = torch.device("cuda:0")
    h, teacher = batch(args.tokens, args.hidden, args.vocab, 0, dev)
    ids, top = alternatives(teacher, args.alternatives)
    student = Student(args.hidden, args.inner, args.vocab, args.rank, args.tokens, dev)
    weight = torch.full((args.tokens,), 1.0 / args.tokens, device=dev)
    losses = distill_steps(student, h, ids, top, weight, args.steps)
    print(f"divergence from the teacher's alternatives {losses[0]:.4f} -> {losses[-1]:.4f}")


if __name__ == "__main__":
    main()
