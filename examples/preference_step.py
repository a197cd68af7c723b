"""Adapters of a 4-bit output head trained on preferences, then by policy steps.

    python examples/preference_step.py [--pairs 8] [--steps 20]

One process, one GPU, every step on it: dropout of the hidden states (its mask
is drawn again in the backward, never stored), the adapted 4-bit head, the
log-probabilities of the answers' tokens, the preference loss against the head
without its adapters, the logits' gradient in the logits' own memory, and the
head's backward with the Adam step of A and B fused in.  The policy steps take
the objective from the logits to their gradient in one call.  Hidden states and
answers are random: what it shows is how the calls fit together.
"""

import argparse
import os
import sys

import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)

from quantized_rank_fine_amd import qlora as q  # noqa: E402


class AdaptedHead:
    """A frozen 4-bit head [hidden, vocab] with adapters of rank r and the
    buffers of one batch of `tokens` tokens."""

    def __init__(self, W0, rank, tokens, seed=0):
        dev = W0.device
        self.hidden, self.vocab = W0.shape
        self.rank, self.tokens = rank, tokens
        self.wq = q.NF4Weight(self.hidden, self.vocab, dev)
        q.qlora_quantize(W0, self.wq)
        g = torch.Generator(dev)
        g.manual_seed(seed)
        A = torch.randn(self.hidden, rank, generator=g, device=dev) / self.hidden ** 0.5
        B = torch.zeros(rank, self.vocab, device=dev)
        self.state = [[p, torch.zeros_like(p), torch.zeros_like(p), p.to(torch.bfloat16)]
                      for p in (A, B)]
        bf16 = lambda *s: torch.empty(*s, dtype=torch.bfloat16, device=dev)  # noqa: E731
        self.x, self.dx = bf16(tokens, self.hidden), bf16(tokens, self.hidden)
        self.logits = bf16(tokens, self.vocab)
        self.xa = torch.empty(tokens, rank, device=dev)
        n = max(q.qlora_fwd_workspace_bytes(tokens, self.hidden, self.vocab, rank),
                q.qlora_bwd_workspace_bytes(tokens, self.hidden, self.vocab, rank),
                q.qlora_fwd_workspace_bytes(tokens, self.hidden, self.vocab, 0))
        self.ws, self.ws_bytes = torch.empty(n, dtype=torch.uint8, device=dev), n
        self.step = 0

    def forward(self, h, p=0.0, seed=0, adapters=True):
        """logits of dropout(h); adapters=False: of h under the frozen head."""
        if not adapters:
            q.qlora_linear_fwd(self.wq, h, self.tokens, q.BF16, None, None, 0, q.BF16,
                               self.logits, None, self.ws, self.ws_bytes)
            return self.logits
        self.drop = (p, seed, self.step)
        q.qlora_dropout(h, self.hidden, None, 0, self.tokens, self.hidden, q.BF16, p, seed,
                        self.step, self.x, self.hidden)
        A, B = self.state[0][3], self.state[1][3]
        q.qlora_linear_fwd(self.wq, self.x, self.tokens, q.BF16, A, B, self.rank, q.BF16,
                           self.logits, self.xa, self.ws, self.ws_bytes)
        return self.logits

    def backward_and_update(self, dlogits, lr):
        """Adam step of A and B; returns the gradient of h."""
        self.step += 1
        A, B = self.state[0][3], self.state[1][3]
        q.qlora_linear_bwd_adam(self.wq, self.x, dlogits, self.tokens, q.BF16, A, B, self.rank,
                                q.BF16, self.xa, self.dx, *self.state, self.step, lr, self.ws,
                                self.ws_bytes)
        p, seed, counter = self.drop
        q.qlora_dropout(self.dx, self.hidden, None, 0, self.tokens, self.hidden, q.BF16, p, seed,
                        counter, self.dx, self.hidden)
        return self.dx


class TokenScores:
    """log-probabilities of labels under logits, and the way back."""

    def __init__(self, tokens, vocab, device):
        f = lambda *s: torch.empty(*s, device=device)  # noqa: E731
        self.T, self.V = tokens, vocab
        self.logp, self.stats, self.entropy = f(tokens), f(tokens, 2), f(tokens)
        n = q.qlora_token_logp_workspace_bytes(tokens, vocab, q.BF16)
        self.ws, self.ws_bytes = torch.empty(max(n, 1), dtype=torch.uint8, device=device), n

    def __call__(self, logits, labels):
        q.qlora_token_logp_fwd(logits, self.V, self.T, self.V, q.BF16, labels, 1.0, self.logp,
                               self.stats, self.entropy, self.ws, self.ws_bytes)
        return self.logp

    def backward_(self, logits, labels, g):
        """The logits' gradient, in the logits' memory."""
        q.qlora_token_logp_bwd(logits, self.V, self.T, self.V, q.BF16, labels, 1.0, self.stats,
                               None, g, None, logits, self.V)
        return logits


def preference_steps(head, h, labels, mask, cu, steps, lr=1e-3, p=0.05, seed=1, beta=0.1):
    """Losses of `steps` preference steps, and the last rewards."""
    dev, T = h.device, head.tokens
    P = (cu.numel() - 1) // 2
    score = TokenScores(T, head.vocab, dev)
    ref = score(head.forward(h, adapters=False), labels).clone()
    loss, rewards = torch.empty(1, device=dev), torch.empty(2 * P, device=dev)
    g = torch.empty(T, device=dev)
    n = q.qlora_pref_workspace_bytes(P, T)
    ws = torch.empty(max(n, 1), dtype=torch.uint8, device=dev)
    pref = q.pref_struct(q.PREF_SIGMOID, beta)
    losses = []
    for _ in range(steps):
        logits = head.forward(h, p, seed)
        q.qlora_pref_loss(score(logits, labels), ref, mask, cu, P, T, pref, loss, rewards, g, ws, n)
        head.backward_and_update(score.backward_(logits, labels, g), lr)
        losses.append(loss.clone())
    return torch.cat(losses).tolist(), rewards


def policy_steps(head, h, labels, weight, adv, steps, lr=1e-4, p=0.0, seed=2):
    """Losses of `steps` clipped policy steps on one batch of answers."""
    dev, T, V = h.device, head.tokens, head.vocab
    score = TokenScores(T, V, dev)
    ref = score(head.forward(h, adapters=False), labels).clone()
    old = score(head.forward(h), labels).clone()
    out = torch.empty(4, device=dev)
    n = q.qlora_policy_logits_workspace_bytes(T, V, q.BF16)
    ws = torch.empty(n, dtype=torch.uint8, device=dev)
    policy = q.policy_struct(q.OBJ_CLIP, 0.2, 0.28, 0.0, kl_coef=0.02)
    losses = []
    for _ in range(steps):
        logits = head.forward(h, p, seed)
        q.qlora_policy_logits(logits, V, T, V, q.BF16, labels, 1.0, weight, adv, old, ref, policy,
                              out, None, logits, V, ws, n)
        head.backward_and_update(logits, lr)
        losses.append(out[:1].clone())
    return torch.cat(losses).tolist()


def batch(pairs, hidden, vocab, seed, device, longest=48):
    """Random hidden states and packed answers: chosen ones first, the first
    quarter of each its prompt."""
    g = torch.Generator().manual_seed(seed)
    n = torch.randint(longest // 2, longest + 1, (2 * pairs,), generator=g)
    cu = torch.cat([torch.zeros(1, dtype=torch.int64), n.cumsum(0)])
    T = int(cu[-1])
    mask = torch.cat([(torch.arange(k) >= k // 4).to(torch.uint8) for k in n.tolist()])
    h = torch.randn(T, hidden, generator=g).to(torch.bfloat16)
    labels = torch.randint(0, vocab, (T,), generator=g)
    return [t.to(device) for t in (h, labels, mask, cu)]


def main():
    ap = argparse.ArgumentParser()
    ap.add_argument("--pairs", type=int, default=8)
    ap.add_argument("--steps", type=int, default=20)
    ap.add_argument("--hidden", type=int, default=1024)
    ap.add_argument("--vocab", type=int, default=32000)
    ap.add_argument("--rank", type=int, default=16)
    args = ap.parse_args()
    dev = torch.device("cuda:0")
    h, labels, mask, cu = batch(args.pairs, args.hidden, args.vocab, 0, dev)
    W0 = torch.randn(args.hidden, args.vocab, device=dev) * 0.02
    head = AdaptedHead(W0, args.rank, h.shape[0])
    losses, rewards = preference_steps(head, h, labels, mask, cu, args.steps)
    margin = (rewards[:args.pairs] - rewards[args.pairs:]).mean().item()
    print(f"preference loss {losses[0]:.4f} -> {losses[-1]:.4f}, reward margin {margin:.3f}")
    live = mask.float()
    adv = torch.randn(h.shape[0], device=dev)
    losses = policy_steps(head, h, labels, live / live.sum(), adv, args.steps)
    print(f"policy loss {losses[0]:.4f} -> {losses[-1]:.4f}")


if __name__ == "__main__":
    main()
