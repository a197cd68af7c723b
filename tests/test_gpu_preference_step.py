"""The example's training steps: dropout, the adapted 4-bit head, the token
scores, the losses and the update together."""

import os
import sys

import numpy as np
import pytest

from oracle import objective as ob
from gpu_harness import bf16_to_f64, torch_dev

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                                "examples"))

pytestmark = pytest.mark.gpu


def test_preference_and_policy_steps():
    import preference_step as ex
    torch, dev = torch_dev()
    P, hidden, vocab = 3, 256, 640
    h, labels, mask, cu = ex.batch(P, hidden, vocab, 4, dev)
    torch.manual_seed(5)
    W0 = torch.randn(hidden, vocab, device=dev) * 0.05
    head = ex.AdaptedHead(W0, 16, h.shape[0])
    losses, rewards = ex.preference_steps(head, h, labels, mask, cu, 12)
    # B = 0 at the start: without dropout the model is its reference, so the
    # first loss is near log 2; then the pairs are learned
    assert abs(losses[0] - np.log(2)) < 0.2
    assert losses[-1] < 0.7 * losses[0]
    assert bool((rewards[:P] > rewards[P:]).all())
    live = mask.float()
    torch.manual_seed(6)
    adv = torch.randn(h.shape[0], device=dev)
    pol = ex.policy_steps(head, h, labels, live / live.sum(), adv, 6)
    assert pol[-1] < pol[0]
    assert all(np.isfinite(losses)) and all(np.isfinite(pol))


def test_first_preference_loss_is_the_oracles():
    """The loss of the chain's own logits (read back in bf16) in float64."""
    import preference_step as ex
    from quantized_rank_fine_amd import qlora as q
    torch, dev = torch_dev()
    P, hidden, vocab = 2, 192, 320
    h, labels, mask, cu = ex.batch(P, hidden, vocab, 7, dev)
    T = h.shape[0]
    torch.manual_seed(8)
    W0 = torch.randn(hidden, vocab, device=dev) * 0.05
    head = ex.AdaptedHead(W0, 8, T)
    read = lambda: bf16_to_f64(head.logits).reshape(T, vocab)  # noqa: E731
    y = labels.cpu().numpy()
    head.forward(h, adapters=False)
    ref = ob.token_logp(read(), y)[0]
    head.forward(h, 0.05, 1)
    lp = ob.token_logp(read(), y)[0]
    want, rewards, g = ob.pref_loss("sigmoid", lp, ref, mask.cpu().numpy(), cu.cpu().numpy(), 0.1)
    losses, got = ex.preference_steps(head, h, labels, mask, cu, 1, p=0.05, seed=1)
    # logp to 1e-6 each, under 48 tokens an answer, beta 0.1
    assert abs(losses[0] - want) <= 1e-5
    assert np.all(np.abs(got.cpu().numpy() - rewards) <= 1e-5 * (1 + np.abs(rewards)))
    assert q.qlora_pref_workspace_bytes(P, T) == 0        # one launch at this size
