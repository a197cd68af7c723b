"""Adam and orthogonalised updates of the adapter matrices, in float64 (oracle).

TEST INFRASTRUCTURE ONLY -- see ``oracle/__init__.py``.

"QLoRA (low-rank adapters on a quantized model)", "The code, line by line":
the optimizer is handed only A and B (Adam over the adapter matrices), so
nothing else changes; "LoRA & QLoRA" builds the same step with AdamW.  The
pages print neither the update nor its constants, so this follows the
published algorithm (Kingma & Ba, "Adam: A Method for Stochastic
Optimization", Algorithm 1), with decoupled weight decay as in AdamW
(Loshchilov & Hutter, "Decoupled Weight Decay Regularization"): at step t,

  m <- beta1 m + (1 - beta1) g
  v <- beta2 v + (1 - beta2) g^2
  theta <- theta - lr ( (m / (1 - beta1^t)) / (sqrt(v / (1 - beta2^t)) + eps)
                        + weight_decay * theta )

``weight_decay = 0`` is plain Adam.

The orthogonalised update (Jordan et al., "Muon: an optimizer for hidden
layers in neural networks") puts f(s) in the place of each singular value s of
the momentum's direction over its Frobenius norm, f being `steps` times
s -> a s + b s^3 + c s^5; computed here from the singular value decomposition.
"""

import numpy as np


def adam_step(theta, g, m, v, t, lr, beta1=0.9, beta2=0.999, eps=1e-8, weight_decay=0.0):
    """One step; returns new (theta, m, v) as float64 arrays (inputs unchanged)."""
    theta = np.asarray(theta, np.float64)
    g = np.asarray(g, np.float64)
    m = beta1 * np.asarray(m, np.float64) + (1.0 - beta1) * g
    v = beta2 * np.asarray(v, np.float64) + (1.0 - beta2) * g * g
    m_hat = m / (1.0 - beta1 ** t)
    v_hat = v / (1.0 - beta2 ** t)
    theta = theta - lr * (m_hat / (np.sqrt(v_hat) + eps) + weight_decay * theta)
    return theta, m, v


def orthogonalize(u, coef=(3.4445, -4.7750, 2.0315), steps=5, eps=1e-7):
    """The Newton-Schulz image of u (2-D), as float64."""
    u = np.asarray(u, np.float64)
    norm = np.linalg.norm(u) + eps
    if norm == 0.0:
        return np.zeros_like(u)
    left, s, right = np.linalg.svd(u / norm, full_matrices=False)
    for _ in range(steps):
        s = s * (coef[0] + s * s * (coef[1] + s * s * coef[2]))
    return (left * s) @ right


def muon_step(theta, g, m, lr, momentum=0.95, nesterov=True, weight_decay=0.0, eps=1e-7,
              steps=5, coef=(3.4445, -4.7750, 2.0315), scale=1.0):
    """One step; returns new (theta, m, X) as float64 arrays (m None: no momentum)."""
    g = np.asarray(g, np.float64)
    u = g
    if m is not None:
        m = momentum * np.asarray(m, np.float64) + g
        u = g + momentum * m if nesterov else m
    x = orthogonalize(u, coef, steps, eps)
    theta = np.asarray(theta, np.float64)
    return theta - lr * (scale * x + weight_decay * theta), m, x
