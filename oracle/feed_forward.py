"""64-bit definition of the gated feed-forward block and of its gradients."""
from __future__ import annotations

import numpy as np

from .block import sigmoid, swiglu


def _halves(pre, layout):
    a, b = np.split(pre, 2, axis=1)
    return (a, b) if layout == 0 else (b, a)


def forward(x, w13, w2, layout=0, limit=np.inf, alpha=1.0, beta=0.0):
    """(pre [M, 2 I] in w13's order, h, y)."""
    pre = x @ w13.T
    h = swiglu(*_halves(pre, layout), limit, alpha, beta)
    return pre, h, h @ w2.T


def act_grad(pre, dh, layout=0, limit=np.inf, alpha=1.0, beta=0.0):
    """d(up, gate) [M, 2 I] in w13's order, of dh [M, I]."""
    u, g = _halves(pre, layout)
    uc, gc = np.clip(u, -limit, limit), np.minimum(g, limit)
    s = sigmoid(alpha * gc)
    du = dh * gc * s * (np.abs(u) <= limit)
    dg = dh * (uc + beta) * (s + alpha * gc * s * (1 - s)) * (g <= limit)
    return np.concatenate((du, dg) if layout == 0 else (dg, du), axis=1)


def backward(dy, x, w13, w2, layout=0, limit=np.inf, alpha=1.0, beta=0.0):
    """(dx, dw13, dw2) of y at dy."""
    pre, h, _ = forward(x, w13, w2, layout, limit, alpha, beta)
    d = act_grad(pre, dy @ w2, layout, limit, alpha, beta)
    return d @ w13, d.T @ x, dy.T @ h
