"""Linear cross entropy in 64 bits, from the definitions (numpy; test
infrastructure only).

x: [tokens, width], w: [vocab, width] float64; target: [tokens] int64.
Tokens whose target is `ignore` take part in nothing.
"""
import numpy as np


def logits(x, w, target, ignore):
    """Logits of the live tokens, and the mask of those."""
    live = target != ignore
    return x[live] @ w.T, live


def forward(x, w, target, ignore=-100):
    """(loss, lse)."""
    z, live = logits(x, w, target, ignore)
    loss, lse = np.zeros(len(target)), np.zeros(len(target))
    m = z.max(1, keepdims=True)
    lse[live] = (m + np.log(np.exp(z - m).sum(1, keepdims=True)))[:, 0]
    # log(1 + the others' exp(z - z_target)): no cancellation of two large
    # numbers, and no loss of a small one against 1
    at = target[live]
    rel = z - z[np.arange(len(z)), at][:, None]
    rel[np.arange(len(z)), at] = -np.inf
    top = np.maximum(rel.max(1, keepdims=True), -1e300)
    with np.errstate(divide="ignore"):
        others = (top + np.log(np.exp(rel - top).sum(1, keepdims=True)))[:, 0]
    loss[live] = np.logaddexp(0.0, others)
    return loss, lse


def dlogits(x, w, target, dloss, dlse=None, ignore=-100):
    """(g, p) of the live tokens, and their mask."""
    z, live = logits(x, w, target, ignore)
    p = np.exp(z - z.max(1, keepdims=True))
    p /= p.sum(1, keepdims=True)
    both = dloss[live] + (0.0 if dlse is None else dlse[live])
    g = p * both[:, None]
    g[np.arange(len(z)), target[live]] -= dloss[live]
    return g, p, live


def backward(x, w, target, dloss, dlse=None, ignore=-100):
    """(dx, dw)."""
    g, _, live = dlogits(x, w, target, dloss, dlse, ignore)
    dx = np.zeros_like(x)
    dx[live] = g @ w
    return dx, g.T @ x[live]
