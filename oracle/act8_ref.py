"""Activations in 8 bits, in 64 bits from the definitions (numpy; test
infrastructure only).

Of every 32 columns of a row: X = floor(log2(largest |x|)) + 127, at least 7, or
255 where something is not finite; q = x / 2^(X - 133) rounded to nearest even,
held to [-127, 127]; an element stands for q 2^(X - 133).
"""
import numpy as np

BLOCK = 32


def pack(x):
    """(q int8 [rows, cols], scale uint8 [rows, blocks]) of float64 rows."""
    rows, cols = x.shape
    q = np.zeros((rows, cols), np.int8)
    scale = np.zeros((rows, -(-cols // BLOCK)), np.uint8)
    for b in range(scale.shape[1]):
        part = x[:, b * BLOCK:(b + 1) * BLOCK]
        fine = np.isfinite(part).all(1)
        top = np.where(fine, np.abs(np.where(fine[:, None], part, 0)).max(1), 0)
        X = np.where(top > 0, np.frexp(top)[1] - 1 + 127, 0)
        X = np.where(fine, np.maximum(X, 7), 255)
        with np.errstate(invalid="ignore"):
            steps = np.clip(np.rint(np.ldexp(part, (133 - X)[:, None])), -127, 127)
        q[:, b * BLOCK:(b + 1) * BLOCK] = np.where(fine[:, None], steps, 0)
        scale[:, b] = X
    return q, scale


def unpack(q, scale):
    """What 8-bit rows stand for, in float64."""
    X = scale.astype(np.int64)[:, np.arange(q.shape[1]) // BLOCK]
    v = np.ldexp(q.astype(np.float64), X - 133)
    return np.where(X == 255, np.nan, v)


def weight_grad(dy, q, scale):
    """dy^T x for float64 dy [tokens, outputs]."""
    return dy.T @ unpack(q, scale)
