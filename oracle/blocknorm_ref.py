"""A block's norms with its gate and residual, and their gradients, in 64 bits
from the definitions (numpy; test infrastructure only).

    u = N(y) pg + pb (or y),  r' = alpha r + gate u,  h = N(r') g + b

r, y, dh, dr: [rows, cols] float64; gate: [rows, cols] (each row's own, already
spread); vectors [cols] or None.  N: layer norm, or the root mean square norm.
"""
import numpy as np


def norm(x, eps, rms):
    """(N(x), 1 / sqrt(... + eps) per row)."""
    d = x if rms else x - x.mean(1, keepdims=True)
    r = 1.0 / np.sqrt((d * d).mean(1, keepdims=True) + eps)
    return d * r, r


def norm_back(v, hat, rstd, rms):
    """The norm's Jacobian, transposed, on v."""
    return rstd * (v - hat * (v * hat).mean(1, keepdims=True) - (0.0 if rms else v.mean(1, keepdims=True)))


def one(v):
    return 1.0 if v is None else v


def zero(v):
    return 0.0 if v is None else v


def forward(r, y, gate, pg, pb, g, b, alpha, eps, rms, post):
    u = norm(y, eps, rms)[0] * one(pg) + zero(pb) if post else y
    out = alpha * r + one(gate) * u
    return out, norm(out, eps, rms)[0] * one(g) + zero(b)


def spread(gate, rows, span):
    """Gate rows as one for each row."""
    return None if gate is None else gate[np.arange(rows) // span]


def gather(each, span):
    """The sums of each gate row's rows."""
    return np.stack([each[i:i + span].sum(0) for i in range(0, len(each), span)])


def backward(dh, dr, r_out, y, gate, pg, pb, g, alpha, eps, rms, post):
    """A dict of dr, dy, dgate (each row's own), dpg, dpb, dg, db; dh or dr may be None."""
    rows, cols = y.shape
    e = np.zeros((rows, cols)) if dr is None else dr
    out = {}
    if dh is not None:
        hat, rstd = norm(r_out, eps, rms)
        e = e + norm_back(dh * one(g), hat, rstd, rms)
        out.update(dg=(dh * hat).sum(0), db=dh.sum(0))
    du = one(gate) * e
    hat, rstd = norm(y, eps, rms) if post else (y, None)
    out.update(dr=alpha * e, dgate=e * (hat * one(pg) + zero(pb)))
    out["dy"] = norm_back(du * one(pg), hat, rstd, rms) if post else du
    if post:
        out.update(dpg=(du * hat).sum(0), dpb=du.sum(0))
    return out
