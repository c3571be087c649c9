"""GPU test of the linear cross entropy's gradients where G is held as two
numbers, the rounded value and what the rounding left: batches of up to 64
tokens.

Tolerances as in test_gpu_xent.py, with the inputs' half step h squared in the
error of g: the second number is off by h of itself, and itself no more than h
of g.  Results in binary32, so that nothing but G's own rounding could hide it.
"""
import numpy as np
import pytest
import torch

from oracle import xent_ref
from test_gpu_xent import BF16, F16, NAMES, U, Case, _gpu, check, f64, half_step  # noqa: F401

pytestmark = pytest.mark.gpu


def check_gradients(c, **kw):
    dx, dw = c.backward(out_dtype=torch.float32, **kw)
    hl, he = f64(c.dloss), None if c.dlse is None else f64(c.dlse)
    g, p, live = xent_ref.dlogits(c.hx, c.hw, c.ht, hl, he, -100)
    rdx, rdw = xent_ref.backward(c.hx, c.hw, c.ht, hl, he, -100)
    _, _, e, _ = c.bounds()
    both = hl if he is None else hl + he
    s = np.maximum(np.abs(hl), np.abs(both))[live][:, None]
    h = torch.finfo(c.dtype).eps / 2
    least = 2.0 ** -39 if c.dtype == F16 else 2.0 ** -134
    dg = h * h * np.abs(g) + e[:, None] * p * s + least * (s.max() if s.size else 0.0)
    ax, aw, ag = np.abs(c.hx[live]), np.abs(c.hw), np.abs(g)
    tol = np.zeros_like(rdx)
    tol[live] = dg @ aw + U * (2 * c.V + 4) * (ag @ aw)
    check(dx, rdx, half_step(rdx, torch.float32) + tol, c.what + " dx")
    tol = dg.T @ ax + U * (2 * c.T + 4) * (ag.T @ ax)
    check(dw, rdw, half_step(rdw, torch.float32) + tol, c.what + " dw")


@pytest.mark.parametrize("dtype", [F16, BF16], ids=NAMES.get)
@pytest.mark.parametrize("T,V,D", [(1, 40, 16), (2, 300, 64), (31, 130, 33), (63, 65, 264), (64, 500, 72)])
def test_gradients_keep_what_the_rounding_leaves(T, V, D, dtype):
    check_gradients(Case(T, V, D, dtype, seed=T, weights="each"))
    check_gradients(Case(T, V, D, dtype, seed=D, ignored=0.3, dlse=True), piece=64)
