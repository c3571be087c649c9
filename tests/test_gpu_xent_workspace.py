"""GPU test that the linear cross entropy's results do not depend on what its
workspace holds, and that nothing past the workspace's end is written."""
import pytest
import torch

import thread_register_tile_amd as trt
from test_gpu_xent import BF16, F16, Case, _gpu  # noqa: F401

pytestmark = pytest.mark.gpu


def workspace(need, fill, guard):
    ws = torch.full((need + 4096,), fill, dtype=torch.uint8, device="cuda")
    ws[need:] = guard
    return ws


def step(c, lse, fill, guard, piece):
    need = trt.linear_xent_workspace_size(c.T, c.V, c.D)
    ws = workspace(need, fill, guard)
    out = trt.linear_xent(c.x, c.w, c.target, workspace=ws[:need])
    assert (ws[need:] == guard).all(), (c.what, "forward")
    lse = out[1].clone() if lse is None else lse
    need = trt.linear_xent_bwd_workspace_size(c.T, c.V, c.D, piece)
    ws = workspace(need, fill, guard)
    grads = trt.linear_xent_bwd(c.x, c.w, c.target, lse, c.dloss, piece=piece, workspace=ws[:need])
    assert (ws[need:] == guard).all(), (c.what, "backward")
    return lse, (*out, *grads)


# the stream over W, few tokens, the list, 256-wide tiles, operands that the
# copies do not take, and several pieces
@pytest.mark.parametrize("T,V,D,dtype,ignored,piece", [
    (3, 900, 64, BF16, 0.0, 0), (30, 700, 136, F16, 0.2, 0), (400, 5001, 136, F16, 0.3, 0),
    (1030, 12500, 72, BF16, 0.4, 0), (300, 777, 33, F16, 0.3, 0), (260, 1100, 264, BF16, 0.2, 320)])
def test_results_whatever_the_workspace_holds(T, V, D, dtype, ignored, piece):
    c = Case(T, V, D, dtype, seed=T + D, ignored=ignored, weights="each")
    lse, first = step(c, None, 0, 0x5A, piece)
    assert all(t.isfinite().all() for t in first)
    for fill, guard in ((0x3C, 0xA5), (0xFF, 0x11), (0x80, 0x7F), (0, 0xFF)):
        _, again = step(c, lse, fill, guard, piece)
        assert all(torch.equal(a, b) for a, b in zip(first, again)), (fill, c.what)
