"""GPU tests of the linear cross entropy's gradients for upstream gradients that
are not finite, dlse among them: such a token spoils its own row of dX, and dW,
and is never taken for one without weight."""
import pytest
import torch

from test_gpu_xent import BF16, F16, Case, _gpu  # noqa: F401

pytestmark = pytest.mark.gpu

INF, NAN = float("inf"), float("nan")


@pytest.mark.parametrize("dtype", [F16, BF16], ids=["f16", "bf16"])
@pytest.mark.parametrize("T", [40, 100, 300])
@pytest.mark.parametrize("dloss,dlse", [(0.0, NAN), (-0.0, NAN), (0.0, INF), (0.0, -INF), (1e-3, NAN), (1e-3, INF), (INF, -INF),
                                        (NAN, 0.0), (NAN, NAN)])
def test_a_token_spoils_its_own_row(dloss, dlse, T, dtype):
    # the token's weight is never the largest finite one, so no other row changes
    c = Case(T, 500, 64, dtype, seed=16, weights="each", dlse=True)
    c.dloss[3], c.dlse[3] = 0.0, 1e-6
    clean, _ = c.backward()
    c.dloss[3], c.dlse[3] = dloss, dlse
    dx, dw = c.backward()
    rest = torch.arange(T, device="cuda") != 3
    assert not dx[3].isfinite().any() and torch.equal(dx[rest], clean[rest])
    assert not dw.isfinite().all()


@pytest.mark.parametrize("dloss,dlse", [(0.0, 0.0), (-0.0, 0.0), (0.0, -0.0)])
def test_a_token_without_weight_takes_no_part(dloss, dlse):
    c = Case(150, 500, 64, BF16, seed=17, weights="each", dlse=True)
    c.dloss[3], c.dlse[3] = dloss, dlse
    c.x[3] = NAN
    dx, dw = c.backward()
    assert (dx[3] == 0).all() and dx.isfinite().all() and dw.isfinite().all()


def test_weights_that_cancel_leave_the_target_alone():
    # dloss + dlse = 0: g is -dloss at the target and zero elsewhere
    c = Case(30, 200, 64, BF16, seed=18, dlse=True)
    c.dloss[3], c.dlse[3] = 0.5, -0.5
    dx, _ = c.backward(out_dtype=torch.float32)
    want = -0.5 * c.w[c.target[3]].float()
    # the quotient by c, its product with W and with c: three roundings
    assert ((dx[3] - want).abs() <= 4 * 2.0 ** -24 * want.abs()).all()
