"""GPU test of layer norms of rows whose variance is not a binary32 number: the
squares of the deviations overflow, and so does the square of the mean's
correction, whose difference is NaN.  No finite values may come of it."""
import pytest
import torch

import thread_register_tile_amd as trt

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
@pytest.mark.parametrize("cols", [500, 1500, 6000, 12000])
def test_variance_that_is_not_a_number(cols, dtype):
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    gen = torch.Generator(device="cuda").manual_seed(cols)
    x, dy = (torch.randn(9, cols, generator=gen, device="cuda").to(dtype) for _ in range(2))
    clean, (dclean, _, _) = trt.layernorm(x), trt.layernorm_bwd(dy, x)
    # deviations of about 2^108 around 2^112, whose mean binary32 rounds by about
    # 2^88: the squares of both are beyond 2^128, the row's sum is not
    x[4] = x[4] * 2.0 ** 108 + 2.0 ** 112
    y, (dx, dg, _) = trt.layernorm(x), trt.layernorm_bwd(dy, x)
    rest = torch.arange(9, device="cuda") != 4
    assert torch.equal(y[rest], clean[rest]) and torch.equal(dx[rest], dclean[rest])
    # NaN, or zeros where the correction happens to be none (variance infinity)
    assert (y[4].isnan() | (y[4] == 0)).all(), y[4][:8]
    assert (dx[4].isnan() | (dx[4] == 0)).all(), dx[4][:8]
