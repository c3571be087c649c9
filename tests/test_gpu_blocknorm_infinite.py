"""GPU tests of the block norm's gradients where a sum or a factor is infinite:
a result is infinite, not a NaN, wherever its definition is."""
import numpy as np
import pytest
import torch

import thread_register_tile_amd as trt

pytestmark = pytest.mark.gpu

F16, BF16, F32 = torch.float16, torch.bfloat16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    trt.lib()


def f64(t):
    return t.detach().cpu().to(torch.float64).numpy()


def normal(gen, *shape):
    return torch.randn(*shape, device="cuda", generator=gen)


@pytest.mark.parametrize("gate", ["channel", "sequence", "each"])
@pytest.mark.parametrize("post", [False, True])
@pytest.mark.parametrize("dtype", [F16, BF16, F32])
def test_gate_gradient_without_post_beta(gate, post, dtype):
    """dgate = sum of e u: infinite where e is, whatever the gate covers."""
    gen = torch.Generator(device="cuda").manual_seed(0)
    y, dr = (normal(gen, 20, 100).to(dtype) for _ in range(2))
    dr[3, 7], dr[13, 99] = float("inf"), -float("inf")
    gt = torch.ones({"channel": (100,), "sequence": (4, 100), "each": (20, 100)}[gate], dtype=dtype, device="cuda")
    got = f64(trt.block_norm_bwd(None, dr, None, y, gt, post=post, rms=True, rows_per_gate=5 if gate == "sequence" else None)[2])
    got = got.reshape(-1, 100)
    span = {"channel": 20, "sequence": 5, "each": 1}[gate]
    u = f64(y)                                  # (the norm's factor is positive: the sign is y's)
    want = {(3 // span, 7): np.sign(u[3, 7]) * np.inf, (13 // span, 99): -np.sign(u[13, 99]) * np.inf}
    for at, value in want.items():
        assert got[at] == value, (at, got[at], value)
    rest = np.ones(got.shape, bool)
    for at in want:
        rest[at] = False
    assert np.isfinite(got[rest]).all()


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_gate_gradient_where_the_sum_of_e_overflows(dtype):
    """e = 2^127 in two rows, y = 2^-10: dgate = 2^118, though the sum of e alone
    is past binary32."""
    dr, y = (torch.full((2, 40), v, dtype=dtype, device="cuda") for v in (2.0 ** 127, 2.0 ** -10))
    got = trt.block_norm_bwd(None, dr, None, y, torch.ones(40, dtype=dtype, device="cuda"), post=False)[2]
    assert (got.double() == 2.0 ** 118).all()
