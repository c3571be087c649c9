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


# widths of every number of waves to a row whose workgroups take several rows,
# and numbers of rows that leave some of those waves without one
IDLE = [(rows, cols) for cols in (3, 100, 1000, 1200, 2000, 2800, 4000) for rows in (1, 5, 3001)]


@pytest.mark.parametrize("rows,cols", IDLE)
@pytest.mark.parametrize("rms", [False, True])
@pytest.mark.parametrize("bits", [8, 16])
def test_infinite_gate_of_the_first_row(rows, cols, rms, bits):
    """dpost_beta = sum of gate e and dpost_gamma = sum of gate e N(y), in a column
    where the first row's gate is infinite: so are they, whatever the rows are."""
    gen = torch.Generator(device="cuda").manual_seed(cols)
    y, dr, gate = normal(gen, rows, cols).to(BF16), normal(gen, rows, cols).abs().to(BF16) + 0.25, normal(gen, rows, cols).to(BF16)
    at = cols // 2
    y[0, at] = 4 * y[0].abs().max()             # far above the mean
    gate[0, at] = float("inf")
    got = trt.block_norm_bwd(None, dr, None, trt.act8_pack(y) if bits == 8 else y, gate, rms=rms)
    for t in got[3:5]:
        assert t[at] == float("inf")
        assert t.isfinite().sum() == cols - 1


@pytest.mark.parametrize("rows,cols", [(r, c) for r, c in IDLE if c > 3])
@pytest.mark.parametrize("bits", [8, 16])
def test_infinite_gamma(rows, cols, bits):
    """An infinite gamma under the root mean square norm leaves e infinite with
    the sign of -N(r_out) dh[0] N(r_out)[0] in every other column: with equal rows
    the sums over them are too."""
    gen = torch.Generator(device="cuda").manual_seed(cols)
    x, y, dh = (normal(gen, 1, cols).sign().repeat(rows, 1).to(BF16) for _ in range(3))
    gamma = torch.ones(cols, device="cuda")
    gamma[0] = float("inf")
    saved = [trt.act8_pack(t) if bits == 8 else t for t in (x, y)]
    got = trt.block_norm_bwd(dh, None, *saved, None, gamma=gamma, rms=True)
    e = -float("inf") * (x[0] * x[0, 0] * dh[0, 0]).float()
    assert got[4][0].isnan() and torch.equal(got[4][1:], e[1:])                 # dpost_beta
    assert torch.equal(got[3][1:], (e * y[0])[1:])                              # dpost_gamma
    assert torch.equal(got[6], dh.float().sum(0)) and got[5].isfinite().all()   # dbeta, dgamma
