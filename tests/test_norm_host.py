"""CPU tests of the layer norm's entry points: refusals before any HIP call,
workspace sizes, and the oracle's gradients against differences."""
import numpy as np
import pytest
import torch

import thread_register_tile_amd as trt
from oracle import norm_ref

BASE = 1 << 24     # fake, well-separated addresses: never dereferenced


def forward(**kw):
    a = dict(rows=8, cols=64, x=BASE, ldx=64, gamma=BASE * 2, beta=BASE * 3, eps=1e-5, y=BASE * 4, ldy=64,
             dtype=trt.F16, pdt=trt.F32)
    a.update(kw)
    return trt.lib().trt_layernorm(a["rows"], a["cols"], a["x"], a["ldx"], a["gamma"], a["beta"], a["eps"], a["y"],
                                   a["ldy"], a["dtype"], a["pdt"], None)


def backward(**kw):
    a = dict(rows=8, cols=64, dy=BASE, lddy=64, x=BASE * 2, ldx=64, gamma=BASE * 3, eps=1e-5, dx=BASE * 4, lddx=64,
             dgamma=BASE * 5, dbeta=BASE * 6, dtype=trt.F16, pdt=trt.F32, ws=BASE * 7, wsb=1 << 20)
    a.update(kw)
    return trt.lib().trt_layernorm_bwd(a["rows"], a["cols"], a["dy"], a["lddy"], a["x"], a["ldx"], a["gamma"],
                                       a["eps"], a["dx"], a["lddx"], a["dgamma"], a["dbeta"], a["dtype"], a["pdt"],
                                       a["ws"], a["wsb"], None)


@pytest.mark.parametrize("kw,code", [
    (dict(rows=0), trt.ERR_SIZE), (dict(cols=0), trt.ERR_SIZE), (dict(rows=-1), trt.ERR_SIZE),
    (dict(rows=(1 << 30) + 1), trt.ERR_SIZE), (dict(rows=1 << 30, ldx=1 << 60), trt.ERR_SIZE),
    (dict(ldx=0), trt.ERR_STRIDE), (dict(ldy=63), trt.ERR_STRIDE),
    (dict(x=0), trt.ERR_NULL), (dict(y=0), trt.ERR_NULL),
    (dict(x=BASE + 1), trt.ERR_ALIGN), (dict(y=BASE * 4 + 1), trt.ERR_ALIGN), (dict(gamma=BASE * 2 + 2), trt.ERR_ALIGN),
    (dict(y=BASE), trt.ERR_OVERLAP), (dict(y=BASE + 2 * 8 * 64 - 2), trt.ERR_OVERLAP),
    (dict(y=BASE * 2), trt.ERR_OVERLAP), (dict(y=BASE * 3), trt.ERR_OVERLAP),
    (dict(dtype=0), trt.ERR_DTYPE), (dict(dtype=trt.F16, pdt=trt.BF16), trt.ERR_DTYPE),
    (dict(dtype=trt.F32, pdt=trt.F16), trt.ERR_DTYPE),
    (dict(eps=-1.0), trt.ERR_ARG), (dict(eps=float("nan")), trt.ERR_ARG), (dict(eps=float("inf")), trt.ERR_ARG),
    (dict(cols=32769, ldx=32769, ldy=32769), trt.ERR_UNSUPPORTED),
    (dict(dtype=trt.F32, cols=16385, ldx=16385, ldy=16385), trt.ERR_UNSUPPORTED),
])
def test_forward_refusals(kw, code):
    assert forward(**kw) == code
    assert trt.last_error() != ""


@pytest.mark.parametrize("kw,code", [
    (dict(rows=0), trt.ERR_SIZE), (dict(lddy=0), trt.ERR_STRIDE), (dict(lddx=10), trt.ERR_STRIDE),
    (dict(dy=0), trt.ERR_NULL), (dict(x=0), trt.ERR_NULL), (dict(dx=0), trt.ERR_NULL),
    (dict(ws=0), trt.ERR_NULL), (dict(ws=0, dgamma=0), trt.ERR_NULL), (dict(wsb=100), trt.ERR_SIZE),
    (dict(wsb=-1), trt.ERR_SIZE), (dict(ws=BASE * 7 + 8), trt.ERR_ALIGN),
    (dict(dx=BASE), trt.ERR_OVERLAP), (dict(dx=BASE * 2), trt.ERR_OVERLAP), (dict(dgamma=BASE * 3), trt.ERR_OVERLAP),
    (dict(dbeta=BASE * 5), trt.ERR_OVERLAP), (dict(dgamma=BASE * 7), trt.ERR_OVERLAP), (dict(ws=BASE * 2), trt.ERR_OVERLAP),
    (dict(dgamma=BASE * 5 + 2), trt.ERR_ALIGN), (dict(pdt=9), trt.ERR_DTYPE), (dict(eps=-0.5), trt.ERR_ARG),
    (dict(cols=40000, lddy=40000, ldx=40000, lddx=40000), trt.ERR_UNSUPPORTED),
])
def test_backward_refusals(kw, code):
    assert backward(**kw) == code
    assert trt.last_error() != ""


def test_workspace_size():
    for dt in (trt.F16, trt.BF16, trt.F32):
        for rows, cols in ((1, 1), (7, 500), (100000, 4096), (1 << 30, 8)):
            n = trt.layernorm_bwd_workspace_size(rows, cols, dt)
            assert n > 0 and n % (8 * cols) == 0 and n // (8 * cols) <= min(rows, 512)
    for bad in ((0, 4, trt.F16), (4, 0, trt.F16), (4, 4, 7), (4, 40000, trt.F16)):
        with pytest.raises(trt.TrtError):
            trt.layernorm_bwd_workspace_size(*bad)


def test_binding_refuses_what_it_cannot_pass():
    x = torch.zeros(4, 8)
    with pytest.raises(trt.TrtError):          # not on a GPU
        trt.layernorm(x)
    with pytest.raises(trt.TrtError) as e:     # rows on top of each other
        trt.layernorm(x[:1].expand(4, 8))
    assert e.value.status == trt.ERR_STRIDE
    with pytest.raises(trt.TrtError) as e:     # columns apart
        trt.layernorm(torch.zeros(8, 4).t())
    assert e.value.status == trt.ERR_STRIDE
    with pytest.raises(trt.TrtError) as e:
        trt.layernorm(x, torch.ones(7))
    assert e.value.status == trt.ERR_SIZE
    with pytest.raises(trt.TrtError) as e:
        trt.layernorm(x, torch.ones(8), torch.ones(8, dtype=torch.float16))
    assert e.value.status == trt.ERR_DTYPE
    with pytest.raises(trt.TrtError) as e:
        trt.layernorm(torch.zeros(4, 8, dtype=torch.float64))
    assert e.value.status == trt.ERR_DTYPE
    with pytest.raises(trt.TrtError) as e:
        trt.layernorm_bwd(torch.zeros(4, 7), x)
    assert e.value.status == trt.ERR_SIZE


def test_oracle_gradients_against_differences():
    rng = np.random.default_rng(0)
    x, dy = rng.normal(size=(3, 11)), rng.normal(size=(3, 11))
    g, b = rng.normal(size=11), rng.normal(size=11)
    dx, dg, db = norm_ref.backward(dy, x, g, 1e-3)
    step = 1e-6

    def L(x, g, b):
        return (dy * norm_ref.forward(x, g, b, 1e-3)).sum()

    for i in range(3):
        for j in range(11):
            e = np.zeros_like(x)
            e[i, j] = step
            assert abs((L(x + e, g, b) - L(x - e, g, b)) / (2 * step) - dx[i, j]) < 1e-7
    for j in range(11):
        e = np.zeros(11)
        e[j] = step
        assert abs((L(x, g + e, b) - L(x, g - e, b)) / (2 * step) - dg[j]) < 1e-7
        assert abs((L(x, g, b + e) - L(x, g, b - e)) / (2 * step) - db[j]) < 1e-7
