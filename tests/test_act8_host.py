"""CPU tests of the 8-bit activations' entry points: refusals before any HIP
call, workspace sizes, and the oracle's format against its definition."""
import numpy as np
import pytest
import torch

import thread_register_tile_amd as trt
from oracle import act8_ref

BASE = 1 << 24     # fake, well-separated addresses: never dereferenced


def pack(**kw):
    a = dict(rows=8, cols=70, x=BASE, ldx=70, q=BASE * 2, ldq=70, scale=BASE * 3, lds=3, dtype=trt.F16)
    a.update(kw)
    return trt.lib().trt_act8_pack(a["rows"], a["cols"], a["x"], a["ldx"], a["q"], a["ldq"], a["scale"], a["lds"],
                                   a["dtype"], None)


def unpack(**kw):
    a = dict(rows=8, cols=70, x=BASE, ldx=70, q=BASE * 2, ldq=70, scale=BASE * 3, lds=3, dtype=trt.F16)
    a.update(kw)
    return trt.lib().trt_act8_unpack(a["rows"], a["cols"], a["q"], a["ldq"], a["scale"], a["lds"], a["x"], a["ldx"],
                                     a["dtype"], None)


def weight(**kw):
    a = dict(tokens=100, outputs=64, inputs=70, dy=BASE, lddy=64, q=BASE * 2, ldq=70, scale=BASE * 3, lds=3,
             dw=BASE * 4, lddw=70, dt=trt.BF16, odt=trt.F32, ws=BASE * 8, wsb=1 << 24)
    a.update(kw)
    return trt.lib().trt_act8_weight_grad(a["tokens"], a["outputs"], a["inputs"], a["dy"], a["lddy"], a["q"], a["ldq"],
                                          a["scale"], a["lds"], a["dw"], a["lddw"], a["dt"], a["odt"], a["ws"],
                                          a["wsb"], None)


COMMON = [
    (dict(rows=0), trt.ERR_SIZE), (dict(cols=0), trt.ERR_SIZE), (dict(rows=(1 << 30) + 1), trt.ERR_SIZE),
    (dict(rows=1 << 30, cols=1 << 12, ldx=1 << 12, ldq=1 << 12, lds=128), trt.ERR_SIZE),
    (dict(rows=1 << 30, ldx=1 << 60), trt.ERR_SIZE),
    (dict(x=0), trt.ERR_NULL), (dict(q=0), trt.ERR_NULL), (dict(scale=0), trt.ERR_NULL),
    (dict(x=BASE + 1), trt.ERR_ALIGN), (dict(dtype=trt.F32, x=BASE + 2), trt.ERR_ALIGN),
    (dict(dtype=0), trt.ERR_DTYPE), (dict(dtype=9), trt.ERR_DTYPE),
]


@pytest.mark.parametrize("kw,code", COMMON + [
    (dict(ldx=0), trt.ERR_STRIDE), (dict(ldq=69), trt.ERR_STRIDE), (dict(lds=2), trt.ERR_STRIDE),
    (dict(q=BASE + 100), trt.ERR_OVERLAP), (dict(scale=BASE + 2 * 8 * 70 - 1), trt.ERR_OVERLAP),
    (dict(scale=BASE * 2 + 5), trt.ERR_OVERLAP),
])
def test_pack_refusals(kw, code):
    assert pack(**kw) == code
    assert trt.last_error() != ""


@pytest.mark.parametrize("kw,code", COMMON + [
    (dict(ldx=69), trt.ERR_STRIDE), (dict(ldq=0), trt.ERR_STRIDE), (dict(lds=0), trt.ERR_STRIDE),
    (dict(x=BASE * 2), trt.ERR_OVERLAP), (dict(x=BASE * 3 - 2), trt.ERR_OVERLAP),
])
def test_unpack_refusals(kw, code):
    assert unpack(**kw) == code
    assert trt.last_error() != ""


@pytest.mark.parametrize("kw,code", [
    (dict(tokens=0), trt.ERR_SIZE), (dict(outputs=0), trt.ERR_SIZE), (dict(inputs=0), trt.ERR_SIZE),
    (dict(tokens=(1 << 23) + 1), trt.ERR_SIZE), (dict(outputs=(1 << 20) + 1, lddy=1 << 21), trt.ERR_SIZE),
    (dict(inputs=(1 << 20) + 1, ldq=1 << 21, lds=1 << 16, lddw=1 << 21), trt.ERR_SIZE),
    (dict(tokens=1, outputs=1 << 20, inputs=1 << 20, lddy=1 << 20, ldq=1 << 20, lds=1 << 15, lddw=1 << 20), trt.ERR_SIZE),
    (dict(tokens=1 << 23, outputs=1 << 20, lddy=1 << 20), trt.ERR_SIZE),
    (dict(tokens=1 << 23, outputs=1 << 18, inputs=1 << 18, lddy=1 << 18, ldq=1 << 18, lds=1 << 13, lddw=1 << 18), trt.ERR_SIZE),
    (dict(lddy=0), trt.ERR_STRIDE), (dict(ldq=0), trt.ERR_STRIDE), (dict(lds=0), trt.ERR_STRIDE), (dict(lddw=69), trt.ERR_STRIDE),
    (dict(dy=0), trt.ERR_NULL), (dict(q=0), trt.ERR_NULL), (dict(scale=0), trt.ERR_NULL), (dict(dw=0), trt.ERR_NULL),
    (dict(ws=0), trt.ERR_NULL), (dict(wsb=100), trt.ERR_SIZE), (dict(wsb=-1), trt.ERR_SIZE), (dict(ws=BASE * 8 + 8), trt.ERR_ALIGN),
    (dict(dy=BASE + 1), trt.ERR_ALIGN), (dict(dw=BASE * 4 + 2), trt.ERR_ALIGN),
    (dict(dw=BASE), trt.ERR_OVERLAP), (dict(dw=BASE * 2), trt.ERR_OVERLAP), (dict(dw=BASE * 3), trt.ERR_OVERLAP),
    (dict(ws=BASE), trt.ERR_OVERLAP), (dict(ws=BASE * 4), trt.ERR_OVERLAP),
    (dict(dt=trt.F32), trt.ERR_DTYPE), (dict(odt=0), trt.ERR_DTYPE),
])
def test_weight_grad_refusals(kw, code):
    assert weight(**kw) == code
    assert trt.last_error() != ""


def test_workspace_size():
    size = trt.act8_weight_grad_workspace_size
    x = 16384 * 8192 * 2
    assert size(16384, 8192, 8192) == x                          # one slice, dy in place
    assert size(16384, 8192, 8192, 8) == 2 * x                   # dy off 16 bytes
    assert size(16384, 8192, 8192, 0, 8196) == 2 * x             # rows off 16 bytes
    assert size(16384, 8191, 8192, 0, 8192) == 2 * x             # a cut last chunk
    assert size(16384, 8192, 8192, 0, 64) == 2 * x               # rows on top of each other
    assert size(100, 64, 70) == -(-100 * 72 * 2 // 256) * 256
    assert size(16384, 256, 256) > 16384 * 256 * 2 + 2 * 256 * 256 * 4   # sliced
    # a dy of more than 2 GiB is cut
    assert size(1 << 18, 8192, 8192) >= (1 << 18) * 8192 * 2 + 3 * 8192 * 8192 * 4
    for bad in ((0, 4, 4), (4, 0, 4), (4, 4, 0), (4, 1 << 21, 4)):
        with pytest.raises(trt.TrtError):
            size(*bad)


def test_binding_refuses_what_it_cannot_pass():
    x = torch.zeros(4, 70)
    q, s = torch.zeros(4, 70, dtype=torch.int8), torch.zeros(4, 3, dtype=torch.uint8)
    dy = torch.zeros(4, 8, dtype=torch.bfloat16)

    def refused(code, call, *a, **kw):
        with pytest.raises(trt.TrtError) as e:
            call(*a, **kw)
        assert e.value.status == code

    refused(trt.ERR_ARG, trt.act8_pack, x)                                     # not on a GPU
    refused(trt.ERR_SIZE, trt.act8_pack, x, q=q[:3])
    refused(trt.ERR_SIZE, trt.act8_pack, x, scale=s[:, :2])
    refused(trt.ERR_DTYPE, trt.act8_pack, x, scale=s.to(torch.int8))
    refused(trt.ERR_STRIDE, trt.act8_pack, torch.zeros(70, 4).t())
    refused(trt.ERR_DTYPE, trt.act8_unpack, q.to(torch.uint8), s, torch.float16)
    refused(trt.ERR_SIZE, trt.act8_unpack, q, s, torch.float16, out=x)
    refused(trt.ERR_ARG, trt.act8_unpack, q, s, torch.float16)
    refused(trt.ERR_SIZE, trt.act8_unpack, q, s[:, :2], torch.float16)
    refused(trt.ERR_SIZE, trt.act8_weight_grad, dy[:3], q, s)
    refused(trt.ERR_SIZE, trt.act8_weight_grad, dy, q, s, dw=torch.zeros(8, 71))
    refused(trt.ERR_SIZE, trt.act8_weight_grad, dy, q, s, out_dtype=torch.float32, dw=torch.zeros(8, 70, dtype=torch.bfloat16))
    refused(trt.ERR_ARG, trt.act8_weight_grad, dy, q, s)


def test_oracle_format():
    rng = np.random.default_rng(0)
    x = rng.normal(size=(50, 70)) * np.exp2(rng.integers(-160, 120, size=(50, 3)))[:, np.arange(70) // 32]
    x[3, 40], x[4, 2], x[5, :32] = np.inf, np.nan, 0
    q, scale = act8_ref.pack(x)
    v = act8_ref.unpack(q, scale)
    for r in range(50):
        for b in range(3):
            part, back, X = x[r, 32 * b:32 * b + 32], v[r, 32 * b:32 * b + 32], int(scale[r, b])
            if not np.isfinite(part).all():
                assert X == 255 and np.isnan(back).all()
                continue
            step = 2.0 ** (X - 133)
            assert 7 <= X <= 254 and (np.abs(back - part) <= step / 2 + (np.abs(part) > 127 * step) * step / 2).all()
            top = np.abs(part).max()
            assert X == 7 or (64 <= top / step < 128 and np.abs(q[r, 32 * b:32 * b + 32]).max() >= 64)
    # halves go to the even neighbour, and what rounds up to 128 stays at 127
    edge = np.array([[64.0, 0.5, 1.5, 2.5, -0.5, -1.5, -2.5], [127.75, 127.5, 126.5, -127.6, 0, 0, 0]])
    q, scale = act8_ref.pack(edge)
    assert (scale == 133).all()
    assert q.tolist() == [[64, 0, 2, 2, 0, -2, -2], [127, 127, 126, -127, 0, 0, 0]]
