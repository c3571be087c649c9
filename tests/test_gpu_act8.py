"""GPU parity of activations saved in 8 bits against the 64-bit oracle.

Packing and unpacking are one rounding each of exact arithmetic: bit for bit.
The weight gradient's products of 16-bit values (8 or 11 bits by 7) are exact
in binary32; a sum of T of them, in any order, is off by at most T - 1 roundings
of partial sums no larger than the sum of the magnitudes:

    |error of dw| <= half step of its type + T 2^-24 sum |dy x|

and with small integers no sum rounds at all: bit for bit.
"""
import numpy as np
import pytest
import torch

import thread_register_tile_amd as trt
from oracle import act8_ref

pytestmark = pytest.mark.gpu

DTYPES = [torch.float16, torch.bfloat16, torch.float32]


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    trt.lib()


def f64(t):
    return t.detach().cpu().to(torch.float64).numpy()


def values(rows, cols, dtype, seed):
    """Rows whose blocks lie at scales over the whole range of dtype, with
    halves of a step, block maxima that round up, zeros and subnormals."""
    rng = np.random.default_rng(seed)
    low, high = {torch.float16: (-26, 15), torch.bfloat16: (-135, 126), torch.float32: (-150, 126)}[dtype]
    blocks = -(-cols // 32)
    e = rng.integers(low, high, size=(rows, blocks))[:, np.arange(cols) // 32]
    x = rng.normal(size=(rows, cols))
    pick = rng.random((rows, cols))
    x = np.where(pick < 0.1, rng.integers(-255, 256, size=(rows, cols)) / 128, x)     # ties
    x = np.where(pick > 0.97, 1.9999, x)
    x[rng.random((rows, cols)) < 0.05] = 0
    x = np.ldexp(x, e)
    x[rng.random(rows) < 0.1] = 0
    return torch.from_numpy(x).to(dtype)


def strided(t, ld, offset, fill):
    """t in rows ld apart, `offset` elements into a buffer of `fill`."""
    rows, cols = t.shape
    buf = torch.full((offset + rows * ld + 64,), fill, dtype=t.dtype, device="cuda")
    view = buf[offset:offset + rows * ld].view(rows, ld)[:, :cols]
    view.copy_(t.cuda())
    return buf, view


def untouched(buf, rows, cols, ld, offset, fill):
    b = buf.cpu()
    body = b[offset:offset + rows * ld].view(rows, ld)
    return bool((b[:offset] == fill).all() and (b[offset + rows * ld:] == fill).all() and (body[:, cols:] == fill).all())


SHAPES = [(1, 1), (1, 31), (3, 32), (5, 33), (2, 4096), (77, 1000), (1000, 77), (64, 1024), (130, 5000), (4096, 24), (3, 70001)]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("rows,cols", SHAPES)
@pytest.mark.parametrize("pad,offset", [(0, 0), (3, 1), (8, 8)])
def test_pack_and_unpack(rows, cols, dtype, pad, offset):
    x = values(rows, cols, dtype, rows + cols)
    blocks = -(-cols // 32)
    _, xd = strided(x, cols + pad, offset, float("nan"))
    qbuf, q = strided(torch.zeros(rows, cols, dtype=torch.int8), cols + pad, offset, 77)
    sbuf, s = strided(torch.zeros(rows, blocks, dtype=torch.uint8), blocks + pad, offset, 177)
    got = trt.act8_pack(xd, q=q, scale=s)
    assert got[0] is q and got[1] is s
    rq, rs = act8_ref.pack(f64(x))
    assert (s.cpu().numpy() == rs).all()
    assert (q.cpu().numpy() == rq).all()
    assert untouched(qbuf, rows, cols, cols + pad, offset, 77)
    assert untouched(sbuf, rows, blocks, blocks + pad, offset, 177)
    obuf, out = strided(torch.zeros(rows, cols, dtype=dtype), cols + pad, offset, 77)
    trt.act8_unpack(q, s, dtype, out=out)
    # exact, in the type they came from (some blocks reached infinity in it)
    assert np.array_equal(f64(out), act8_ref.unpack(rq, rs), equal_nan=True)
    assert untouched(obuf, rows, cols, cols + pad, offset, 77)


@pytest.mark.parametrize("dtype", DTYPES)
def test_not_finite(dtype):
    x = torch.ones(6, 100, dtype=dtype)
    x[0, 5], x[1, 40], x[2, 99], x[3, 64], x[3, 95] = float("inf"), float("nan"), -float("inf"), float("nan"), float("inf")
    q, s = trt.act8_pack(x.cuda())
    rq, rs = act8_ref.pack(f64(x))
    assert (s.cpu().numpy() == rs).all() and (q.cpu().numpy() == rq).all()
    back = f64(trt.act8_unpack(q, s, dtype))
    want = act8_ref.unpack(rq, rs)
    assert np.array_equal(back, want, equal_nan=True)
    assert np.isnan(back[0, :32]).all() and (back[0, 32:] == 1).all() and (back[4] == 1).all()


@pytest.mark.parametrize("dtype", DTYPES)
def test_unpack_of_any_bytes(dtype):
    """Every scale with every integer, rounded to the type from 64 bits."""
    q = torch.arange(-128, 128, dtype=torch.int8).repeat(256, 1)
    s = torch.arange(256, dtype=torch.int32).to(torch.uint8)[:, None].repeat(1, 8).contiguous()
    got = trt.act8_unpack(q.cuda(), s.cuda(), dtype).cpu()
    want = torch.from_numpy(act8_ref.unpack(q.numpy(), s.numpy())).to(dtype)
    # (binary32 holds every one but -128 * 2^121 = -2^128, which is infinite in all three types)
    assert torch.equal(got.isnan(), want.isnan()) and torch.equal(got.nan_to_num(7.0), want.nan_to_num(7.0))


def test_leading_dimensions():
    x = torch.randn(3, 5, 40, dtype=torch.bfloat16, device="cuda")
    q, s = trt.act8_pack(x)
    assert q.shape == (3, 5, 40) and s.shape == (3, 5, 2)
    assert torch.equal(trt.act8_unpack(q, s, x.dtype).view(15, 40),
                       trt.act8_unpack(*trt.act8_pack(x.view(15, 40)), x.dtype))
    q1, s1 = trt.act8_pack(x[0, 0])
    assert torch.equal(q1, q[0, 0]) and torch.equal(s1, s[0, 0])


def test_offsets_past_32_bits():
    rows, ld = 3, (1 << 31) + 64            # bytes of q: rows 2 GiB apart
    q = torch.empty(rows * ld, dtype=torch.int8, device="cuda").view(rows, ld)[:, :100]
    x = torch.randn(rows, 100, device="cuda")
    _, s = trt.act8_pack(x, q=q)
    q2, s2 = trt.act8_pack(x)
    assert torch.equal(q, q2) and torch.equal(s, s2)
    assert torch.equal(trt.act8_unpack(q, s, torch.float32), trt.act8_unpack(q2, s2, torch.float32))


# tokens, outputs, inputs: one slice and several, small and large tiles, cut tiles,
# tokens on both sides of a K step, no multiple of anything
PRODUCTS = [(1, 1, 1), (1, 64, 64), (77, 1024, 1024), (33, 100, 31), (64, 129, 257), (65, 8, 2049), (513, 40, 40),
            (1500, 264, 520), (3000, 7, 9), (4097, 129, 70), (900, 4104, 3080), (1025, 4099, 3079)]


def case(tokens, outputs, inputs, dtype, seed, small):
    rng = np.random.default_rng(seed)
    if small:
        dy = torch.from_numpy(rng.integers(-2, 3, size=(tokens, outputs)).astype(np.float64)).to(dtype)
        x = torch.from_numpy(rng.integers(-3, 4, size=(tokens, inputs)).astype(np.float64)).to(dtype)
    else:
        dy = torch.from_numpy(rng.normal(size=(tokens, outputs))).to(dtype)
        x = torch.from_numpy(rng.normal(size=(tokens, inputs)) * np.exp(rng.normal(size=(tokens, 1)))).to(dtype)
    return dy, x


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("tokens,outputs,inputs", PRODUCTS)
def test_weight_grad_exact(tokens, outputs, inputs, dtype):
    """Integers up to 6 times the tokens, below 2^24: the binary32 result is exact."""
    dy, x = case(tokens, outputs, inputs, dtype, tokens + outputs, True)
    q, s = trt.act8_pack(x.cuda())
    ld = inputs + 5
    buf, dw = strided(torch.zeros(outputs, inputs), ld, 3, 77.0)
    need = trt.act8_weight_grad_workspace_size(tokens, outputs, inputs)
    ws = torch.full((need + 64,), 0xFF, dtype=torch.uint8, device="cuda")
    trt.act8_weight_grad(dy.cuda(), q, s, dw=dw, workspace=ws[:need])
    want = act8_ref.weight_grad(f64(dy), q.cpu().numpy(), s.cpu().numpy())
    assert (f64(dw) == want).all()
    assert untouched(buf, outputs, inputs, ld, 3, 77.0) and (ws[need:] == 0xFF).all()


@pytest.mark.parametrize("odt", [None, torch.float16, torch.bfloat16, torch.float32])
@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("tokens,outputs,inputs", PRODUCTS)
def test_weight_grad(tokens, outputs, inputs, dtype, odt):
    dy, x = case(tokens, outputs, inputs, dtype, tokens * 3 + inputs, False)
    q, s = trt.act8_pack(x.cuda())
    got = trt.act8_weight_grad(dy.cuda(), q, s, out_dtype=odt)
    assert got.dtype == (odt or dtype) and got.shape == (outputs, inputs)
    hdy, hx = f64(dy), act8_ref.unpack(q.cpu().numpy(), s.cpu().numpy())
    want, mags = hdy.T @ hx, np.abs(hdy).T @ np.abs(hx)
    fi = torch.finfo(got.dtype)
    tol = np.maximum(np.abs(want), fi.tiny) * (fi.eps / 2) + tokens * 2.0 ** -24 * mags
    bad = ~(np.abs(f64(got) - want) <= tol)
    assert not bad.any(), (int(bad.sum()), float(np.max(np.abs(f64(got) - want) / tol)))


@pytest.mark.parametrize("pad,offset", [(0, 0), (8, 8), (8, 4), (3, 0), (-30, 0)])
def test_weight_grad_of_any_dy(pad, offset):
    """In place and copied: aligned rows, bases and rows off 16 bytes, rows on
    top of each other."""
    tokens, outputs, inputs = 300, 72, 88
    ld = outputs + pad
    base = torch.from_numpy(np.random.default_rng(5).integers(-2, 3, size=offset + tokens * ld + 64).astype(np.float32))
    dy = base.to(torch.bfloat16).cuda()[offset:].as_strided((tokens, outputs), (ld, 1))
    _, x = case(tokens, outputs, inputs, torch.bfloat16, 6, True)
    q, s = trt.act8_pack(x.cuda())
    got = trt.act8_weight_grad(dy, q, s, out_dtype=torch.float32)
    assert (f64(got) == act8_ref.weight_grad(f64(dy), q.cpu().numpy(), s.cpu().numpy())).all()


def test_weight_grad_not_finite():
    """A NaN in dy spoils its output's row, a block of NaN its 32 columns."""
    dy, x = case(200, 40, 100, torch.bfloat16, 7, True)
    dy[17, 3] = float("nan")
    x[50, 70] = float("inf")
    q, s = trt.act8_pack(x.cuda())
    got = f64(trt.act8_weight_grad(dy.cuda(), q, s, out_dtype=torch.float32))
    spoilt = np.zeros((40, 100), bool)
    spoilt[3], spoilt[:, 64:96] = True, True
    assert (np.isnan(got) == spoilt).all()
    dy[17, 3] = 0
    x[50, 64:96] = 0
    want = act8_ref.weight_grad(f64(dy), *act8_ref.pack(f64(x)))
    assert (got[~spoilt] == want[~spoilt]).all()


def test_graph_and_streams():
    """Captured and replayed with new inputs, on a stream of its own, while the
    current stream runs the same operators on other data."""
    dy, x = (t.cuda() for t in case(500, 136, 264, torch.bfloat16, 8, True))
    dy2, x2 = (t.cuda() for t in case(500, 136, 264, torch.bfloat16, 9, True))
    q, s = trt.act8_pack(x)
    ws = torch.empty(trt.act8_weight_grad_workspace_size(500, 136, 264), dtype=torch.uint8, device="cuda")
    dw, back = torch.empty(136, 264, device="cuda"), torch.empty_like(x)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for _ in range(2):
            trt.act8_pack(x, q=q, scale=s)
            trt.act8_unpack(q, s, x.dtype, out=back)
            trt.act8_weight_grad(dy, q, s, dw=dw, workspace=ws)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        trt.act8_pack(x, q=q, scale=s)
        trt.act8_unpack(q, s, x.dtype, out=back)
        trt.act8_weight_grad(dy, q, s, dw=dw, workspace=ws)
    for turn in range(4):
        a, b = (dy2, x2) if turn % 2 else (dy2 * 2, x2 + 1)
        dy.copy_(a)
        x.copy_(b)
        torch.cuda.synchronize()
        dw.fill_(float("nan"))
        graph.replay()
        eager = trt.act8_weight_grad(a, *trt.act8_pack(b), out_dtype=torch.float32)
        torch.cuda.synchronize()
        assert torch.equal(back, b) and torch.equal(dw, eager)
        assert (f64(dw) == f64(a).T @ f64(b)).all()


@pytest.mark.parametrize("odt", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("tokens,outputs,inputs", [(8200, 2999, 1501), (8192, 3000, 1500), (6000, 1000, 1000), (16384, 512, 520),
                                                   (2048, 2048, 2048), (1700, 3000, 3000)])
def test_weight_grad_of_slices_and_tiles(tokens, outputs, inputs, odt):
    """Either size of tile, in one slice and in several: integers whose every
    partial sum is below 2^24, so that torch's binary32 product is exact too."""
    gen = torch.Generator(device="cuda").manual_seed(tokens)
    dy = torch.randint(-2, 3, (tokens, outputs), device="cuda", generator=gen).to(torch.bfloat16)
    x = torch.randint(-3, 4, (tokens, inputs), device="cuda", generator=gen).to(torch.bfloat16)
    need = trt.act8_weight_grad_workspace_size(tokens, outputs, inputs, dy.data_ptr())
    ws = torch.full((need + 64,), 0xFF, dtype=torch.uint8, device="cuda")
    got = trt.act8_weight_grad(dy, *trt.act8_pack(x), out_dtype=odt, workspace=ws[:need])
    assert torch.equal(got, torch.mm(dy.float().t().contiguous(), x.float()).to(odt))
    assert (ws[need:] == 0xFF).all()


@pytest.mark.parametrize("tokens,outputs,inputs", [(2_097_252, 72, 1100), (2_097_252, 1101, 40), (66_000, 128, 16400), (140_000, 8200, 300)])
def test_weight_grad_of_operands_past_2_gib(tokens, outputs, inputs):
    """x or dy of 2 to 4.6 GB, taken in slices: exact as above."""
    gen = torch.Generator(device="cuda").manual_seed(1)
    dy = torch.randint(-1, 2, (tokens, outputs), device="cuda", generator=gen).to(torch.bfloat16)
    x = torch.randint(-3, 4, (tokens, inputs), device="cuda", generator=gen).to(torch.bfloat16)
    got = trt.act8_weight_grad(dy, *trt.act8_pack(x), out_dtype=torch.float32)
    want = torch.zeros(outputs, inputs, device="cuda")
    for at in range(0, tokens, 30_000):
        want += torch.mm(dy[at:at + 30_000].float().t().contiguous(), x[at:at + 30_000].float())
    assert torch.equal(got, want)
