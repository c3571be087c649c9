"""GPU parity of the layer norm and its gradients against the 64-bit oracle.

Tolerances count roundings.  u = 2^-24 is binary32's half step.  A sum over a
row runs through at most 32 elements of a lane, 6 steps across the wave and 16
waves: 54 additions, so its error is at most 54 u times the sum of the
magnitudes; the few roundings of the surrounding arithmetic make that 64.
With sigma the row's spread, mean |x - mu| <= sigma, so the corrected mean is
off by at most 64 u sigma and the variance by 2 * 64 u of itself, i.e.
1/sqrt(v + eps) by at most 64 u (relative).  Hence

    |error of h|  <= u (64 + 72 |h|)
    |error of y|  <= half step of y's type + u (|gamma| (64 + 72 |h|) + 4 |y| + 4 |beta|)

and with w = dy gamma, U = rms(w) >= mean |w|, mean |w h|:

    |error of dx| <= half step + u r (200 U + 80 |w| + 260 U |h|)

A parameter gradient adds rows / slices rows in a workgroup's running sums, 16
groups, slices / 16 slices in a wave and 16 waves: with `depth` their sum,

    |error of dgamma| <= half step + u (depth sum |dy h| + sum |dy| (64 + 72 |h|))
    |error of dbeta|  <= half step + u depth sum |dy|
"""
import numpy as np
import pytest
import torch

import thread_register_tile_amd as trt
from oracle import norm_ref

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
DTYPES = [torch.float16, torch.bfloat16, torch.float32]
NAMES = {torch.float16: "f16", torch.bfloat16: "bf16", torch.float32: "f32"}
CODE = {torch.float16: trt.F16, torch.bfloat16: trt.BF16, torch.float32: trt.F32}


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    trt.lib()


def f64(t):
    return t.detach().cpu().to(torch.float64).numpy()


def half_step(ref, dtype):
    """Half a step of dtype at ref (the smallest one in the subnormal range)."""
    fi = torch.finfo(dtype)
    return np.maximum(np.abs(ref), fi.tiny) * (fi.eps / 2)


def check(got, ref, tol, what):
    got = f64(got)
    assert got.shape == ref.shape, what
    bad = ~(np.abs(got - ref) <= tol)
    assert not bad.any(), (what, int(bad.sum()), float(np.nanmax(np.abs(got - ref) / tol)))


def padded(rows, cols, ld, dtype, offset, gen, scale=1.0, mean=0.0):
    """A [rows, cols] view with row stride ld, `offset` elements into a buffer
    of NaN, so that a read outside the view shows."""
    buf = torch.full((offset + rows * ld + 64,), float("nan"), dtype=dtype)
    view = buf[offset:offset + rows * ld].view(rows, ld)[:, :cols]
    view.copy_(torch.randn(rows, cols, generator=gen, dtype=torch.float64) * scale + mean)
    dev = buf.cuda()
    return dev[offset:offset + rows * ld].view(rows, ld)[:, :cols]


def guarded(rows, cols, ld, dtype, offset):
    buf = torch.full((offset + rows * ld + 64,), 77.0, dtype=dtype, device="cuda")
    return buf, buf[offset:offset + rows * ld].view(rows, ld)[:, :cols]


def untouched(buf, rows, cols, ld, offset):
    b = f64(buf)
    body = b[offset:offset + rows * ld].reshape(rows, ld)
    return (b[:offset] == 77).all() and (b[offset + rows * ld:] == 77).all() and (body[:, cols:] == 77).all()


def tol_forward(x, gamma, beta, eps, dtype):
    h, _ = norm_ref.stats(x, eps)
    y = norm_ref.forward(x, gamma, beta, eps)
    g = 1.0 if gamma is None else np.abs(gamma)
    b = 0.0 if beta is None else np.abs(beta)
    return y, half_step(y, dtype) + U * (g * (64 + 72 * np.abs(h)) + 4 * np.abs(y) + 4 * b)


def run_case(rows, cols, dtype, pdtype, *, pad=0, offset=0, eps=1e-5, seed=0, mean=0.0, scale=1.0,
             gamma=True, beta=True):
    gen = torch.Generator().manual_seed(seed)
    ld = cols + pad
    x = padded(rows, cols, ld, dtype, offset, gen, scale, mean)
    dy = padded(rows, cols, ld, dtype, offset, gen)
    g = (1 + 0.3 * torch.randn(cols, generator=gen)).to(pdtype).cuda() if gamma else None
    b = torch.randn(cols, generator=gen).to(pdtype).cuda() if beta else None
    hx, hdy = f64(x), f64(dy)
    hg, hb = (None if t is None else f64(t) for t in (g, b))
    what = f"{rows}x{cols} {NAMES[dtype]}/{NAMES[pdtype]} pad {pad} offset {offset}"

    ybuf, y = guarded(rows, cols, ld, dtype, offset)
    trt.layernorm(x, g, b, eps=eps, out=y)
    ref, tol = tol_forward(hx, hg, hb, eps, dtype)
    check(y, ref, tol, what)
    assert untouched(ybuf, rows, cols, ld, offset), what

    dxbuf, dx = guarded(rows, cols, ld, dtype, offset)
    need = trt.layernorm_bwd_workspace_size(rows, cols, CODE[dtype])
    ws = torch.full((need + 64,), 0xAB, dtype=torch.uint8, device="cuda")
    dgamma, dbeta = (torch.empty(cols, dtype=pdtype, device="cuda") for _ in range(2))
    trt.layernorm_bwd(dy, x, g, eps=eps, dx=dx, dgamma=dgamma, dbeta=dbeta, workspace=ws[:need])
    assert (ws[need:] == 0xAB).all(), what
    rdx, rdg, rdb = norm_ref.backward(hdy, hx, hg, eps)
    h, r = norm_ref.stats(hx, eps)
    w = np.abs(hdy * (1.0 if hg is None else hg))
    rms = np.sqrt((w * w).mean(1, keepdims=True))
    check(dx, rdx, half_step(rdx, dtype) + U * r * (200 * rms + 80 * w + 260 * rms * np.abs(h)), what + " dx")
    slices = need // (8 * cols)
    depth = -(-rows // slices) + 16 + -(-slices // 16) + 16
    check(dgamma, rdg, half_step(rdg, pdtype) + U * (depth * np.abs(hdy * h).sum(0) +
                                                     (np.abs(hdy) * (64 + 72 * np.abs(h))).sum(0)), what + " dgamma")
    check(dbeta, rdb, half_step(rdb, pdtype) + U * depth * np.abs(hdy).sum(0), what + " dbeta")
    assert untouched(dxbuf, rows, cols, ld, offset), what


# widths on both sides of every change of the waves or chunks per row, for
# 8-element and 4-element chunks, and odd ones
WIDTHS = [1, 2, 3, 7, 8, 9, 63, 64, 65, 255, 256, 257, 511, 512, 513, 1023, 1024, 1025, 2047, 2048,
          2056, 4095, 4096, 4104, 8192, 8199]


@pytest.mark.parametrize("dtype", DTYPES, ids=NAMES.get)
@pytest.mark.parametrize("cols", WIDTHS)
def test_widths(cols, dtype):
    run_case(5, cols, dtype, torch.float32, seed=cols)


@pytest.mark.parametrize("dtype,cols", [(torch.float16, 16384), (torch.bfloat16, 16391), (torch.float16, 32768),
                                        (torch.bfloat16, 32767), (torch.float32, 16384), (torch.float32, 16381)],
                         ids=lambda v: NAMES.get(v, v))
def test_longest_rows(cols, dtype):
    run_case(3, cols, dtype, dtype, seed=cols)


@pytest.mark.parametrize("dtype,cols", [(torch.bfloat16, 16379), (torch.float16, 20490), (torch.bfloat16, 24577),
                                        (torch.float32, 8201), (torch.float32, 12289)],
                         ids=lambda v: NAMES.get(v, v))
def test_long_rows_in_turns(cols, dtype):
    # each workgroup takes several rows, the last ones fewer
    run_case(515, cols, dtype, torch.float32, seed=cols)


@pytest.mark.parametrize("dtype,cols", [(torch.bfloat16, 1530), (torch.float16, 2047), (torch.bfloat16, 4090),
                                        (torch.float16, 8184), (torch.float32, 765), (torch.float32, 1022)],
                         ids=lambda v: NAMES.get(v, v))
def test_large_workgroups_in_turns(cols, dtype):
    run_case(4111, cols, dtype, torch.float32, seed=cols)


@pytest.mark.parametrize("dtype", DTYPES, ids=NAMES.get)
@pytest.mark.parametrize("rows", [1, 2, 3, 4, 31, 257, 4099])
def test_row_counts(rows, dtype):
    # more rows than workgroups, and counts that leave the last turn short
    run_case(rows, 264, dtype, dtype, seed=rows)


@pytest.mark.parametrize("dtype", DTYPES, ids=NAMES.get)
@pytest.mark.parametrize("cols,pad,offset", [(512, 1, 0), (512, 8, 1), (1000, 24, 3), (1023, 0, 1), (2050, 5, 7)])
def test_strides_and_alignment(cols, pad, offset, dtype):
    run_case(37, cols, dtype, torch.float32, pad=pad, offset=offset, seed=offset)


@pytest.mark.parametrize("gamma,beta", [(False, False), (True, False), (False, True)])
def test_absent_parameters(gamma, beta):
    run_case(19, 300, torch.bfloat16, torch.float32, gamma=gamma, beta=beta)


@pytest.mark.parametrize("dtype", DTYPES, ids=NAMES.get)
def test_mean_large_against_the_spread(dtype):
    # |mean| is 200 spreads (binary32: 20000); the second round corrects the mean
    mean = 20000.0 if dtype == torch.float32 else 200.0
    run_case(9, 1500, dtype, torch.float32, mean=mean, seed=3)


@pytest.mark.parametrize("scale", [1e-3, 1e3])
def test_scales(scale):
    run_case(9, 777, torch.float32, torch.float32, scale=scale, eps=1e-12, seed=4)


def test_one_element_rows_and_constant_rows():
    # v = 0: h = 0 for any eps > 0, so y = beta and dx = 0 exactly
    x = torch.full((6, 640), 3.1415, dtype=torch.float32, device="cuda")
    b = torch.randn(640, device="cuda")
    y = trt.layernorm(x, torch.randn(640, device="cuda"), b)
    assert torch.equal(y, b.expand(6, 640))
    one = torch.randn(50, 1, device="cuda")
    assert (trt.layernorm(one) == 0).all()
    dx, dg, db = trt.layernorm_bwd(one, one)
    assert (dx == 0).all() and (dg == 0).all()


def test_nonfinite_rows_stay_alone():
    x = torch.randn(8, 1000, device="cuda")
    dy = torch.randn(8, 1000, device="cuda")
    clean, (dclean, _, _) = trt.layernorm(x), trt.layernorm_bwd(dy, x)
    bad = x.clone()
    bad[2, 5], bad[6, 999] = float("nan"), float("inf")
    y, (dx, dg, _) = trt.layernorm(bad), trt.layernorm_bwd(dy, bad)
    rows = [0, 1, 3, 4, 5, 7]
    assert torch.equal(y[rows], clean[rows]) and torch.equal(dx[rows], dclean[rows])
    assert y[[2, 6]].isnan().all() and dx[[2, 6]].isnan().all() and dg.isnan().all()


def test_one_gradient_of_two_and_none():
    x, dy = (torch.randn(700, 520, device="cuda") for _ in range(2))
    g = torch.randn(520, device="cuda")
    dx, dg, db = trt.layernorm_bwd(dy, x, g)
    only, none_g, none_b = trt.layernorm_bwd(dy, x, g, params=False)
    assert torch.equal(only, dx) and none_g is None and none_b is None
    need = trt.layernorm_bwd_workspace_size(700, 520, trt.F32)
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")
    out = torch.full((520,), 9.0, device="cuda")
    s = torch.cuda.current_stream().cuda_stream
    for which, ref in ((0, dg), (1, db)):
        out.fill_(9)
        args = [out.data_ptr() if which == i else None for i in range(2)]
        assert trt.lib().trt_layernorm_bwd(700, 520, dy.data_ptr(), 520, x.data_ptr(), 520, g.data_ptr(), 1e-5,
                                           only.data_ptr(), 520, *args, trt.F32, trt.F32, ws.data_ptr(), need,
                                           s or None) == trt.OK
        assert torch.equal(out, ref)


def test_repeats_bit_for_bit():
    x, dy = (torch.randn(3001, 768, device="cuda").bfloat16() for _ in range(2))
    first = trt.layernorm_bwd(dy, x)
    for _ in range(3):
        assert all(torch.equal(a, b) for a, b in zip(trt.layernorm_bwd(dy, x), first))


def test_gradients_against_differences():
    """<dx, v> and <dgamma, v> against central differences of L = sum dy y.

    L is evaluated from binary32 outputs summed in 64 bits: each y is off by at
    most 64 + 72|h| + 8 <= 400 u, so L by 400 u sum |dy| at worst and, the
    errors being of either sign, far less; over 2 step = 2^-4 and n = 3 * 200
    elements that is 16 * 400 u * 600 = 0.23 at worst and sqrt(600) / 600 of
    it, 0.01, as a random sum.  The third derivative's part is step^2 / 6 =
    1.6e-4 of a sum of 600 terms of either sign: under 0.02.  Values are of
    the order of sqrt(600) = 24.
    """
    gen = torch.Generator().manual_seed(5)
    x, dy, v = (torch.randn(3, 200, generator=gen).cuda() for _ in range(3))
    g, b, vg = (torch.randn(200, generator=gen).cuda() for _ in range(3))
    step = 2.0 ** -5

    def L(x, g):
        return float((dy.double() * trt.layernorm(x, g, b).double()).sum())

    dx, dg, _ = trt.layernorm_bwd(dy, x, g)
    along_x = (L(x + step * v, g) - L(x - step * v, g)) / (2 * step)
    along_g = (L(x, g + step * vg) - L(x, g - step * vg)) / (2 * step)
    assert abs(along_x - float((dx.double() * v.double()).sum())) < 0.25
    assert abs(along_g - float((dg.double() * vg.double()).sum())) < 0.25


def test_batched_shapes_and_streams():
    x = torch.randn(4, 33, 384, device="cuda", dtype=torch.float16)
    want = trt.layernorm(x.reshape(-1, 384)).view(4, 33, 384)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = trt.layernorm(x)
        again = trt.layernorm_bwd(x, x)[0]
    side.synchronize()
    assert torch.equal(got, want)
    assert torch.equal(again, trt.layernorm_bwd(x, x)[0])


def test_capture_and_replay():
    x, dy = (torch.randn(300, 1000, device="cuda").half() for _ in range(2))
    g, b = (torch.randn(1000, device="cuda") for _ in range(2))
    y, dx = torch.empty_like(x), torch.empty_like(x)
    dg, db = torch.empty_like(g), torch.empty_like(g)
    ws = torch.empty(trt.layernorm_bwd_workspace_size(300, 1000, trt.F16), dtype=torch.uint8, device="cuda")

    def work():
        trt.layernorm(x, g, b, out=y)
        trt.layernorm_bwd(dy, x, g, dx=dx, dgamma=dg, dbeta=db, workspace=ws)

    work()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        work()
    for seed in range(4):
        gen = torch.Generator(device="cuda").manual_seed(seed)
        x.copy_(torch.randn(300, 1000, device="cuda", generator=gen))
        for t in (y, dx, dg, db):
            t.fill_(5)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, trt.layernorm(x, g, b))
        assert all(torch.equal(p, q) for p, q in zip((dx, dg, db), trt.layernorm_bwd(dy, x, g)))


@pytest.mark.parametrize("dtype", DTYPES, ids=NAMES.get)
def test_rows_far_apart(dtype):
    # rows 16 or 32 MB apart, offsets past 2^32 bytes: the same results as from
    # packed rows
    rows, cols, ld = 300, 520, 8_000_000
    gen = torch.Generator(device="cuda").manual_seed(7)
    x, dy = (torch.randn(rows, cols, generator=gen, device="cuda").to(dtype) for _ in range(2))
    gamma = torch.randn(cols, generator=gen, device="cuda")
    far_x, far_dy, out = (torch.empty(rows * ld, dtype=dtype, device="cuda").view(rows, ld)[:, :cols] for _ in range(3))
    far_x.copy_(x)
    far_dy.copy_(dy)
    assert torch.equal(trt.layernorm(far_x, gamma, out=out), trt.layernorm(x, gamma))
    got = trt.layernorm_bwd(far_dy, far_x, gamma, dx=out)
    for a, b in zip(got, trt.layernorm_bwd(dy, x, gamma)):
        assert torch.equal(a, b)
