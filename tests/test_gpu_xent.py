"""GPU parity of the linear cross entropy and its gradients against the 64-bit
oracle.

Tolerances count roundings.  u = 2^-24 is binary32's half step, h the half
step of the inputs' type, d the width.  A logit is a binary32 sum of d exact
products, in whatever order: off by at most (d + 2) u S, S = sum |x w|; dz is
the largest of these in a row, Z the largest |z|.

An exponential's argument is one fused product (u 1.45 |z|, and as much for the
subtracted maximum or lse), the instruction and its factor add 4 u: a relative
error of e = dz + u (4 Z + 4 |lse| + 8) at most.  A row's sum runs through at
most 32 columns of a lane, 2 exchanges, 4 waves, the tiles of a thread and 8
steps across threads, each pair scaled by two such exponentials:

    |error of lse|  <= e + u (64 + 3 tiles + 2 |lse|)

A loss is log(1 + R), R the sum over the other entries against the target's: R
is off by that relative error and e of its own, and log(1 + R) by no more than
R / (1 + R) <= 1 - exp(-loss) of it:

    |error of loss| <= (1 - exp(-loss)) (2 e + dz + u (80 + 3 tiles)) + 4 u |loss|
                       + V 2^-126    (terms below binary32's smallest normal number)

With c the largest weight max(|dloss|, |dloss + dlse|), g / c is rounded once to
the inputs' type; for at most 64 tokens what that leaves is kept in a second
number, so that the error is h^2 of it:

    |error of g|  <= h |g| + e p s + h_0 c      (s the token's weight; h_0: half
                     the smallest step of the type, over G's scale)
    |error of dX| <= half step + sum |error of g| |W| + u (2 V + 4) sum |g| |W|
    |error of dW| <= half step + sum |error of g| |X| + u (2 T + 4) sum |g| |X|
"""
import numpy as np
import pytest
import torch

import thread_register_tile_amd as trt
from oracle import xent_ref

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
IGNORE = -100
F16, BF16 = torch.float16, torch.bfloat16
NAMES = {F16: "f16", BF16: "bf16", torch.float32: "f32"}


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    trt.lib()


def f64(t):
    return t.detach().cpu().to(torch.float64).numpy()


def half_step(ref, dtype):
    fi = torch.finfo(dtype)
    return np.maximum(np.abs(ref), fi.tiny) * (fi.eps / 2)


def check(got, ref, tol, what):
    got = f64(got)
    assert got.shape == ref.shape, what
    bad = ~(np.abs(got - ref) <= tol)
    assert not bad.any(), (what, int(bad.sum()), float(np.nanmax(np.abs(got - ref) / tol)))


def matrix(values, dtype, pad=0, offset=0):
    """values on the GPU as a view with row stride cols + pad, `offset`
    elements into a buffer of NaN."""
    rows, cols = values.shape
    ld = cols + pad
    buf = torch.full((offset + rows * ld + 64,), float("nan"), dtype=dtype, device="cuda")
    view = buf[offset:offset + rows * ld].view(rows, ld)[:, :cols]
    view.copy_(values)
    return view


def guarded(rows, cols, dtype, pad=0, offset=0):
    ld = cols + pad
    buf = torch.full((offset + rows * ld + 64,), 77.0, dtype=dtype, device="cuda")
    return buf, buf[offset:offset + rows * ld].view(rows, ld)[:, :cols]


def untouched(buf, rows, cols, pad, offset):
    ld = cols + pad
    inside = torch.zeros(buf.numel(), dtype=torch.bool, device="cuda")
    inside[offset:offset + rows * ld].view(rows, ld)[:, :cols] = True
    return bool((buf[~inside] == 77).all())


def dirty(nbytes):
    """A workspace of NaN patterns, with a guard behind it."""
    return torch.full((nbytes + 256,), 0xFF, dtype=torch.uint8, device="cuda")


class Case:
    def __init__(self, T, V, D, dtype, *, seed=0, ignored=0.0, sharp=2.0, pad=0, offset=0, weights="mean", dlse=False,
                 nan_ignored=True):
        gen = torch.Generator().manual_seed(seed)
        self.T, self.V, self.D, self.dtype = T, V, D, dtype
        w = torch.randn(V, D, generator=gen) * (sharp / D ** 0.5)
        target = torch.randint(0, V, (T,), generator=gen)
        x = torch.randn(T, D, generator=gen) + w[target] * torch.rand(T, 1, generator=gen) * 4
        drop = torch.rand(T, generator=gen) < ignored
        self.x, self.w = matrix(x.cuda(), dtype, pad, offset), matrix(w.cuda(), dtype, pad, offset)
        self.hx, self.hw = f64(self.x), f64(self.w)
        if nan_ignored:
            self.x[drop.cuda()] = float("nan")      # what an ignored row holds reaches nothing
        self.target = torch.where(drop, IGNORE, target).cuda()
        self.ht = self.target.cpu().numpy()
        count = max(1, int((~drop).sum()))
        up = torch.full((T,), 1.0 / count)
        if weights == "each":
            up = up * (torch.rand(T, generator=gen) - 0.4)
        if weights == "masked":                      # zero weight: as good as ignored
            off = torch.rand(T, generator=gen) < 0.4
            up = torch.where(off, 0.0, up)
            if nan_ignored:
                self.x[off.cuda()] = float("nan")
        self.dloss = up.float().cuda()
        self.dlse = (0.3 * torch.randn(T, generator=gen) / count).float().cuda() if dlse else None
        self.what = f"{T}x{V}x{D} {NAMES[dtype]} pad {pad} offset {offset} ignored {ignored} {weights}"

    def bounds(self):
        z, live = xent_ref.logits(self.hx, self.hw, self.ht, IGNORE)
        S = (np.abs(self.hx[live]) @ np.abs(self.hw).T).max(1) if len(z) else np.zeros(0)
        dz = (self.D + 2) * U * S
        Z = np.abs(z).max(1) if len(z) else np.zeros(0)
        _, lse = xent_ref.forward(self.hx, self.hw, self.ht, IGNORE)
        e = dz + U * (4 * Z + 4 * np.abs(lse[live]) + 8)
        return live, dz, e, lse

    def forward(self):
        need = trt.linear_xent_workspace_size(self.T, self.V, self.D)
        ws = dirty(need)
        loss, lse = (torch.full((self.T,), 9.0, device="cuda") for _ in range(2))
        trt.linear_xent(self.x, self.w, self.target, loss=loss, lse=lse, workspace=ws[:need])
        assert (ws[need:] == 0xFF).all(), self.what
        return loss, lse

    def check_forward(self):
        loss, lse = self.forward()
        rloss, rlse = xent_ref.forward(self.hx, self.hw, self.ht, IGNORE)
        live, dz, e, _ = self.bounds()
        tiles = -(-self.V // 128)
        tol = np.zeros(self.T)
        tol[live] = e + U * (64 + 3 * tiles + 2 * np.abs(rlse[live]))
        check(lse, rlse, tol, self.what + " lse")
        l = rloss[live]
        tol[live] = -np.expm1(-l) * (2 * e + dz + U * (80 + 3 * tiles)) + 4 * U * np.abs(l) + self.V * 2.0 ** -126
        check(loss, rloss, tol, self.what + " loss")

    def backward(self, piece=0, out_dtype=None, pad=0, offset=0, need_dx=True, need_dw=True):
        odt = out_dtype or self.dtype
        _, lse = xent_ref.forward(self.hx, self.hw, self.ht, IGNORE)
        need = trt.linear_xent_bwd_workspace_size(self.T, self.V, self.D, piece)
        ws = dirty(need)
        xbuf, dx = guarded(self.T, self.D, odt, pad, offset)
        wbuf, dw = guarded(self.V, self.D, odt, pad, offset)
        got = trt.linear_xent_bwd(self.x, self.w, self.target, torch.from_numpy(lse).float().cuda(), self.dloss,
                                  self.dlse, need_dx=need_dx, need_dw=need_dw, piece=piece, out_dtype=odt,
                                  dx=dx if need_dx else None, dw=dw if need_dw else None, workspace=ws[:need])
        assert (ws[need:] == 0xFF).all(), self.what
        assert untouched(xbuf, self.T, self.D, pad, offset) and untouched(wbuf, self.V, self.D, pad, offset), self.what
        return got

    def check_backward(self, **kw):
        odt = kw.get("out_dtype") or self.dtype
        dx, dw = self.backward(**kw)
        hl, he = f64(self.dloss), None if self.dlse is None else f64(self.dlse)
        g, p, live = xent_ref.dlogits(self.hx, self.hw, self.ht, hl, he, IGNORE)
        rdx, rdw = xent_ref.backward(self.hx, self.hw, self.ht, hl, he, IGNORE)
        _, _, e, _ = self.bounds()
        both = hl if he is None else hl + he
        s = np.maximum(np.abs(hl), np.abs(both))[live][:, None]
        h = torch.finfo(self.dtype).eps / 2
        if self.T <= 64:
            h = h * h
        least = 2.0 ** -39 if self.dtype == F16 else 2.0 ** -134
        dg = h * np.abs(g) + e[:, None] * p * s + least * (s.max() if s.size else 0.0)
        ax, aw, ag = np.abs(self.hx[live]), np.abs(self.hw), np.abs(g)
        tol = np.zeros_like(rdx)
        tol[live] = dg @ aw + U * (2 * self.V + 4) * (ag @ aw)
        check(dx, rdx, half_step(rdx, odt) + tol, self.what + " dx")
        tol = dg.T @ ax + U * (2 * self.T + 4) * (ag.T @ ax)
        check(dw, rdw, half_step(rdw, odt) + tol, self.what + " dw")


# tokens, vocabulary and width on both sides of the tiles' edges; widths that
# the copies take (multiples of 8) and that they do not
SIZES = [(1, 1, 8), (1, 2, 1), (2, 63, 16), (3, 64, 7), (16, 65, 32), (17, 127, 40), (127, 128, 64), (128, 129, 72),
         (129, 255, 33), (130, 257, 136), (255, 300, 100), (257, 1000, 512), (64, 5000, 256), (300, 130, 1024),
         (1, 4099, 264), (5, 100, 2056)]


@pytest.mark.parametrize("dtype", [F16, BF16], ids=NAMES.get)
@pytest.mark.parametrize("T,V,D", SIZES)
def test_sizes(T, V, D, dtype):
    c = Case(T, V, D, dtype, seed=T + V, ignored=0.25 if T > 2 else 0.0)
    c.check_forward()
    c.check_backward()


@pytest.mark.parametrize("dtype", [F16, BF16], ids=NAMES.get)
@pytest.mark.parametrize("T,V,D", [(1030, 12500, 64), (700, 16391, 776), (300, 12800, 1000), (2100, 6100, 257)])
def test_wide_tiles(T, V, D, dtype):
    # 256-wide tiles in one product or another
    c = Case(T, V, D, dtype, seed=D, ignored=0.1)
    c.check_forward()
    c.check_backward()


@pytest.mark.parametrize("piece", [64, 128, 256, 320, 1024, 4096])
def test_pieces(piece):
    for T, V, D, dtype in ((150, 1000, 64, F16), (40, 645, 24, BF16), (33, 500, 19, BF16), (260, 1100, 264, F16)):
        Case(T, V, D, dtype, seed=piece, ignored=0.2).check_backward(piece=piece)


@pytest.mark.parametrize("dtype", [F16, BF16], ids=NAMES.get)
@pytest.mark.parametrize("pad,offset", [(8, 0), (0, 8), (1, 0), (24, 3), (4, 4)])
def test_strides_and_alignment(pad, offset, dtype):
    c = Case(140, 333, 64, dtype, pad=pad, offset=offset, seed=pad, ignored=0.3)
    c.check_forward()
    c.check_backward(pad=pad, offset=offset)


@pytest.mark.parametrize("out_dtype", [F16, BF16, torch.float32], ids=NAMES.get)
@pytest.mark.parametrize("dtype", [F16, BF16], ids=NAMES.get)
def test_output_types(dtype, out_dtype):
    c = Case(200, 700, 96, dtype, seed=6)
    c.check_backward(out_dtype=out_dtype)
    c.check_backward(out_dtype=out_dtype, pad=5, offset=2)


@pytest.mark.parametrize("dtype", [F16, BF16], ids=NAMES.get)
@pytest.mark.parametrize("weights,dlse", [("each", False), ("mean", True), ("each", True), ("masked", False)])
def test_weights(weights, dlse, dtype):
    for T, V, D in ((150, 500, 64), (20, 300, 31), (300, 900, 128)):
        Case(T, V, D, dtype, weights=weights, dlse=dlse, seed=7, ignored=0.2, nan_ignored=not dlse).check_backward()


@pytest.mark.parametrize("T", [1, 100, 200, 9000])
def test_every_token_ignored(T):
    c = Case(T, 300, 64, BF16, ignored=2.0)
    loss, lse = c.forward()
    assert (loss == 0).all() and (lse == 0).all()
    dx, dw = c.backward()
    assert (dx == 0).all() and (dw == 0).all()


@pytest.mark.parametrize("ignored", [0.0, 0.5, 0.97])
def test_many_tokens(ignored):
    # more tokens than one turn of the list takes
    c = Case(9001, 200, 16, F16, ignored=ignored, seed=9)
    c.check_forward()
    c.check_backward()


@pytest.mark.parametrize("sharp", [0.01, 12.0])
def test_flat_and_sharp_logits(sharp):
    # near uniform, and logits of hundreds with probabilities near one
    for dtype in (F16, BF16):
        c = Case(140, 400, 64, dtype, sharp=sharp, seed=11)
        c.check_forward()
        c.check_backward()


def test_one_of_the_gradients():
    c = Case(150, 500, 64, BF16, seed=12, ignored=0.2)
    dx, dw = c.backward()
    only, none = c.backward(need_dw=False)
    assert torch.equal(only, dx) and none is None
    none, only = c.backward(need_dx=False)
    assert torch.equal(only, dw) and none is None


def test_target_outside_the_vocabulary():
    for T in (9, 200):
        c = Case(T, 300, 64, BF16, seed=13)
        clean, clean_lse = c.forward()
        cdx, _ = c.backward()
        for bad in (300, -1, 2 ** 40, -2 ** 40):
            c.target[5] = bad
            loss, lse = c.forward()
            rest = torch.arange(T, device="cuda") != 5
            assert loss[5].isnan() and torch.equal(loss[rest], clean[rest]) and torch.equal(lse, clean_lse)
            lse_in = lse.clone()
            dx, dw = trt.linear_xent_bwd(c.x, c.w, c.target, lse_in, c.dloss)
            assert dx[5].isnan().all() and dw.isnan().all() and not dx[rest].isnan().any()


def test_ignore_index_may_be_a_vocabulary_entry():
    c = Case(60, 100, 32, BF16, seed=14)
    c.target[::3] = 7
    loss, lse = trt.linear_xent(c.x, c.w, c.target, ignore_index=7)
    assert (loss[::3] == 0).all() and (lse[::3] == 0).all()
    dx, dw = trt.linear_xent_bwd(c.x, c.w, c.target, lse, c.dloss, ignore_index=7)
    assert (dx[::3] == 0).all()


def test_nonfinite_logits_stay_alone():
    for T in (40, 300):
        c = Case(T, 500, 64, BF16, seed=15)
        clean, _ = c.forward()
        c.x[3, 5], c.x[T - 1, 0] = float("nan"), float("inf")
        loss, _ = c.forward()
        rest = torch.ones(T, dtype=torch.bool, device="cuda")
        rest[[3, T - 1]] = False
        assert loss[[3, T - 1]].isnan().all() and torch.equal(loss[rest], clean[rest])


@pytest.mark.parametrize("dtype", [F16, BF16], ids=["f16", "bf16"])
@pytest.mark.parametrize("T", [40, 300])
def test_nonfinite_upstream_gradients_stay_alone(T, dtype):
    # a token whose dloss overflowed takes its own row of dX and dW, no other row
    c = Case(T, 500, 64, dtype, seed=16, weights="each")
    c.dloss[3] = 0.5 * c.dloss.abs().max()
    clean, _ = c.backward()
    rest = torch.arange(T, device="cuda") != 3
    for bad in ("inf", "-inf", "nan"):
        c.dloss[3] = float(bad)
        dx, dw = c.backward()
        assert not dx[3].isfinite().any() and torch.equal(dx[rest], clean[rest])
        assert not dw.isfinite().all()
    c.dloss[:] = float("inf")
    dx, _ = c.backward()
    assert not dx.isfinite().any()


@pytest.mark.parametrize("T", [40, 300])
def test_subnormal_upstream_gradients(T):
    # powers of two: every step but the last product is the same but for its
    # exponent, and that one rounds to a multiple of 2^-149
    c = Case(T, 500, 64, BF16, seed=17)
    c.dloss.fill_(1.0)
    one, _ = c.backward(out_dtype=torch.float32)
    c.dloss.fill_(2.0 ** -130)
    dx, dw = c.backward(out_dtype=torch.float32)
    assert ((dx.double() - one.double() * 2.0 ** -130).abs() <= 2.0 ** -150).all() and dw.isfinite().all()


def test_minus_infinity_logits():
    # a vocabulary entry whose logit is -inf has probability zero
    x = torch.zeros(5, 16, dtype=F16, device="cuda")
    x[:, 0] = 1
    w = torch.zeros(700, 16, dtype=F16, device="cuda")
    w[64:, 0] = float("-inf")        # whole tiles, and part of one
    target = torch.tensor([0, 1, 63, 5, 64], device="cuda")
    loss, lse = trt.linear_xent(x, w, target)
    want = np.log(64)
    assert torch.allclose(lse.cpu().double(), torch.full((5,), want, dtype=torch.float64), atol=1e-6, rtol=0)
    assert torch.allclose(loss[:4].cpu().double(), torch.full((4,), want, dtype=torch.float64), atol=1e-6, rtol=0)
    assert loss[4] == float("inf")


def test_one_value_of_dloss_for_all():
    c = Case(100, 300, 64, BF16, seed=16)
    _, lse = c.forward()
    full = trt.linear_xent_bwd(c.x, c.w, c.target, lse, torch.full((100,), 0.25, device="cuda"))
    one = torch.tensor(0.25, device="cuda")
    for d in (one, one.view(1), one.expand(100)):
        assert all(torch.equal(a, b) for a, b in zip(trt.linear_xent_bwd(c.x, c.w, c.target, lse, d), full))
    strided = torch.full((100, 3), 0.25, device="cuda")[:, 1]
    assert all(torch.equal(a, b) for a, b in zip(trt.linear_xent_bwd(c.x, c.w, c.target, lse, strided), full))


def test_gradients_against_differences():
    """The directional derivative of sum dloss loss against <dx, v> and <dw, v>,
    with inputs that are exact in binary16 on both sides of the step.

    x is a multiple of 2^-6 and moves by +-2^-4 along a sign vector; logits
    are sums of 32 products of a few units each, off by 34 u 32 <= 7e-5 at
    worst, so a difference of losses over 2^-3 is off by 16 * 7e-5 = 1.1e-3 a
    token and 20 tokens' by 0.023 at worst.  The third derivative's part is
    step^2 / 6 times a third cumulant of the row's directional logits
    (|dz/ds| <= sum |w| <= 32 * 0.5): 6.5e-4 * 8 a token, 0.1 for 20.
    The gradient itself is rounded to 2^-11 of 20 tokens' 16: 0.16.
    """
    gen = torch.Generator().manual_seed(17)
    T, V, D = 20, 90, 32
    x = (torch.randint(-64, 65, (T, D), generator=gen) / 64.0).cuda()
    w = (torch.randint(-32, 33, (V, D), generator=gen) / 64.0).cuda()
    target = torch.randint(0, V, (T,), generator=gen).cuda()
    vx = (torch.randint(0, 2, (T, D), generator=gen) * 2 - 1).float().cuda()
    vw = (torch.randint(0, 2, (V, D), generator=gen) * 2 - 1).float().cuda()
    up = torch.ones(T, device="cuda")
    step = 2.0 ** -4

    def L(x, w):
        return float(trt.linear_xent(x.half(), w.half(), target)[0].double().sum())

    _, lse = trt.linear_xent(x.half(), w.half(), target)
    dx, dw = trt.linear_xent_bwd(x.half(), w.half(), target, lse, up)
    along = (L(x + step * vx, w) - L(x - step * vx, w)) / (2 * step)
    assert abs(along - float((dx.double() * vx.double()).sum())) < 0.3
    along = (L(x, w + step * vw) - L(x, w - step * vw)) / (2 * step)
    assert abs(along - float((dw.double() * vw.double()).sum())) < 0.3


def test_repeats_bit_for_bit_whatever_the_workspace_holds():
    c = Case(400, 3000, 136, F16, seed=18, ignored=0.3, weights="each", nan_ignored=True)
    first = (*c.forward(), *c.backward())
    for fill in (0, 0x3C):
        need = trt.linear_xent_bwd_workspace_size(c.T, c.V, c.D)
        torch.full((need,), fill, dtype=torch.uint8, device="cuda")
        again = (*c.forward(), *c.backward())
        assert all(torch.equal(a, b) for a, b in zip(first, again))


def test_batched_shapes_and_another_stream():
    c = Case(120, 300, 64, BF16, seed=19, ignored=0.2)
    loss, lse = trt.linear_xent(c.x, c.w, c.target)
    dx, dw = trt.linear_xent_bwd(c.x, c.w, c.target, lse, c.dloss)
    x3, t3 = c.x.contiguous().view(4, 30, 64), c.target.view(4, 30)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        l3, e3 = trt.linear_xent(x3, c.w, t3)
        dx3, dw3 = trt.linear_xent_bwd(x3, c.w, t3, e3, c.dloss.view(4, 30))
    side.synchronize()
    assert l3.shape == (4, 30) and dx3.shape == (4, 30, 64)
    assert torch.equal(l3.view(-1), loss) and torch.equal(dx3.view(-1, 64), dx) and torch.equal(dw3, dw)


def test_norm_head_loss_and_back_in_one_graph():
    """The four operators as a training step chains them, captured once and
    replayed on new inputs, against the same calls made eagerly; and the
    chain's gradient with respect to the norm's input against 64 bits.

    The oracle takes the norm's rounded output as the head's input, so what is
    left of the last comparison is the rounding of dh to bf16 (h |dh| an
    element, through the norm's Jacobian: r (|u| + mean |u| + |h| mean |u h|) <=
    r h 3 max |dh gamma| (1 + max |h|)), dh's own error and the norm's, each no
    larger than that: four times it.
    """
    T, V, D = 200, 900, 96
    gen = torch.Generator(device="cuda").manual_seed(20)
    x = torch.randn(T, D, device="cuda", generator=gen).bfloat16()
    gamma, beta = (torch.randn(D, device="cuda", generator=gen) for _ in range(2))
    w = (torch.randn(V, D, device="cuda", generator=gen) * 0.2).bfloat16()
    target = torch.randint(0, V, (T,), device="cuda", generator=gen)
    target[::5] = IGNORE
    up = torch.full((T,), 1.0 / T, device="cuda")

    def step():
        y = trt.layernorm(x, gamma, beta)
        loss, lse = trt.linear_xent(y, w, target)
        dy, dw = trt.linear_xent_bwd(y, w, target, lse, up)
        return (y, loss, lse, dy, dw, *trt.layernorm_bwd(dy, x, gamma))

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for seed in range(4):
        gen.manual_seed(100 + seed)
        x.copy_(torch.randn(T, D, device="cuda", generator=gen))
        target.copy_(torch.randint(0, V, (T,), device="cuda", generator=gen))
        target[seed::3] = IGNORE
        for t in out:
            t.fill_(3)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, step())), seed

    from oracle import norm_ref
    y, dxn = out[0], out[5]
    dh, _ = xent_ref.backward(f64(y), f64(w), target.cpu().numpy(), f64(up))
    want, _, _ = norm_ref.backward(dh, f64(x), f64(gamma), 1e-5)
    h, r = norm_ref.stats(f64(x), 1e-5)
    most = np.abs(dh * f64(gamma)).max(1, keepdims=True)
    check(dxn, want, half_step(want, BF16) + 4 * r * 2.0 ** -8 * 3 * most * (1 + np.abs(h).max(1, keepdims=True)), "chain")


# ---- offsets past 2^31 and 2^32 bytes --------------------------------------------------

def test_rows_far_apart():
    # rows of x and w 16 MB apart: offsets of 4.8 and 8 GB
    c = Case(300, 500, 64, BF16, seed=31, pad=8_000_000, ignored=0.3, weights="each")
    c.check_forward()
    c.check_backward()


@pytest.fixture(scope="module")
def large_weight():
    # 4.4 GB of W, entries of a fixed size each, the last vocabulary entries as any other
    gen = torch.Generator(device="cuda").manual_seed(32)
    w = torch.empty(540_000, 4096, dtype=BF16, device="cuda")
    for v in range(0, len(w), 60_000):
        w[v:v + 60_000] = torch.randn(60_000, 4096, generator=gen, device="cuda") / 64
    yield w
    del w
    torch.cuda.empty_cache()


@pytest.mark.parametrize("T", [3, 40, 200])
def test_large_weight(large_weight, T):
    w = large_weight
    V, D = w.shape
    gen = torch.Generator(device="cuda").manual_seed(T)
    x = (2 * torch.randn(T, D, generator=gen, device="cuda")).to(BF16)
    target = torch.randint(0, V, (T,), generator=gen, device="cuda")
    target[0], target[1], target[2] = V - 1, 262_143, 262_145
    dloss = torch.full((T,), 1.0 / T, device="cuda")
    loss, lse = trt.linear_xent(x, w, target)
    dx, dw = trt.linear_xent_bwd(x, w, target, lse, dloss, out_dtype=torch.float32)
    steps = [slice(v, min(v + 60_000, V)) for v in range(0, V, 60_000)]
    z = torch.cat([x.double() @ w[s].double().T for s in steps], 1)
    want = torch.logsumexp(z, 1)
    S = max(float((x.abs().double() @ w[s].abs().double().T).max()) for s in steps)
    dz = (D + 2) * U * S
    tol = dz + U * (4 * float(z.abs().max()) + 4 * float(want.max()) + 8 + 64 + 3 * V / 64)
    assert ((lse.double() - want).abs() <= tol).all()
    assert ((loss.double() - (want - z.gather(1, target[:, None])[:, 0])).abs() <= 2 * tol).all()
    # G is off by half a step (its square with two rows a token) and by lse's and
    # the logits' errors; dX's sums run over V, dW's over T
    p = torch.exp(z - want[:, None])
    g = p / T
    g[torch.arange(T), target] -= 1.0 / T
    h = torch.finfo(BF16).eps / 2
    dg = (h * h if T <= 64 else h) * g.abs() + 2 * tol * p / T
    rdx, tdx = torch.zeros(T, D, dtype=torch.float64, device="cuda"), torch.zeros(T, D, dtype=torch.float64, device="cuda")
    for s in steps:
        ws = w[s].double()
        rdx += g[:, s] @ ws
        tdx += dg[:, s] @ ws.abs() + U * (2 * V + 4) * (g[:, s].abs() @ ws.abs())
        rdw = g[:, s].T.contiguous() @ x.double()
        tdw = dg[:, s].T.contiguous() @ x.abs().double() + U * (2 * T + 5) * (g[:, s].abs().T.contiguous() @ x.abs().double())
        assert ((dw[s].double() - rdw).abs() <= tdw + 2.0 ** -140).all(), s
    assert ((dx.double() - rdx).abs() <= tdx + U * rdx.abs()).all()


# ---- calls at once, graphs that share a workspace --------------------------------------

def test_two_streams_at_once():
    cases = [Case(300, 9000, 264, BF16, seed=41, ignored=0.2), Case(60, 20000, 136, BF16, seed=42)]

    def step(c):
        loss, lse = trt.linear_xent(c.x, c.w, c.target, ignore_index=IGNORE)
        return (loss, lse) + trt.linear_xent_bwd(c.x, c.w, c.target, lse, c.dloss, ignore_index=IGNORE)

    want = [step(c) for c in cases]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in cases]
    got = [[], []]
    for _ in range(5):
        for c, st, g in zip(cases, streams, got):
            with torch.cuda.stream(st):
                g.append(step(c))
    torch.cuda.synchronize()
    for w, g in zip(want, got):
        for one in g:
            assert all(torch.equal(a, b) for a, b in zip(one, w))


def test_two_graphs_share_a_workspace():
    T, V, D = 200, 5000, 128
    cases = [Case(T, V, D, BF16, seed=s, ignored=0.3) for s in (43, 44)]
    ws = dirty(max(trt.linear_xent_workspace_size(T, V, D), trt.linear_xent_bwd_workspace_size(T, V, D)))

    def step(c):
        loss, lse = trt.linear_xent(c.x, c.w, c.target, ignore_index=IGNORE, workspace=ws)
        return (loss, lse) + trt.linear_xent_bwd(c.x, c.w, c.target, lse, c.dloss, ignore_index=IGNORE, workspace=ws)

    want = [[t.clone() for t in step(c)] for c in cases]
    side = torch.cuda.Stream()
    graphs, outs = [], []
    for c in cases:
        with torch.cuda.stream(side):
            step(c)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(step(c))
        graphs.append(g)
    for turn in range(6):
        k = turn % 2
        for t in outs[k]:
            t.fill_(-1)
        graphs[k].replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(outs[k], want[k])), turn
