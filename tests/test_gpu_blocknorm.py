"""GPU parity of a block's norms with its gate and residual, and of their
gradients, against the 64-bit oracle.

Tolerances count roundings, first order, u = 2^-24 (see test_gpu_norm.py for
what a norm's sums leave: at most 54 additions to a sum there and here):

    |error of N(x)| <= eN(x) = u (64 + 72 |N(x)|)

A perturbation d of x moves N(x) by at most rstd (|d| + mean |d| + |N| mean(|N| d)).
Forward, with E the stream's error:

    E     <= |gate pg| eN(y) + u (4 |gate pg N(y)| + 3 |gate pb| + 2 |alpha r| + 2 |r'|)
    |error of r'| <= half step + E
    |error of h|  <= half step + |g| (eN(r') + rstd (E + mean E + |N| mean(|N| E))) + 4 u (|h| + |b|)

(without the norm behind the block: N(y) = y, eN(y) = 0).  Backward, the
Jacobian of v comes out to J(v) = u rstd (200 rms(v) + 80 |v| + 260 rms(v) |N|), so

    Ee    <= J(dh g) + u (|e| + |dr|),           |error of dr| <= half step + |alpha| Ee + 2 u |dr|
    Es    <= |gate pg| Ee + 3 u |s|
    |error of dy| <= half step + J(s) + rstd (Es + mean Es + |N| mean(|N| Es))

and a sum over rows of terms x, each off by Ex, is off by sum Ex + u depth sum |x|,
with depth the rows of a slice, the groups of a workgroup (8), a wave's slices and
the 16 waves.
"""
import itertools

import numpy as np
import pytest
import torch

import thread_register_tile_amd as trt
from oracle import act8_ref, blocknorm_ref as ref

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
CODE = {torch.float16: trt.F16, torch.bfloat16: trt.BF16, torch.float32: trt.F32}
F16, BF16, F32 = torch.float16, torch.bfloat16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    trt.lib()


def f64(t):
    return None if t is None else t.detach().cpu().to(torch.float64).numpy()


def half_step(want, dtype):
    fi = torch.finfo(dtype)
    return np.maximum(np.abs(want), fi.tiny) * (fi.eps / 2)


def check(got, want, err, what):
    """err: the error before the result's own rounding."""
    hg = f64(got)
    assert hg.shape == want.shape, what
    tol = half_step(want, got.dtype) + 1.01 * err
    bad = ~(np.abs(hg - want) <= tol)
    assert not bad.any(), (what, int(bad.sum()), float(np.nanmax(np.abs(hg - want) / tol)))


def strided(t, pad, offset, fill):
    rows, cols = t.shape
    ld = cols + pad
    buf = torch.full((offset + rows * ld + 64,), fill, dtype=t.dtype)
    view = buf[offset:offset + rows * ld].view(rows, ld)[:, :cols]
    view.copy_(t)
    dev = buf.cuda()
    return dev, dev[offset:offset + rows * ld].view(rows, ld)[:, :cols]


def untouched(buf, rows, cols, pad, offset):
    ld = cols + pad
    b = f64(buf)
    body = b[offset:offset + rows * ld].reshape(rows, ld)
    return (b[:offset] == 77).all() and (b[offset + rows * ld:] == 77).all() and (body[:, cols:] == 77).all()


def e_norm(hat):
    return U * (64 + 72 * np.abs(hat))


def moved(E, hat, rstd):
    return rstd * (E + E.mean(1, keepdims=True) + np.abs(hat) * (np.abs(hat) * E).mean(1, keepdims=True))


def jacobian_error(v, hat, rstd):
    rms = np.sqrt((v * v).mean(1, keepdims=True))
    return U * rstd * (200 * rms + 80 * np.abs(v) + 260 * rms * np.abs(hat))


def mag(v):
    return 1.0 if v is None else np.abs(v)


def forward_errors(h, out, want_h, m):
    hat, _ = ref.norm(h["y"], m["eps"], m["rms"]) if m["post"] else (h["y"], None)
    gp, gb = mag(h["gate"]) * mag(h["pg"]), mag(h["gate"]) * (0.0 if h["pb"] is None else np.abs(h["pb"]))
    E = U * (4 * gp * np.abs(hat) + 3 * gb + 2 * np.abs(m["alpha"] * h["r"]) + 2 * np.abs(out))
    if m["post"]:
        E = E + gp * e_norm(hat)
    nh, rstd = ref.norm(out, m["eps"], m["rms"])
    b = 0.0 if h["b"] is None else np.abs(h["b"])
    return E, mag(h["g"]) * (e_norm(nh) + moved(E, nh, rstd)) + 4 * U * (np.abs(want_h) + b)


def run_case(rows, cols, dtype, *, pdt=F32, gdt=None, rms=False, post=True, gate="channel", span=None, alpha=1.0, eps=1e-5,
             vectors="all", up="both", saved="same", pad=0, offset=0, mean=0.0, scale=1.0, seed=0):
    gen = torch.Generator().manual_seed(seed)
    what = (rows, cols, dtype, pdt, gdt, rms, post, gate, span, alpha, vectors, up, saved, pad, offset)
    gdt = gdt or dtype

    def normal(*shape):
        return torch.randn(*shape, generator=gen, dtype=torch.float64)

    def made(t):
        return strided(t.to(dtype), pad, offset, float("nan"))[1]

    r, y = made(normal(rows, cols) * scale + mean), made(normal(rows, cols) * torch.exp(normal(rows, 1)) * scale + mean)
    dh, dr = made(normal(rows, cols)), made(normal(rows, cols) * torch.exp(0.5 * normal(rows, 1)))
    give = {"all": (1, 1, 1, 1), "gammas": (1, 0, 1, 0), "none": (0, 0, 0, 0), "betas": (0, 1, 0, 1)}[vectors]
    pg, pb, g, b = ((1 + 0.3 * normal(cols)).to(pdt).cuda() if on else None for on in give)
    if not post:
        pg = pb = None
    shape = {"none": None, "channel": (cols,), "sequence": (-(-rows // span) if span else 0, cols), "each": (rows, cols)}[gate]
    gt = None if shape is None else (0.5 + 0.4 * normal(*shape)).to(gdt).cuda()
    rpg = span if gate == "sequence" else None
    m = dict(rms=rms, post=post, alpha=alpha, eps=eps)
    kw = dict(post_gamma=pg, post_beta=pb, gamma=g, rows_per_gate=rpg, **m)

    # forward
    h = {k: f64(v) for k, v in dict(r=r, y=y, pg=pg, pb=pb, g=g, b=b).items()}
    full = None if gt is None else ref.spread(f64(gt).reshape(-1, cols), rows, {"channel": rows, "each": 1}.get(gate, span))
    h["gate"] = full
    want_r, want_h = ref.forward(h["r"], h["y"], full, h["pg"], h["pb"], h["g"], h["b"], alpha, eps, rms, post)
    bufs = [strided(torch.full((rows, cols), 77.0, dtype=dtype), pad, offset, 77.0) for _ in range(4)]
    out, hh = bufs[0][1], bufs[1][1]
    trt.block_norm(r, y, gt, beta=b, r_out=out, h=hh, **kw)
    E, Eh = forward_errors(h, want_r, want_h, m)
    check(out, want_r, E, (what, "r_out"))
    check(hh, want_h, Eh, (what, "h"))
    only, no_h = trt.block_norm(r, y, gt, beta=b, need_h=False, **kw)
    assert no_h is None and torch.equal(only, out), what

    # backward, from the stream that the forward pass stored
    has_h, has_r = up != "r", up != "h"
    sr, sy = out.clone(), y
    if saved == "8bit":
        sr, sy = trt.act8_pack(out), trt.act8_pack(y)
        hx, hy = (f64(torch.from_numpy(act8_ref.unpack(q.cpu().numpy(), s.cpu().numpy())).to(dtype)) for q, s in (sr, sy))
    else:
        hx, hy = f64(sr), h["y"]
    need = trt.block_norm_bwd_workspace_size(rows, cols, 0 if gt is None else (rpg or {"channel": rows, "each": 1}[gate]), CODE[dtype])
    ws = torch.full((need + 64,), 0xFF, dtype=torch.uint8, device="cuda")
    d_r, d_y = bufs[2][1], bufs[3][1]
    got = trt.block_norm_bwd(dh if has_h else None, dr if has_r else None, sr if has_h else None, sy, gt, dr=d_r, dy=d_y,
                             workspace=ws[:need], **kw)
    assert (ws[need:] == 0xFF).all(), what
    hdh, hdr = f64(dh) if has_h else None, f64(dr) if has_r else None
    want = ref.backward(hdh, hdr, hx, hy, full, h["pg"], h["pb"], h["g"], alpha, eps, rms, post)
    e = want["dr"] / alpha
    Ee = U * (np.abs(e) + (np.abs(hdr) if has_r else 0))
    if has_h:
        nx, rx = ref.norm(hx, eps, rms)
        Ee = Ee + jacobian_error(hdh * (1.0 if g is None else h["g"]), nx, rx)
    check(got[0], want["dr"], abs(alpha) * Ee + 2 * U * np.abs(want["dr"]), (what, "dr"))
    gp = mag(full) * mag(h["pg"])
    s = (1.0 if full is None else full) * e * (1.0 if pg is None else h["pg"])
    Es = gp * Ee + 3 * U * np.abs(s)
    if post:
        ny, ry = ref.norm(hy, eps, rms)
        check(got[1], want["dy"], jacobian_error(s, ny, ry) + moved(Es, ny, ry), (what, "dy"))
        En = e_norm(ny)
    else:
        ny, En = hy, 0.0
        check(got[1], want["dy"], Es + U * np.abs(s), (what, "dy"))
    slices = need // (16 * cols)
    rows_of = span if gate == "sequence" else rows
    groups = -(-rows // rows_of)
    depth = -(-rows_of // max(1, slices // groups)) + 8 + -(-slices // 16) + 16 + 4
    if gt is not None:
        apg, apb = mag(h["pg"]), 0.0 if h["pb"] is None else np.abs(h["pb"])
        dgate = want["dgate"]
        ey, Ey = np.abs(e * ny), np.abs(ny) * Ee + np.abs(e) * En
        if gate == "each":
            err = (apg * np.abs(ny) + apb) * Ee + apg * np.abs(e) * En + U * (4 * apg * ey + 3 * apb * np.abs(e))
        else:
            dgate = ref.gather(dgate, rows_of)
            err = apg * ref.gather(Ey + U * (depth + 3) * ey, rows_of) + apb * ref.gather(Ee + U * (depth + 3) * np.abs(e), rows_of)
        assert got[2].dtype == gdt and got[2].shape == gt.shape, what
        check(got[2].view(-1, cols), dgate.reshape(-1, cols), err.reshape(-1, cols), (what, "dgate"))
    else:
        assert got[2] is None
    if post:
        ge = mag(full) * np.abs(e)
        check(got[3], want["dpg"], (mag(full) * (np.abs(ny) * Ee + np.abs(e) * En) + U * (depth + 4) * ge * np.abs(ny)).sum(0), (what, "dpg"))
        check(got[4], want["dpb"], (mag(full) * Ee + U * (depth + 4) * ge).sum(0), (what, "dpb"))
    else:
        assert got[3] is None and got[4] is None
    if has_h:
        a = np.abs(hdh)
        check(got[5], want["dg"], (a * e_norm(nx) + U * depth * a * np.abs(nx)).sum(0), (what, "dg"))
        check(got[6], want["db"], U * depth * a.sum(0), (what, "db"))
        pt = pdt if (g is not None or pg is not None or pb is not None) else F32
        assert got[5].dtype == pt
    else:
        assert got[5] is None and got[6] is None
    for buf, _ in bufs:
        assert untouched(buf, rows, cols, pad, offset), what
    again = trt.block_norm_bwd(dh if has_h else None, dr if has_r else None, sr if has_h else None, sy, gt, params=False, **kw)
    assert torch.equal(again[0], got[0]) and torch.equal(again[1], got[1]) and again[2:] == (None,) * 5, what


# widths on both sides of every change of the waves to a row, and odd ones
W16 = [1, 7, 8, 100, 511, 512, 513, 1024, 1025, 2000, 2049, 4096, 4097, 5000, 6144, 6145, 8192, 8200, 12288, 12289, 16383, 16384]
W32 = [1, 3, 4, 255, 257, 511, 513, 1023, 1025, 2047, 2050, 3100, 4096, 4099, 6144, 6148, 8190, 8192]
MIX = list(itertools.product([False, True], [True, False], ["channel", "sequence", "each", "none"]))


@pytest.mark.parametrize("i,cols", list(enumerate(W16)))
@pytest.mark.parametrize("dtype", [F16, BF16])
def test_widths_16(i, cols, dtype):
    for j, rows in enumerate((1, 5, 67)):
        rms, post, gate = MIX[(5 * i + 3 * j + (dtype == BF16)) % len(MIX)]
        run_case(rows, cols, dtype, rms=rms, post=post, gate=gate, span=3 if gate == "sequence" else None, pdt=F32 if i % 2 else dtype,
                 gdt=F32 if (i + j) % 3 == 0 else None, saved="8bit" if (i + j) % 2 else "same", seed=i)


@pytest.mark.parametrize("i,cols", list(enumerate(W32)))
def test_widths_32(i, cols):
    for j, rows in enumerate((1, 5, 67)):
        rms, post, gate = MIX[(5 * i + 3 * j) % len(MIX)]
        run_case(rows, cols, F32, rms=rms, post=post, gate=gate, span=3 if gate == "sequence" else None,
                 saved="8bit" if (i + j) % 2 else "same", seed=i)


@pytest.mark.parametrize("rms,post,gate", MIX)
@pytest.mark.parametrize("dtype,gdt", [(F16, F32), (BF16, BF16), (F32, F32)])
def test_every_form(rms, post, gate, dtype, gdt):
    for cols, saved in ((264, "same"), (1500, "8bit"), (2304, "same")):
        run_case(37, cols, dtype, rms=rms, post=post, gate=gate, gdt=gdt, span=8 if gate == "sequence" else None, alpha=-2.5,
                 saved=saved, pad=3, offset=1, seed=cols)


@pytest.mark.parametrize("up", ["h", "r"])
@pytest.mark.parametrize("vectors", ["none", "gammas", "betas"])
@pytest.mark.parametrize("gate", ["none", "sequence", "each"])
def test_absent_operands(up, vectors, gate):
    run_case(21, 1100, BF16, pdt=BF16, vectors=vectors, up=up, gate=gate, span=10 if gate == "sequence" else None)


# workgroups of several turns, slices of gate rows, more gate rows than units, a
# last gate row of one row
@pytest.mark.parametrize("rows,cols,gate,span", [
    (9000, 64, "channel", None), (9000, 64, "sequence", 1000), (5001, 520, "sequence", 5), (5001, 100, "sequence", 2500),
    (3001, 1030, "each", None), (2500, 2056, "none", None), (2500, 2056, "sequence", 39), (700, 8200, "channel", None),
    (513, 5000, "sequence", 256), (300, 16384, "sequence", 77)])
@pytest.mark.parametrize("dtype,rms,saved", [(BF16, True, "8bit"), (F16, False, "same")])
def test_many_rows(rows, cols, gate, span, dtype, rms, saved):
    run_case(rows, cols, dtype, gate=gate, span=span, rms=rms, saved=saved)


@pytest.mark.parametrize("rows,cols,gate,span", [(4001, 1023, "none", None), (3000, 300, "sequence", 7), (600, 8192, "channel", None)])
def test_many_rows_32(rows, cols, gate, span):
    run_case(rows, cols, F32, gate=gate, span=span, alpha=0.5)


@pytest.mark.parametrize("mean,scale", [(100.0, 1.0), (0.0, 1e-3), (0.0, 1e4)])
def test_rows_far_from_zero(mean, scale):
    run_case(40, 1111, F32, mean=mean, scale=scale)
    run_case(40, 4100, BF16, mean=mean, scale=scale, rms=True)


@pytest.mark.parametrize("mean,scale", [(100.0, 1.0), (0.0, 1e-3), (0.0, 1e4)])
def test_rows_far_from_zero_in_8_bits(mean, scale):
    for cols, dtype in ((1111, F32), (4100, BF16), (16384, BF16)):
        run_case(20, cols, dtype, mean=mean, scale=scale, saved="8bit")


def test_leading_dimensions_and_broadcast_gates():
    x, y = (torch.randn(3, 5, 40, dtype=BF16, device="cuda") for _ in range(2))
    for gate, rows in ((torch.randn(3, 1, 40, device="cuda"), 5), (torch.randn(1, 1, 40, device="cuda"), 15),
                       (torch.randn(3, 5, 40, device="cuda"), 1)):
        a = trt.block_norm(x, y, gate)
        b = trt.block_norm(x.view(15, 40), y.view(15, 40), gate.reshape(-1, 40), rows_per_gate=rows)
        assert all(torch.equal(p.view(15, 40), q) for p, q in zip(a, b))
        a = trt.block_norm_bwd(x, y, trt.act8_pack(x), trt.act8_pack(y), gate)
        b = trt.block_norm_bwd(x.view(15, 40), y.view(15, 40), trt.act8_pack(x.view(15, 40)), trt.act8_pack(y.view(15, 40)), gate.reshape(-1, 40),
                               rows_per_gate=rows)
        assert a[2].shape == gate.shape
        assert all(torch.equal(p.reshape(q.shape), q) for p, q in zip(a, b))
    # a row without leading dimensions
    assert trt.block_norm(x[0, 0], y[0, 0])[0].shape == (40,)


def test_not_finite_rows_stay_alone():
    x, y, dh, dr = (torch.randn(40, 600, dtype=BF16, device="cuda") for _ in range(4))
    gate = torch.randn(4, 600, device="cuda", dtype=BF16)
    clean = trt.block_norm(x, y, gate, rows_per_gate=10), trt.block_norm_bwd(dh, dr, x, y, gate, rows_per_gate=10)
    y[13, 5], x[27, 599] = float("nan"), float("inf")
    out, h = trt.block_norm(x, y, gate, rows_per_gate=10)
    keep = torch.ones(40, dtype=torch.bool)
    keep[[13, 27]] = False
    for got, want in zip((out, h), clean[0]):
        assert torch.equal(got[keep], want[keep])
    assert out[13].isnan().all() and h[13].isnan().all() and out[27, 599].isinf() and h[27].isnan().any()
    got = trt.block_norm_bwd(dh, dr, x, y, gate, rows_per_gate=10)
    assert torch.equal(got[0][keep], clean[1][0][keep]) and torch.equal(got[1][keep], clean[1][1][keep])
    assert got[0][27].isnan().all() and got[1][13].isnan().all() and not got[0][13].isnan().any()
    # gate rows 0 and 3 are not touched, 1 and 2 are
    assert torch.equal(got[2][[0, 3]], clean[1][2][[0, 3]]) and got[2][1].isnan().all() and got[2][2].isnan().all()


def test_constant_rows():
    """No spread: the layer norm is 0 / sqrt(eps)."""
    x = torch.full((6, 300), 3.0, device="cuda")
    out, h = trt.block_norm(x, x, gamma=torch.ones(300, device="cuda"), eps=1e-5)
    assert torch.equal(out, x) and (h == 0).all()
    out, h = trt.block_norm(torch.zeros_like(x), torch.zeros_like(x), rms=True)
    assert (out == 0).all() and (h == 0).all()
    got = trt.block_norm_bwd(x, x, x, x)
    assert all(torch.isfinite(t).all() for t in got if t is not None)


def test_offsets_past_32_bits():
    rows, ld = 3, (1 << 30) + 64           # 16-bit rows 2 GiB apart
    buf = torch.empty(rows * ld, dtype=BF16, device="cuda").view(rows, ld)[:, :1000]
    x, y, dh, dr = (torch.randn(rows, 1000, dtype=BF16, device="cuda") for _ in range(4))
    buf.copy_(x)
    want, got = trt.block_norm(x, y), trt.block_norm(buf, y)
    assert torch.equal(want[0], got[0]) and torch.equal(want[1], got[1])
    want = trt.block_norm_bwd(dh, dr, x, y)
    got = trt.block_norm_bwd(dh, dr, buf, y)
    assert all(torch.equal(a, b) for a, b in zip(want, got) if a is not None)
    trt.block_norm(x, y, r_out=buf)
    assert torch.equal(buf, trt.block_norm(x, y)[0])


def test_graph_on_a_stream_of_its_own():
    """Captured and replayed with new inputs while the current stream runs the
    same operators with another workspace."""
    rows, cols = 700, 1500
    gen = torch.Generator(device="cuda").manual_seed(3)
    x, y, dh, dr = (torch.randn(rows, cols, dtype=BF16, device="cuda", generator=gen) for _ in range(4))
    gate, g = torch.randn(7, cols, device="cuda", generator=gen), torch.randn(cols, device="cuda", generator=gen)
    kw = dict(rows_per_gate=100, post_gamma=g, gamma=g)
    ws = torch.empty(trt.block_norm_bwd_workspace_size(rows, cols, 100, trt.BF16), dtype=torch.uint8, device="cuda")
    side = torch.cuda.Stream()

    def work():
        out, h = trt.block_norm(x, y, gate, **kw)
        return out, h, *trt.block_norm_bwd(dh, dr, trt.act8_pack(out), trt.act8_pack(y), gate, workspace=ws, **kw)

    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        work()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        captured = work()
    for turn in range(4):
        for t in (x, y, dh, dr):
            t.copy_(torch.randn(rows, cols, device="cuda", generator=gen))
        torch.cuda.synchronize()
        graph.replay()
        out, h = trt.block_norm(x, y, gate, **kw)
        eager = (out, h, *trt.block_norm_bwd(dh, dr, trt.act8_pack(out), trt.act8_pack(y), gate, **kw))
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(captured, eager)), turn
