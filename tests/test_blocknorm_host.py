"""CPU tests of the block norm's entry points: refusals before any HIP call,
workspace sizes, the binding's shapes, and the oracle's gradients against
differences."""
import numpy as np
import pytest
import torch

import thread_register_tile_amd as trt
from oracle import blocknorm_ref

BASE = 1 << 24     # fake, well-separated addresses: never dereferenced
BLOCK = dict(gate=BASE * 10, ldg=64, rows_per_gate=3, post_gamma=BASE * 11, post_beta=BASE * 12, gamma=BASE * 13,
             beta=BASE * 14, alpha=1.0, eps=1e-5, post=1, rms=0, gate_dtype=trt.F16, param_dtype=trt.F32)


def block(kw):
    return trt.Block(**{k: (v or None) if k in ("gate", "post_gamma", "post_beta", "gamma", "beta") else v
                        for k, v in {**BLOCK, **{k: kw.pop(k) for k in list(kw) if k in BLOCK}}.items()})


def forward(**kw):
    b = block(kw) if not kw.pop("no_block", False) else None
    a = dict(rows=8, cols=64, r=BASE, ldr=64, y=BASE * 2, ldy=64, r_out=BASE * 3, ldro=64, h=BASE * 4, ldh=64, dtype=trt.F16)
    a.update(kw)
    return trt.lib().trt_block_norm(a["rows"], a["cols"], a["r"], a["ldr"], a["y"], a["ldy"], b, a["r_out"], a["ldro"],
                                    a["h"], a["ldh"], a["dtype"], None)


def backward(**kw):
    b = block(kw) if not kw.pop("no_block", False) else None
    a = dict(rows=8, cols=64, dh=BASE, lddh=64, dro=BASE * 2, lddro=64, r=BASE * 3, ldr=64, rs=0, rls=2, y=BASE * 4, ldy=64,
             ys=0, yls=2, dr=BASE * 5, lddr=64, dy=BASE * 6, lddy=64, dgate=BASE * 20, lddg=64, dpg=BASE * 21, dpb=BASE * 22,
             dg=BASE * 23, db=BASE * 24, dtype=trt.F16, ws=BASE * 30, wsb=1 << 20, no_grads=False, no_y=False)
    a.update(kw)
    grads = None if a["no_grads"] else trt.BlockGrads(a["dgate"] or None, a["lddg"], a["dpg"] or None, a["dpb"] or None,
                                                      a["dg"] or None, a["db"] or None)
    sr = trt.Saved(a["r"] or None, a["ldr"], a["rs"] or None, a["rls"])
    sy = None if a["no_y"] else trt.Saved(a["y"] or None, a["ldy"], a["ys"] or None, a["yls"])
    return trt.lib().trt_block_norm_bwd(a["rows"], a["cols"], a["dh"] or None, a["lddh"], a["dro"] or None, a["lddro"], sr,
                                        sy, b, a["dr"], a["lddr"], a["dy"], a["lddy"], grads, a["dtype"], a["ws"], a["wsb"],
                                        None)


COMMON = [
    (dict(rows=0), trt.ERR_SIZE), (dict(cols=0), trt.ERR_SIZE), (dict(rows=(1 << 30) + 1), trt.ERR_SIZE),
    (dict(no_block=True), trt.ERR_NULL), (dict(dtype=0), trt.ERR_DTYPE), (dict(param_dtype=trt.BF16), trt.ERR_DTYPE),
    (dict(gate_dtype=trt.BF16), trt.ERR_DTYPE), (dict(gate_dtype=0), trt.ERR_DTYPE), (dict(rows_per_gate=0), trt.ERR_SIZE),
    (dict(rows_per_gate=-1), trt.ERR_SIZE), (dict(ldg=0), trt.ERR_STRIDE), (dict(gate=BASE * 10 + 1), trt.ERR_ALIGN),
    (dict(post_gamma=BASE * 11 + 2), trt.ERR_ALIGN), (dict(post=2), trt.ERR_ARG), (dict(rms=-1), trt.ERR_ARG),
    (dict(post=0), trt.ERR_ARG), (dict(post=0, post_gamma=0), trt.ERR_ARG),
    (dict(eps=-1.0), trt.ERR_ARG), (dict(eps=float("nan")), trt.ERR_ARG), (dict(eps=float("inf")), trt.ERR_ARG),
    (dict(alpha=float("nan")), trt.ERR_ARG), (dict(alpha=float("-inf")), trt.ERR_ARG),
]


@pytest.mark.parametrize("kw,code", COMMON + [
    (dict(r=0), trt.ERR_NULL), (dict(y=0), trt.ERR_NULL), (dict(r_out=0), trt.ERR_NULL),
    (dict(ldr=0), trt.ERR_STRIDE), (dict(ldy=0), trt.ERR_STRIDE), (dict(ldro=63), trt.ERR_STRIDE), (dict(ldh=63), trt.ERR_STRIDE),
    (dict(r=BASE + 1), trt.ERR_ALIGN), (dict(h=BASE * 4 + 1), trt.ERR_ALIGN),
    (dict(r_out=BASE), trt.ERR_OVERLAP), (dict(h=BASE), trt.ERR_OVERLAP), (dict(h=BASE * 3), trt.ERR_OVERLAP),
    (dict(h=BASE * 2 + 1022), trt.ERR_OVERLAP), (dict(r_out=BASE * 10 + 2 * 128), trt.ERR_OVERLAP), (dict(h=BASE * 14), trt.ERR_OVERLAP),
    (dict(cols=16385, ldr=20000, ldy=20000, ldro=20000, ldh=20000), trt.ERR_UNSUPPORTED),
    (dict(dtype=trt.F32, gate_dtype=trt.F32, cols=8193, ldr=9000, ldy=9000, ldro=9000, ldh=9000), trt.ERR_UNSUPPORTED),
    (dict(rows=1 << 30, ldr=1 << 60), trt.ERR_SIZE),
])
def test_forward_refusals(kw, code):
    assert forward(**dict(kw)) == code
    assert trt.last_error() != ""


@pytest.mark.parametrize("kw,code", COMMON + [
    (dict(no_grads=True), trt.ERR_NULL), (dict(no_y=True), trt.ERR_NULL), (dict(y=0), trt.ERR_NULL), (dict(r=0), trt.ERR_NULL),
    (dict(dr=0), trt.ERR_NULL), (dict(dy=0), trt.ERR_NULL), (dict(dh=0, dro=0), trt.ERR_NULL), (dict(dh=0), trt.ERR_NULL),
    (dict(dh=0, dg=0), trt.ERR_NULL), (dict(gate=0), trt.ERR_NULL), (dict(ws=0), trt.ERR_NULL),
    (dict(wsb=3 * 4 * 64 * 4 - 1), trt.ERR_SIZE), (dict(wsb=-1), trt.ERR_SIZE), (dict(ws=BASE * 30 + 8), trt.ERR_ALIGN),
    (dict(post=0, post_gamma=0, post_beta=0), trt.ERR_ARG), (dict(post=0, post_gamma=0, post_beta=0, dpg=0), trt.ERR_ARG),
    (dict(lddh=0), trt.ERR_STRIDE), (dict(lddr=63), trt.ERR_STRIDE), (dict(lddy=63), trt.ERR_STRIDE), (dict(lddg=63), trt.ERR_STRIDE),
    (dict(ldr=0), trt.ERR_STRIDE), (dict(rs=BASE * 8, ys=BASE * 7, yls=0), trt.ERR_STRIDE),
    (dict(rs=BASE * 8), trt.ERR_ARG), (dict(ys=BASE * 8), trt.ERR_ARG),          # one of them in 8 bits
    (dict(dh=BASE + 1), trt.ERR_ALIGN), (dict(r=BASE * 3 + 1), trt.ERR_ALIGN), (dict(dgate=BASE * 20 + 1), trt.ERR_ALIGN),
    (dict(dr=BASE), trt.ERR_OVERLAP), (dict(dy=BASE * 2), trt.ERR_OVERLAP), (dict(dr=BASE * 3), trt.ERR_OVERLAP),
    (dict(dy=BASE * 4), trt.ERR_OVERLAP), (dict(dy=BASE * 5), trt.ERR_OVERLAP), (dict(dgate=BASE * 10), trt.ERR_OVERLAP),
    (dict(dpg=BASE * 11), trt.ERR_OVERLAP), (dict(db=BASE * 23), trt.ERR_OVERLAP), (dict(ws=BASE * 2), trt.ERR_OVERLAP),
    (dict(rs=BASE * 7, ys=BASE * 8, dy=BASE * 7), trt.ERR_OVERLAP), (dict(rs=BASE * 8, ys=BASE * 7, dr=BASE * 7 - 2), trt.ERR_OVERLAP),
    (dict(cols=16385, lddh=20000, lddro=20000, ldr=20000, ldy=20000, lddr=20000, lddy=20000, lddg=20000), trt.ERR_UNSUPPORTED),
    (dict(rows=1 << 24, rows_per_gate=2), trt.ERR_SIZE),
])
def test_backward_refusals(kw, code):
    assert backward(**dict(kw)) == code
    assert trt.last_error() != ""


def test_an_8_bit_row_needs_no_alignment():
    # (refused later, for the overlap, so that nothing is launched)
    assert backward(rs=BASE * 7 + 1, ys=BASE * 8 + 1, r=BASE * 3 + 1, dr=BASE) == trt.ERR_OVERLAP


def test_workspace_size():
    size = trt.block_norm_bwd_workspace_size
    for dt in (trt.F16, trt.BF16, trt.F32):
        for rows, cols, span in ((1, 1, 0), (7, 500, 3), (100000, 4096, 0), (100000, 4096, 1), (100000, 4096, 700),
                                 (1 << 30, 8, 0), (1 << 30, 8, 1), (5000, 64, 2)):
            n = size(rows, cols, span, dt)
            groups = -(-rows // span) if span > 1 else 1
            assert n % (16 * cols) == 0 and n // (16 * cols) % groups == 0
            assert groups <= n // (16 * cols) <= max(groups, min(rows, 1024))
    for bad in ((0, 4, 0, trt.F16), (4, 0, 0, trt.F16), (4, 4, -1, trt.F16), (4, 4, 0, 7), (4, 16385, 0, trt.F16),
                (1 << 30, 8, 2, trt.F16)):
        with pytest.raises(trt.TrtError):
            size(*bad)


def test_binding_refuses_what_it_cannot_pass():
    x = torch.zeros(4, 6, 8)
    q, s = torch.zeros(4, 6, 8, dtype=torch.int8), torch.zeros(4, 6, 1, dtype=torch.uint8)

    def refused(code, call, *a, **kw):
        with pytest.raises(trt.TrtError) as e:
            call(*a, **kw)
        assert e.value.status == code, e.value

    refused(trt.ERR_ARG, trt.block_norm, x, x)                                 # not on a GPU
    refused(trt.ERR_SIZE, trt.block_norm, x, x[:3])
    refused(trt.ERR_SIZE, trt.block_norm, x, x.half())
    refused(trt.ERR_STRIDE, trt.block_norm, x.transpose(0, 1), x.transpose(0, 1))
    refused(trt.ERR_SIZE, trt.block_norm, x, x, gamma=torch.ones(7))
    refused(trt.ERR_DTYPE, trt.block_norm, x, x, gamma=torch.ones(8), beta=torch.ones(8).half())
    refused(trt.ERR_ARG, trt.block_norm, x, x, need_h=False, h=x)
    refused(trt.ERR_ARG, trt.block_norm, x, x, rows_per_gate=2)
    # a gate that torch would broadcast over leading sizes, or not at all
    for shape in ((6, 8), (1, 6, 8), (4, 6, 1), (4, 1, 7), (3, 1, 8), (24, 8), (1,)):
        refused(trt.ERR_SIZE, trt.block_norm, x, x, torch.zeros(shape))
    refused(trt.ERR_SIZE, trt.block_norm, x, x, torch.zeros(4, 8), rows_per_gate=5)
    refused(trt.ERR_SIZE, trt.block_norm, x, x, torch.zeros(4, 8), rows_per_gate=0)
    for shape in ((8,), (4, 1, 8), (1, 1, 8), (4, 6, 8)):                      # taken, up to the device's check
        refused(trt.ERR_ARG, trt.block_norm, x, x, torch.zeros(shape))
    refused(trt.ERR_ARG, trt.block_norm, x, x, torch.zeros(5, 8), rows_per_gate=5)
    refused(trt.ERR_NULL, trt.block_norm_bwd, None, None, x, x)
    refused(trt.ERR_NULL, trt.block_norm_bwd, x, None, None, x)
    refused(trt.ERR_SIZE, trt.block_norm_bwd, x, x[:3], x, x)
    refused(trt.ERR_SIZE, trt.block_norm_bwd, x, x, x, x.half())
    refused(trt.ERR_SIZE, trt.block_norm_bwd, x, x, (q, s[:, :5]), x)
    refused(trt.ERR_SIZE, trt.block_norm_bwd, x, x, x, (q[:3], s[:3]))
    refused(trt.ERR_DTYPE, trt.block_norm_bwd, x, x, x, (q, s.to(torch.int8)))
    refused(trt.ERR_ARG, trt.block_norm_bwd, x, x, (q, s), (q, s))


def test_gate_spans():
    span = trt._gate_span
    x = torch.zeros(4, 6, 8)
    assert span(torch.zeros(8), x.shape, 24, 8, None) == 24
    assert span(torch.zeros(4, 1, 8), x.shape, 24, 8, None) == 6
    assert span(torch.zeros(1, 1, 8), x.shape, 24, 8, None) == 24
    assert span(torch.zeros(4, 6, 8), x.shape, 24, 8, None) == 1
    assert span(torch.zeros(5, 8), x.shape, 24, 8, 5) == 5
    assert span(torch.zeros(1, 8), torch.zeros(1, 8).shape, 1, 8, None) == 1


@pytest.mark.parametrize("rms", [False, True])
@pytest.mark.parametrize("post", [False, True])
def test_oracle_gradients_against_differences(rms, post):
    rng = np.random.default_rng(1)
    rows, cols, alpha, eps = 3, 7, 1.7, 1e-3
    v = {k: rng.normal(size=(rows, cols)) for k in ("r", "y", "gate", "dh", "dr")}
    v.update({k: rng.normal(size=cols) for k in (("pg", "pb") if post else ()) + ("g", "b")})

    def L(v):
        out, h = blocknorm_ref.forward(v["r"], v["y"], v["gate"], v.get("pg"), v.get("pb"), v["g"], v["b"], alpha, eps, rms, post)
        return (v["dr"] * out + v["dh"] * h).sum()

    out, _ = blocknorm_ref.forward(v["r"], v["y"], v["gate"], v.get("pg"), v.get("pb"), v["g"], v["b"], alpha, eps, rms, post)
    got = blocknorm_ref.backward(v["dh"], v["dr"], out, v["y"], v["gate"], v.get("pg"), v.get("pb"), v["g"], alpha, eps, rms, post)
    step = 1e-6
    for name, grad in (("r", "dr"), ("y", "dy"), ("gate", "dgate"), ("pg", "dpg"), ("pb", "dpb"), ("g", "dg"), ("b", "db")):
        if name not in v:
            continue
        for at in np.ndindex(v[name].shape):
            up, down = dict(v), dict(v)
            up[name], down[name] = v[name].copy(), v[name].copy()
            up[name][at] += step
            down[name][at] -= step
            assert abs((L(up) - L(down)) / (2 * step) - got[grad][at]) < 1e-6, (name, at)
