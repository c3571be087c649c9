"""CPU tests of the linear cross entropy's entry points: refusals before any HIP
call, workspace sizes, and the oracle's gradients against differences."""
import numpy as np
import pytest
import torch

import thread_register_tile_amd as trt
from oracle import xent_ref

BASE = 1 << 32     # fake, well-separated addresses: never dereferenced


def forward(**kw):
    a = dict(T=64, V=512, D=32, x=BASE, ldx=32, w=BASE * 2, ldw=32, target=BASE * 3, ignore=-100, loss=BASE * 4,
             lse=BASE * 5, dtype=trt.BF16, ws=BASE * 6, wsb=1 << 30)
    a.update(kw)
    return trt.lib().trt_linear_xent(a["T"], a["V"], a["D"], a["x"], a["ldx"], a["w"], a["ldw"], a["target"],
                                     a["ignore"], a["loss"], a["lse"], a["dtype"], a["ws"], a["wsb"], None)


def backward(**kw):
    a = dict(T=64, V=512, D=32, x=BASE, ldx=32, w=BASE * 2, ldw=32, target=BASE * 3, ignore=-100, lse=BASE * 4,
             dloss=BASE * 5, inc=1, dlse=BASE * 6, inc2=1, dx=BASE * 7, lddx=32, dw=BASE * 8, lddw=32, dtype=trt.BF16,
             odt=trt.F32, piece=0, ws=BASE * 9, wsb=1 << 30)
    a.update(kw)
    return trt.lib().trt_linear_xent_bwd(a["T"], a["V"], a["D"], a["x"], a["ldx"], a["w"], a["ldw"], a["target"],
                                         a["ignore"], a["lse"], a["dloss"], a["inc"], a["dlse"], a["inc2"], a["dx"],
                                         a["lddx"], a["dw"], a["lddw"], a["dtype"], a["odt"], a["piece"], a["ws"],
                                         a["wsb"], None)


SHARED = [
    (dict(T=0), trt.ERR_SIZE), (dict(V=0), trt.ERR_SIZE), (dict(D=0), trt.ERR_SIZE), (dict(T=-3), trt.ERR_SIZE),
    (dict(T=(1 << 23) + 1), trt.ERR_SIZE), (dict(V=(1 << 30) + 1), trt.ERR_SIZE),
    (dict(D=(1 << 20) + 1, ldx=1 << 21, ldw=1 << 21), trt.ERR_SIZE), (dict(T=1 << 23, V=1 << 20), trt.ERR_SIZE),
    (dict(dtype=trt.F32), trt.ERR_DTYPE), (dict(dtype=0), trt.ERR_DTYPE),
    (dict(x=0), trt.ERR_NULL), (dict(w=0), trt.ERR_NULL), (dict(target=0), trt.ERR_NULL), (dict(lse=0), trt.ERR_NULL),
    (dict(ldx=31), trt.ERR_STRIDE), (dict(ldw=31), trt.ERR_STRIDE),
    (dict(ws=0), trt.ERR_NULL), (dict(wsb=1000), trt.ERR_SIZE), (dict(wsb=-1), trt.ERR_SIZE),
    (dict(x=BASE + 1), trt.ERR_ALIGN), (dict(w=BASE * 2 + 1), trt.ERR_ALIGN), (dict(target=BASE * 3 + 4), trt.ERR_ALIGN),
    (dict(ws=BASE), trt.ERR_OVERLAP), (dict(ws=BASE * 2), trt.ERR_OVERLAP), (dict(ws=BASE * 3), trt.ERR_OVERLAP),
    (dict(ldx=1 << 61), trt.ERR_SIZE),
]


@pytest.mark.parametrize("kw,code", SHARED + [
    (dict(loss=0), trt.ERR_NULL), (dict(loss=BASE * 4 + 2), trt.ERR_ALIGN), (dict(ws=BASE * 6 + 4), trt.ERR_ALIGN),
    (dict(lse=BASE * 4 + 4), trt.ERR_OVERLAP), (dict(loss=BASE * 3), trt.ERR_OVERLAP), (dict(lse=BASE), trt.ERR_OVERLAP),
    (dict(loss=BASE * 6), trt.ERR_OVERLAP),
])
def test_forward_refusals(kw, code):
    assert forward(**kw) == code
    assert trt.last_error() != ""


@pytest.mark.parametrize("kw,code", SHARED + [
    (dict(odt=0), trt.ERR_DTYPE), (dict(dx=0, dw=0), trt.ERR_NULL), (dict(dloss=0), trt.ERR_NULL),
    (dict(inc=-1), trt.ERR_STRIDE), (dict(inc2=-1), trt.ERR_STRIDE), (dict(lddx=31), trt.ERR_STRIDE),
    (dict(lddw=31), trt.ERR_STRIDE), (dict(piece=-64), trt.ERR_ARG), (dict(piece=100), trt.ERR_ARG),
    (dict(piece=(1 << 20) + 64), trt.ERR_ARG), (dict(ws=BASE * 9 + 4), trt.ERR_ALIGN),
    (dict(dx=BASE * 7 + 2), trt.ERR_ALIGN), (dict(lse=BASE * 4 + 2), trt.ERR_ALIGN), (dict(dloss=BASE * 5 + 1), trt.ERR_ALIGN),
    (dict(dx=BASE), trt.ERR_OVERLAP), (dict(dw=BASE * 2), trt.ERR_OVERLAP), (dict(dw=BASE * 7), trt.ERR_OVERLAP),
    (dict(dx=BASE * 4), trt.ERR_OVERLAP), (dict(dx=BASE * 5), trt.ERR_OVERLAP), (dict(dx=BASE * 6), trt.ERR_OVERLAP),
    (dict(ws=BASE * 7), trt.ERR_OVERLAP), (dict(ws=BASE * 8), trt.ERR_OVERLAP),
])
def test_backward_refusals(kw, code):
    assert backward(**kw) == code
    assert trt.last_error() != ""


def test_workspace_sizes():
    assert trt.linear_xent_workspace_size(1, 1, 1) > 0
    # the pairs: 8 bytes for a token and 128 entries, nothing like the logits
    n = trt.linear_xent_workspace_size(8192, 131072, 4096)
    assert 8192 * 1024 * 8 <= n < 8192 * 1024 * 8 + (1 << 20)
    # one piece of G, X, and dX's sums, of which there are no more than 1024
    # tiles of 256x256
    small = trt.linear_xent_bwd_workspace_size(8192, 131072, 4096, 8192)
    base = 8192 * 8192 * 2 + 8192 * 4096 * 2
    assert base + 8192 * 4096 * 4 <= small < base + 1024 * 65536 * 4 + (1 << 20)
    assert trt.linear_xent_bwd_workspace_size(8192, 131072, 4096) > small
    # a piece beyond the vocabulary is the vocabulary
    assert trt.linear_xent_bwd_workspace_size(10, 100, 8, 128) == trt.linear_xent_bwd_workspace_size(10, 100, 8, 1 << 20)
    for bad in ((0, 1, 1), (1, 0, 1), (1, 1, 0), (1 << 24, 1, 1)):
        with pytest.raises(trt.TrtError):
            trt.linear_xent_workspace_size(*bad)
        with pytest.raises(trt.TrtError):
            trt.linear_xent_bwd_workspace_size(*bad)
    with pytest.raises(trt.TrtError):
        trt.linear_xent_bwd_workspace_size(1, 1, 1, 65)


def test_binding_refuses_what_it_cannot_pass():
    x, w = torch.zeros(4, 8, dtype=torch.bfloat16), torch.zeros(10, 8, dtype=torch.bfloat16)
    t, f = torch.zeros(4, dtype=torch.int64), torch.zeros(4)

    def status(call):
        with pytest.raises(trt.TrtError) as e:
            call()
        return e.value.status

    assert status(lambda: trt.linear_xent(x, w, t)) == trt.ERR_ARG                     # not on a GPU
    assert status(lambda: trt.linear_xent(x, w[:, :7], t)) == trt.ERR_SIZE
    assert status(lambda: trt.linear_xent(x, w.half(), t)) == trt.ERR_DTYPE
    assert status(lambda: trt.linear_xent(x, w, t.int())) == trt.ERR_DTYPE
    assert status(lambda: trt.linear_xent(x, w, t[:3])) == trt.ERR_SIZE
    assert status(lambda: trt.linear_xent(x, w.t().contiguous().t(), t)) == trt.ERR_STRIDE
    assert status(lambda: trt.linear_xent(x, w, t, loss=f.double())) == trt.ERR_SIZE
    assert status(lambda: trt.linear_xent_bwd(x, w, t, f[:3], f)) == trt.ERR_SIZE
    assert status(lambda: trt.linear_xent_bwd(x, w, t, f, f.double())) == trt.ERR_DTYPE
    assert status(lambda: trt.linear_xent_bwd(x, w, t, f, f[:3])) == trt.ERR_SIZE
    assert status(lambda: trt.linear_xent_bwd(x, w, t, f, None)) == trt.ERR_NULL
    assert status(lambda: trt.linear_xent_bwd(x, w, t, f, f, dx=torch.zeros(4, 8), dw=w.clone())) == trt.ERR_SIZE
    assert status(lambda: trt.linear_xent_bwd(x, w, t, f, f, piece=7)) == trt.ERR_ARG
    assert status(lambda: trt.linear_xent(x[:1].expand(4, 8), w, t)) == trt.ERR_STRIDE


def test_oracle_gradients_against_differences():
    rng = np.random.default_rng(1)
    x, w = rng.normal(size=(5, 6)), rng.normal(size=(9, 6))
    target = np.array([0, 8, -100, 3, 3])
    up, ue = rng.normal(size=5), rng.normal(size=5)
    dx, dw = xent_ref.backward(x, w, target, up, ue)
    assert (dx[2] == 0).all()
    step = 1e-6

    def L(x, w):
        loss, lse = xent_ref.forward(x, w, target)
        return (up * loss + ue * lse).sum()

    for a, da, f in ((x, dx, lambda e: L(x + e, w) - L(x - e, w)), (w, dw, lambda e: L(x, w + e) - L(x, w - e))):
        for i in range(a.shape[0]):
            for j in range(a.shape[1]):
                e = np.zeros_like(a)
                e[i, j] = step
                assert abs(f(e) / (2 * step) - da[i, j]) < 1e-7


def test_oracle_matches_torch():
    rng = np.random.default_rng(2)
    x, w = rng.normal(size=(7, 5)), rng.normal(size=(11, 5))
    target = np.array([0, 1, 10, -100, 4, 4, 9])
    loss, lse = xent_ref.forward(x, w, target)
    z = torch.from_numpy(x) @ torch.from_numpy(w).t()
    want = torch.nn.functional.cross_entropy(z, torch.from_numpy(target), reduction="none")
    live = target != -100
    assert np.allclose(loss, want.numpy(), atol=1e-12, rtol=0)
    assert np.allclose(lse[live], torch.logsumexp(z, 1).numpy()[live], atol=1e-12, rtol=0)
