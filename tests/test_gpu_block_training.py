"""A training step of a small residual model through the library's calls, with
its activations saved in 8 bits, against the same model in 64 bits.

Two blocks of one projection each between the norms, a vocabulary head behind
them.  Every stored tensor is rounded to bf16 once (half a step 2^-8 of an
element) and the saved ones to 8 bits (2^-7 of a block's largest element, under
2^-6 of a row's norm).  An error in an activation reaches a gradient through
factors near one, so a gradient collects the roundings of its path: at most 20
of 2^-8 and 4 of 2^-6, 0.14 of its norm; a gradient with a wrong term, factor or
row is off by its own size.
"""
import pytest
import torch

import thread_register_tile_amd as trt

pytestmark = pytest.mark.gpu

ROWS, COLS, VOCAB, SPAN, EPS, ALPHA = 300, 256, 640, 100, 1e-5, 1.25


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    trt.lib()


def model():
    gen = torch.Generator().manual_seed(11)

    def normal(*shape):
        return torch.randn(*shape, generator=gen, dtype=torch.float64)

    p = {"x": normal(ROWS, COLS), "head": normal(VOCAB, COLS) / 8}
    for i in (0, 1):
        p[f"w{i}"] = normal(COLS, COLS) / 16
        p[f"gate{i}"] = 0.7 + 0.3 * normal(-(-ROWS // SPAN), COLS)
        p[f"pg{i}"], p[f"g{i}"] = 1 + 0.2 * normal(COLS), 1 + 0.2 * normal(COLS)
        p[f"pb{i}"], p[f"b{i}"] = 0.1 * normal(COLS), 0.1 * normal(COLS)
    # what the kernels are given, in both
    p = {k: v.to(torch.bfloat16).double() for k, v in p.items()}
    return p, torch.randint(0, VOCAB, (ROWS,), generator=gen)


def reference(p, target, rms):
    p = {k: v.clone().requires_grad_() for k, v in p.items()}

    def norm(x):
        d = x if rms else x - x.mean(1, keepdim=True)
        return d / torch.sqrt((d * d).mean(1, keepdim=True) + EPS)

    r, h = p["x"], norm(p["x"])
    for i in (0, 1):
        u = norm(h @ p[f"w{i}"].t()) * p[f"pg{i}"] + p[f"pb{i}"]
        r = ALPHA * r + p[f"gate{i}"].repeat_interleave(SPAN, 0)[:ROWS] * u
        h = norm(r) * p[f"g{i}"] + p[f"b{i}"]
    loss = torch.nn.functional.cross_entropy(h @ p["head"].t(), target)
    loss.backward()
    return loss.item(), {k: v.grad for k, v in p.items()}


def step(p, target, rms):
    d = {k: v.to(torch.bfloat16).cuda() for k, v in p.items()}
    target = target.cuda()
    made = [dict(post_gamma=d[f"pg{i}"], post_beta=d[f"pb{i}"], gamma=d[f"g{i}"], alpha=ALPHA, rms=rms, eps=EPS, rows_per_gate=SPAN)
            for i in (0, 1)]
    # the first norm has nothing behind it: a block whose output is zero
    zero = torch.zeros_like(d["x"])
    r, h = trt.block_norm(d["x"], zero, post=False, rms=rms, eps=EPS)
    saved = []
    for i in (0, 1):
        y = trt.gemm(h, d[f"w{i}"], opB="T")
        packed = trt.act8_pack(h), trt.act8_pack(y)
        r, h = trt.block_norm(r, y, d[f"gate{i}"], beta=d[f"b{i}"], **made[i])
        saved.append((*packed, trt.act8_pack(r)))
    loss, lse = trt.linear_xent(h, d["head"], target)
    dh, dhead = trt.linear_xent_bwd(h, d["head"], target, lse, torch.full((1,), 1 / ROWS, device="cuda"))
    grads, dr = {"head": dhead}, None
    for i in (1, 0):
        h8, y8, r8 = saved[i]
        dr, dy, grads[f"gate{i}"], grads[f"pg{i}"], grads[f"pb{i}"], grads[f"g{i}"], grads[f"b{i}"] = trt.block_norm_bwd(
            dh, dr, r8, y8, d[f"gate{i}"], **made[i])
        grads[f"w{i}"] = trt.act8_weight_grad(dy, *h8)
        dh = trt.gemm(dy, d[f"w{i}"])
    grads["x"] = trt.block_norm_bwd(dh, dr, d["x"], zero, post=False, rms=rms, eps=EPS)[0]
    return loss.mean().item(), grads


@pytest.mark.parametrize("rms", [False, True])
def test_step(rms):
    p, target = model()
    want_loss, want = reference(p, target, rms)
    loss, got = step(p, target, rms)
    assert abs(loss - want_loss) < 0.02 * want_loss
    assert set(got) == set(want)
    off = {k: ((got[k].double().cpu() - want[k]).norm() / want[k].norm()).item() for k in want}
    print(off, flush=True)
    assert all(v < 0.14 for v in off.values()), off
