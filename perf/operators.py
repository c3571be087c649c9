"""The measured cases of the layer norm and linear cross entropy operators.

Four operators, the last stretch of a training step and the first of its
backward pass: the layer norm in front of a vocabulary head, its gradients,
the head's product with its softmax cross entropy (the logits are never
stored), and the gradients of that.  Each case names one operator, its sizes
and its types; run() makes one pass, in plain torch operations or, with own
set, through the package's calls.
"""
import math

import torch

own = False

IGNORE = -100
EPS = 1e-5
DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
BYTES = {"bf16": 2, "f16": 2, "f32": 4}


def listed():
    return [
        # one token of a decoding step, in front of the head: latency only
        {"name": "norm-one-token", "op": "norm", "rows": 1, "cols": 4096, "pad": 0, "dtype": "bf16", "params": "bf16"},
        # odd rows in a padded buffer, as a slice of a fused activation is
        {"name": "norm-ragged", "op": "norm", "rows": 4000, "cols": 5000, "pad": 64, "dtype": "f16", "params": "f16"},
        # a training batch: 8 sequences of 2048 tokens
        {"name": "norm-batch", "op": "norm", "rows": 16384, "cols": 8192, "pad": 0, "dtype": "bf16", "params": "f32"},
        # one short sequence of a small model
        {"name": "norm-grad-short", "op": "norm_grad", "rows": 128, "cols": 1024, "pad": 0, "dtype": "f16", "params": "f32"},
        # binary32 activations of an odd width
        {"name": "norm-grad-odd", "op": "norm_grad", "rows": 4001, "cols": 1023, "pad": 0, "dtype": "f32", "params": "f32"},
        # the training batch's backward pass
        {"name": "norm-grad-batch", "op": "norm_grad", "rows": 16384, "cols": 8192, "pad": 0, "dtype": "bf16", "params": "f32"},
        # the score of one token, as a server asks for it: reads the head once
        {"name": "xent-one-token", "op": "xent", "tokens": 1, "vocab": 65536, "width": 4096, "dtype": "bf16", "ignored": 0.0},
        # an odd vocabulary and a ragged batch, a third of it prompt
        {"name": "xent-ragged", "op": "xent", "tokens": 4000, "vocab": 50001, "width": 2048, "dtype": "f16", "ignored": 0.33},
        # a training batch over a large vocabulary
        {"name": "xent-batch", "op": "xent", "tokens": 8192, "vocab": 131072, "width": 4096, "dtype": "bf16", "ignored": 0.0},
        # a few tokens of a small model, weighted one by one
        {"name": "xent-grad-short", "op": "xent_grad", "tokens": 77, "vocab": 16384, "width": 1024, "dtype": "bf16", "ignored": 0.0, "weights": "each"},
        # fine-tuning: half of the batch is prompt and carries no loss
        {"name": "xent-grad-ragged", "op": "xent_grad", "tokens": 4097, "vocab": 32003, "width": 2560, "dtype": "f16", "ignored": 0.5, "weights": "mean"},
        # the training batch's backward pass
        {"name": "xent-grad-batch", "op": "xent_grad", "tokens": 8192, "vocab": 131072, "width": 4096, "dtype": "bf16", "ignored": 0.0, "weights": "mean"},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "norm_grad", "xent", "xent_grad"])
    if op in ("norm", "norm_grad"):
        # widths of small to large models, mostly of whole 8s; rows from one
        # token to a large batch, no more elements than the largest listed
        cols = _log(rng, 64, 16384)
        if rng.random() < 0.7:
            cols = max(8, cols // 8 * 8)
        rows = min(_log(rng, 1, 65536), (1 << 27) // cols)
        return {"op": op, "rows": rows, "cols": cols, "pad": rng.choice([0, 0, 0, 8, 24]),
                "dtype": rng.choice(["bf16", "f16", "f32"]), "params": rng.choice(["same", "f32"])}
    # head widths of whole 64s; any vocabulary
    width = 64 * _log(rng, 4, 64)
    vocab = _log(rng, 1000, 131072)
    tokens = _log(rng, 1, 8192)
    case = {"op": op, "tokens": tokens, "vocab": vocab, "width": width, "dtype": rng.choice(["bf16", "f16"]),
            "ignored": rng.choice([0.0, 0.0, 0.1, 0.5])}
    if op == "xent_grad":
        case["weights"] = rng.choice(["mean", "mean", "each", "z"])
    return case


# ---- inputs -----------------------------------------------------------------------

def _generator(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _param_dtype(case):
    return DTYPES[case["dtype"] if case["params"] == "same" else case["params"]]


def _norm_inputs(case, seed):
    """Activations as a residual stream has them: rows of different scales and
    means, some channels much larger than the others."""
    g = _generator(seed)
    rows, cols, dt = case["rows"], case["cols"], DTYPES[case["dtype"]]

    def normal(*shape):
        return torch.randn(*shape, generator=g, device="cuda")

    x = torch.zeros(rows, cols + case["pad"], device="cuda", dtype=dt)[:, :cols]
    channel = torch.exp(0.5 * normal(cols))
    x.copy_((normal(rows, cols) * channel + 0.5 * normal(cols)) * torch.exp(0.5 * normal(rows, 1)) + 0.3 * normal(rows, 1))
    s = {"op": case["op"], "x": x, "gamma": (1 + 0.2 * normal(cols)).to(_param_dtype(case))}
    if case["op"] == "norm":
        s["beta"] = (0.1 * normal(cols)).to(_param_dtype(case))
    else:
        dy = torch.zeros(rows, cols + case["pad"], device="cuda", dtype=dt)[:, :cols]
        dy.copy_(normal(rows, cols) * torch.exp(0.5 * normal(rows, 1)))
        s["dy"] = dy
    return s


def _xent_inputs(case, seed):
    """Normalised activations that lean towards the head's row of their target
    by a different amount each, so that the targets' probabilities run from
    that of chance to near one."""
    g = _generator(seed)
    T, V, D, dt = case["tokens"], case["vocab"], case["width"], DTYPES[case["dtype"]]
    w = torch.randn(V, D, generator=g, device="cuda") * (2 / math.sqrt(D))
    target = torch.randint(0, V, (T,), generator=g, device="cuda")
    x = torch.randn(T, D, generator=g, device="cuda")
    x += w[target] * torch.rand(T, 1, generator=g, device="cuda") * 5
    drop = torch.rand(T, generator=g, device="cuda") < case["ignored"]
    each = torch.rand(T, generator=g, device="cuda") + 0.5
    s = {"op": case["op"], "x": x.to(dt), "w": w.to(dt), "target": torch.where(drop, IGNORE, target)}
    if case["op"] == "xent_grad":
        # what the forward pass and the loss's reduction leave behind
        _, s["lse"] = _plain_xent(s)
        counts = (~drop).float()
        s["dloss"] = counts / counts.sum().clamp(min=1) * (each if case["weights"] == "each" else 1)
        # an auxiliary loss on the log-sum-exp: its own gradient
        s["dlse"] = 2e-4 * s["lse"] * s["dloss"] if case["weights"] == "z" else None
    return s


def prepare(case, seed):
    return _norm_inputs(case, seed) if case["op"].startswith("norm") else _xent_inputs(case, seed)


# ---- the plain forms ----------------------------------------------------------------

def _plain_norm(s):
    x = s["x"].float()
    d = x - x.mean(1, keepdim=True)
    rstd = torch.rsqrt((d * d).mean(1, keepdim=True) + EPS)
    return (d * rstd * s["gamma"].float() + s["beta"].float()).to(s["x"].dtype)


def _plain_norm_grad(s):
    x, dy = s["x"].float(), s["dy"].float()
    d = x - x.mean(1, keepdim=True)
    rstd = torch.rsqrt((d * d).mean(1, keepdim=True) + EPS)
    xhat = d * rstd
    u = dy * s["gamma"].float()
    dx = rstd * (u - u.mean(1, keepdim=True) - xhat * (u * xhat).mean(1, keepdim=True))
    dgamma, dbeta = (dy * xhat).sum(0), dy.sum(0)
    return dx.to(s["x"].dtype), dgamma.to(s["gamma"].dtype), dbeta.to(s["gamma"].dtype)


def _plain_xent(s):
    z = s["x"].float() @ s["w"].float().t()
    keep = s["target"] != IGNORE
    m = z.amax(1)
    total = torch.exp(z - m[:, None]).sum(1)
    at = z.gather(1, torch.where(keep, s["target"], 0)[:, None])[:, 0]
    loss = (m - at) + torch.log(total)
    return torch.where(keep, loss, 0.0), torch.where(keep, m + torch.log(total), 0.0)


def _plain_xent_grad(s):
    x, w = s["x"].float(), s["w"].float()
    keep = s["target"] != IGNORE
    dloss = torch.where(keep, s["dloss"], 0.0)
    both = dloss if s["dlse"] is None else dloss + torch.where(keep, s["dlse"], 0.0)
    g = torch.exp(x @ w.t() - s["lse"][:, None]) * both[:, None]
    g = torch.where(keep[:, None], g, 0.0)
    g.scatter_add_(1, torch.where(keep, s["target"], 0)[:, None], -dloss[:, None])
    return (g @ w).to(s["x"].dtype), (g.t() @ x).to(s["w"].dtype)


def _own_call(s):
    import thread_register_tile_amd as trt
    if s["op"] == "norm":
        return trt.layernorm(s["x"], s["gamma"], s["beta"], eps=EPS)
    if s["op"] == "norm_grad":
        return trt.layernorm_bwd(s["dy"], s["x"], s["gamma"], eps=EPS)
    if s["op"] == "xent":
        return trt.linear_xent(s["x"], s["w"], s["target"], ignore_index=IGNORE)
    return trt.linear_xent_bwd(s["x"], s["w"], s["target"], s["lse"], s["dloss"], s["dlse"], ignore_index=IGNORE)


def run(state):
    if own:
        return _own_call(state)
    return {"norm": _plain_norm, "norm_grad": _plain_norm_grad, "xent": _plain_xent,
            "xent_grad": _plain_xent_grad}[state["op"]](state)


def work(case):
    if case["op"].startswith("norm"):
        n, e = case["rows"] * case["cols"], BYTES[case["dtype"]]
        p = case["cols"] * BYTES[case["dtype"] if case["params"] == "same" else case["params"]]
        if case["op"] == "norm":
            return {"bytes": 2 * n * e + 2 * p, "flops": 8 * n}
        return {"bytes": 3 * n * e + 3 * p, "flops": 16 * n}
    # tokens without a loss take no part in any product
    T, V, D, e = case["tokens"], case["vocab"], case["width"], BYTES[case["dtype"]]
    live = max(1, round(T * (1 - case["ignored"])))
    product = 2 * live * V * D
    if case["op"] == "xent":
        return {"bytes": (live + V) * D * e + 16 * T, "flops": product}
    # the logits are not kept: one product for them again, one for each gradient
    return {"bytes": (live + V + T + V) * D * e + 16 * T, "flops": 3 * product}


# ---- 64-bit values, from the definitions ---------------------------------------------

def _exact_norm(s, grad):
    x = s["x"].double()
    n = x.shape[1]
    mu = x.sum(1, keepdim=True).div(n)
    sigma = ((x - mu).pow(2).sum(1, keepdim=True).div(n) + EPS).sqrt()
    h = (x - mu).div(sigma)
    if not grad:
        return h.mul(s["gamma"].double()).add(s["beta"].double())
    dy = s["dy"].double()
    # y = gamma h + beta, h = (x - mu) / sigma: the Jacobian of h takes the
    # components of dh along 1 and along h out, and divides by sigma
    dh = dy.mul(s["gamma"].double())
    dx = dh.sub(dh.sum(1, keepdim=True).div(n)).sub(h.mul(dh.mul(h).sum(1, keepdim=True).div(n))).div(sigma)
    return dx, dy.mul(h).sum(0), dy.sum(0)


def _exact_xent(s, grad):
    """In blocks of rows, so that the 64-bit probabilities stay small."""
    x, w, target = s["x"].double(), s["w"].double(), s["target"]
    T, V = x.shape[0], w.shape[0]
    loss, lse = torch.zeros(T, device="cuda", dtype=torch.float64), torch.zeros(T, device="cuda", dtype=torch.float64)
    dx, dw = torch.zeros_like(x), torch.zeros_like(w) if grad else None
    live = (target != IGNORE).nonzero()[:, 0]
    for rows in live.split(1024):
        z = torch.mm(x[rows], w.t())
        norm = torch.logsumexp(z, 1)
        at = target[rows]
        # -log of the softmax at the target, without the cancellation of two large numbers
        others = z - z[torch.arange(len(rows), device="cuda"), at][:, None]
        loss[rows], lse[rows] = torch.logsumexp(others, 1), norm
        if grad:
            up = s["dloss"][rows].double()[:, None]
            more = 0 if s["dlse"] is None else s["dlse"][rows].double()[:, None]
            p = torch.softmax(z, 1)
            dz = p.mul(up + more)
            dz[torch.arange(len(rows), device="cuda"), at] -= up[:, 0]
            dx[rows] = torch.mm(dz, w)
            dw += torch.mm(dz.t().contiguous(), x[rows])
    return (dx, dw) if grad else (loss, lse)


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"].startswith("norm"):
        return _exact_norm(s, case["op"] == "norm_grad")
    return _exact_xent(s, case["op"] == "xent_grad")
