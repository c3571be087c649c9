"""GPU tests of the block norm and the 8-bit activations at their limits: more
gate rows than a launch would give workgroups, captured graphs that share a
workspace, two streams at once, and results that repeat bit for bit."""
import pytest
import torch

import thread_register_tile_amd as trt

pytestmark = pytest.mark.gpu

BF16 = torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    trt.lib()


def test_gate_rows_beyond_the_workgroups():
    """A gate row for every 9 of 9.6 million rows is read with each of them, as
    one for each row is: the same bits."""
    rows, cols, span = 9_600_000, 8, 9
    gen = torch.Generator(device="cuda").manual_seed(0)
    x, y = (torch.randn(rows, cols, device="cuda", generator=gen).to(BF16) for _ in range(2))
    gate = torch.randn(-(-rows // span), cols, device="cuda", generator=gen).to(BF16)
    a = trt.block_norm(x, y, gate, rows_per_gate=span)
    b = trt.block_norm(x, y, gate.repeat_interleave(span, 0)[:rows].contiguous())
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_gradients_of_many_gate_rows():
    """Two rows to each of 1.5 million gate rows: each gate row's gradient is the
    sum of two of those that a gate for each row has, which are rounded once to
    binary32 (the sums' own roundings, 4 of 2^-24 of the magnitudes, and theirs)."""
    rows, cols = 3_000_000, 4
    gen = torch.Generator(device="cuda").manual_seed(1)
    x, y, dh, dr = (torch.randn(rows, cols, device="cuda", generator=gen) for _ in range(4))
    gate = torch.randn(rows // 2, cols, device="cuda", generator=gen)
    got = trt.block_norm_bwd(dh, dr, x, y, gate, post=False, rows_per_gate=2)
    each = trt.block_norm_bwd(dh, dr, x, y, gate.repeat_interleave(2, 0), post=False)
    parts = each[2].double().view(-1, 2, cols)
    tol = 8 * 2.0 ** -24 * parts.abs().sum(1)
    assert ((got[2].double() - parts.sum(1)).abs() <= tol).all()
    assert torch.equal(got[0], each[0])


def step(x, y, dh, dr, gate, dy, ws, ws2):
    out, h = trt.block_norm(x, y, gate, rows_per_gate=50)
    back = trt.block_norm_bwd(dh, dr, trt.act8_pack(out), trt.act8_pack(y), gate, rows_per_gate=50, workspace=ws)
    return (out, h, *back, trt.act8_weight_grad(dy, *trt.act8_pack(h), workspace=ws2, out_dtype=torch.float32))


def inputs(seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    t = [torch.randn(1500, 520, device="cuda", generator=gen).to(BF16) for _ in range(4)]
    return (*t, torch.randn(30, 520, device="cuda", generator=gen).to(BF16),
            torch.randn(1500, 136, device="cuda", generator=gen).to(BF16))


def workspaces():
    return (torch.full((trt.block_norm_bwd_workspace_size(1500, 520, 50, trt.BF16),), 0xFF, dtype=torch.uint8, device="cuda"),
            torch.full((trt.act8_weight_grad_workspace_size(1500, 136, 520),), 0xFF, dtype=torch.uint8, device="cuda"))


def same(a, b):
    return all(torch.equal(p, q) for p, q in zip(a, b))


def test_results_repeat():
    """Bit for bit, whatever the workspaces hold."""
    i = inputs(2)
    first = step(*i, *workspaces())
    for fill in (0x00, 0x7F):
        ws = [w.fill_(fill) for w in workspaces()]
        assert same(first, step(*i, *ws))


def test_two_graphs_share_workspaces():
    """Captured on inputs of their own and replayed one after the other, in both
    orders, with eager work of the same workspaces between."""
    ws = workspaces()
    sets, graphs, outs = [inputs(3), inputs(4)], [], []
    want = [step(*i, *workspaces()) for i in sets]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(*sets[0], *ws)
    torch.cuda.synchronize()
    for i in sets:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=side):
            outs.append(step(*i, *ws))
        graphs.append(g)
    for order in ((0, 1), (1, 0), (0, 1)):
        for k in order:
            for t in outs[k]:
                t.zero_()
            graphs[k].replay()
            torch.cuda.synchronize()
            assert same(outs[k], want[k])
            assert same(step(*sets[1 - k], *ws), want[1 - k])
            torch.cuda.synchronize()


def test_two_streams_at_once():
    sets = [inputs(5), inputs(6)]
    want = [step(*i, *workspaces()) for i in sets]
    ws = [workspaces(), workspaces()]
    torch.cuda.synchronize()
    streams, got = [torch.cuda.Stream(), torch.cuda.Stream()], [[], []]
    for _ in range(5):
        for k in (0, 1):
            with torch.cuda.stream(streams[k]):
                got[k].append(step(*sets[k], *ws[k]))
    torch.cuda.synchronize()
    for k in (0, 1):
        assert all(same(g, want[k]) for g in got[k])


def test_gradients_against_differences():
    """Central differences of the forward pass in binary32 for a sum of all its
    results with fixed weights, in directions drawn at random.  With a step of
    2^-6 of unit directions the third derivative leaves about 2^-12 of the
    gradient, and each of the rows * cols binary32 results a rounding: 1e-2 of
    the derivative holds both with room."""
    gen = torch.Generator(device="cuda").manual_seed(7)
    rows, cols = 12, 96

    def normal(*shape):
        return torch.randn(*shape, device="cuda", generator=gen)

    for rms in (False, True):
        for post in (False, True):
            v = {"r": normal(rows, cols), "y": normal(rows, cols), "gate": normal(3, cols), "gamma": 1 + 0.2 * normal(cols),
                 "beta": 0.2 * normal(cols)}
            if post:
                v["post_gamma"], v["post_beta"] = 1 + 0.2 * normal(cols), 0.2 * normal(cols)
            a, b = normal(rows, cols), normal(rows, cols)

            def loss(v):
                out, h = trt.block_norm(v["r"], v["y"], v["gate"], rows_per_gate=4, post=post, rms=rms, alpha=1.5,
                                        **{k: v[k] for k in v if k not in ("r", "y", "gate")})
                return (out.double() * a).sum() + (h.double() * b).sum()

            out, _ = trt.block_norm(v["r"], v["y"], v["gate"], rows_per_gate=4, post=post, rms=rms, alpha=1.5,
                                    **{k: v[k] for k in v if k not in ("r", "y", "gate")})
            got = trt.block_norm_bwd(b, a, out, v["y"], v["gate"], rows_per_gate=4, post=post, rms=rms, alpha=1.5,
                                     **{k: v[k] for k in v if k not in ("r", "y", "gate", "beta")})
            names = ("r", "y", "gate", "post_gamma", "post_beta", "gamma", "beta")
            for name, g in zip(names, got):
                if g is None:
                    continue
                d = normal(*v[name].shape)
                d /= d.norm()
                step_ = 2.0 ** -6
                up, down = ({**v, name: v[name] + sign * step_ * d} for sign in (1, -1))
                fd = ((loss(up) - loss(down)) / (2 * step_)).item()
                an = (g.double() * d).sum().item()
                assert abs(fd - an) <= 1e-2 * max(abs(an), g.norm().item() / g.numel() ** 0.5), (name, rms, post, fd, an)


@pytest.mark.parametrize("cols", [5, 520, 1500, 2056, 8200, 16384])
@pytest.mark.parametrize("rms", [False, True])
@pytest.mark.parametrize("bits", [8, 16])
def test_output_that_is_not_finite_without_its_norm(cols, rms, bits):
    """Without the post norm dy = gate dr_out (h without a gradient) whatever y
    holds: products of two bf16 values, exact in binary32 and rounded once."""
    gen = torch.Generator(device="cuda").manual_seed(cols)
    y, dr = (torch.randn(70, cols, device="cuda", generator=gen).to(BF16) for _ in range(2))
    gate = torch.randn(cols, device="cuda", generator=gen).to(BF16)
    y[3, cols // 2], y[4, 0], y[5, -1] = float("inf"), float("nan"), float("-inf")
    saved = trt.act8_pack(y) if bits == 8 else y
    got = trt.block_norm_bwd(None, dr, None, saved, gate, post=False, rms=rms, params=False)
    assert torch.equal(got[0], dr)
    assert torch.equal(got[1], (gate.float() * dr.float()).to(BF16))
