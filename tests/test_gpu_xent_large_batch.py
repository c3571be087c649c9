"""GPU parity of the linear cross entropy on the kernels that large batches
take: products that walk more tiles than there are compute units, over several
rows of tiles, and dW's on 256-wide tiles.  test_xent_plan.py holds that these
sizes take them.  Tolerances: test_gpu_xent.py."""
import pytest
import torch

from test_gpu_xent import BF16, F16, IGNORE, NAMES, Case, _gpu  # noqa: F401

pytestmark = pytest.mark.gpu

# tokens, vocabulary, width, share of ignored tokens.  WALKS: several rows of
# tiles, one to three turns of a workgroup; widths of one, two and three K steps
WALKS = [(1500, 16391, 72, 0.15), (2000, 20011, 40, 0.1), (1300, 15000, 136, 0.0)]
# dW on 256-wide tiles: live tokens in whole K steps and not
WIDE_DW = [(1000, 12500, 1032, 0.0), (1000, 12501, 1032, 0.4), (1024, 12544, 1024, 0.0), (1100, 14000, 904, 0.93)]
# dX's sums of several pieces over more than two rows of 256-wide tiles; the
# second with dW's 256-wide tiles too
PIECES = [(1000, 9000, 264, 0.1, 4096), (1000, 20000, 1032, 0.2, 12544)]


@pytest.mark.parametrize("dtype", [F16, BF16], ids=NAMES.get)
@pytest.mark.parametrize("T,V,D,ignored", WALKS)
def test_walked_tiles(T, V, D, ignored, dtype):
    c = Case(T, V, D, dtype, seed=D, ignored=ignored, weights="each")
    c.check_forward()
    c.check_backward()


@pytest.mark.parametrize("dtype", [F16, BF16], ids=NAMES.get)
@pytest.mark.parametrize("T,V,D,ignored", WIDE_DW)
def test_wide_tiles_of_dw(T, V, D, ignored, dtype):
    c = Case(T, V, D, dtype, seed=V, ignored=ignored, weights="each")
    c.check_backward(out_dtype=torch.float32 if ignored else None)
    c.check_backward(pad=3, offset=1)     # stores that are not whole runs of four


@pytest.mark.parametrize("dtype", [F16, BF16], ids=NAMES.get)
@pytest.mark.parametrize("T,V,D,ignored,piece", PIECES)
def test_pieces_over_several_rows_of_tiles(T, V, D, ignored, piece, dtype):
    Case(T, V, D, dtype, seed=piece, ignored=ignored, weights="each").check_backward(piece=piece)


@pytest.mark.parametrize("live", [0, 1, 63, 64, 65, 257])
def test_few_live_tokens_of_a_large_batch(live):
    # (what an ignored row holds reaches nothing: NaN)
    c = Case(1000, 12500, 1032, BF16, seed=live, weights="each")
    off = torch.randperm(1000, generator=torch.Generator().manual_seed(live))[live:]
    c.target[off.cuda()] = IGNORE
    c.x[off.cuda()] = float("nan")
    c.ht = c.target.cpu().numpy()
    if live:
        c.check_forward()
        c.check_backward()
    else:
        loss, lse = c.forward()
        dx, dw = c.backward()
        assert all((t == 0).all() for t in (loss, lse, dx, dw))
