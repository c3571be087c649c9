"""GPU parity of the block norm where test_gpu_blocknorm.py's lists leave gaps:
the widths on both sides of the changes to 3, 6, 10 and 12 waves a row, and the
backward workgroups of several rows of 129 to 512 chunks, with rows that leave
some of their waves idle.  Oracle, inputs and tolerances are that file's."""
import pytest
import torch

from test_gpu_blocknorm import BF16, F16, F32, MIX, _gpu, run_case  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("i,cols", list(enumerate([1535, 1536, 1537, 3070, 3073, 5120, 5121])))
@pytest.mark.parametrize("dtype", [F16, BF16])
def test_widths_16(i, cols, dtype):
    for j, rows in enumerate((1, 5, 67)):
        rms, post, gate = MIX[(3 * i + 5 * j + (dtype == BF16)) % len(MIX)]
        run_case(rows, cols, dtype, rms=rms, post=post, gate=gate, span=3 if gate == "sequence" else None, pdt=F32 if i % 2 else dtype,
                 saved="8bit" if (i + j) % 2 else "same", seed=i)


@pytest.mark.parametrize("i,cols", list(enumerate([768, 769, 1536, 1537, 2560, 2561, 3070, 3073])))
def test_widths_32(i, cols):
    for j, rows in enumerate((1, 5, 67)):
        rms, post, gate = MIX[(3 * i + 5 * j) % len(MIX)]
        run_case(rows, cols, F32, rms=rms, post=post, gate=gate, span=3 if gate == "sequence" else None,
                 saved="8bit" if (i + j) % 2 else "same", seed=i)


# 2 rows to a workgroup of 4 waves each, 4 of 2, 2 of 6, 4 of 3; the last
# sequence's rows no multiple of them
GATES = [("channel", None), ("sequence", 97), ("none", None), ("each", None), ("sequence", 130)]


@pytest.mark.parametrize("i,rows,cols", [(0, 515, 4096), (1, 1027, 2048), (2, 515, 2900), (3, 1027, 1400)])
@pytest.mark.parametrize("rms", [False, True])
@pytest.mark.parametrize("saved", ["same", "8bit"])
@pytest.mark.parametrize("dtype", [F16, BF16])
def test_several_rows_16(i, rows, cols, rms, saved, dtype):
    gate, span = GATES[(i + 2 * rms + (saved == "8bit") + 3 * (dtype == BF16)) % 5]
    run_case(rows, cols, dtype, gate=gate, span=span, rms=rms, saved=saved)


@pytest.mark.parametrize("i,rows,cols", [(0, 515, 2000), (1, 1027, 1000), (2, 515, 1400), (3, 1027, 700)])
@pytest.mark.parametrize("rms", [False, True])
@pytest.mark.parametrize("saved", ["same", "8bit"])
def test_several_rows_32(i, rows, cols, rms, saved):
    gate, span = GATES[(i + 2 * rms + (saved == "8bit")) % 5]
    run_case(rows, cols, F32, gate=gate, span=span, rms=rms, saved=saved)
