"""The pipelined kernels' build-time checks (test_build_lint.py) on the cross
entropy's products, which issue the same copies from inline assembly and take
their row counts from device memory.  (The statistics' epilogue spills scalars
around its comparisons, well away from any copy.)"""
import os
import shutil
from concurrent.futures import ThreadPoolExecutor

import pytest

from test_build_lint import B, _asm, valu_to_vmem_hazards

UNITS = ["kern_xent_stats.hip", "kern_xent_grad.hip", "kern_xent_input.hip", "kern_xent_weight.hip"]

pytestmark = pytest.mark.skipif(not os.path.exists(B.HIPCC), reason="hipcc not installed")


@pytest.fixture(scope="module")
def assembly(tmp_path_factory):
    d = str(tmp_path_factory.mktemp("asm"))
    with ThreadPoolExecutor(len(UNITS)) as ex:
        texts = dict(zip(UNITS, ex.map(lambda u: _asm(u, d), UNITS)))
    yield texts
    shutil.rmtree(d, ignore_errors=True)


@pytest.mark.parametrize("unit", UNITS)
def test_no_vector_written_scalar_feeds_a_copy(assembly, unit):
    assert valu_to_vmem_hazards(assembly[unit]) == []
