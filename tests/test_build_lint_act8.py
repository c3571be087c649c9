"""The pipelined kernels' build-time checks (test_build_lint.py) on the weight
gradient from 8-bit rows, whose product issues the same copies from inline
assembly, with row counts and bases of its slice."""
import os
import shutil

import pytest

from test_build_lint import B, _asm, valu_to_vmem_hazards

UNIT = "kern_act8_weight.hip"

pytestmark = pytest.mark.skipif(not os.path.exists(B.HIPCC), reason="hipcc not installed")


@pytest.fixture(scope="module")
def assembly(tmp_path_factory):
    d = str(tmp_path_factory.mktemp("asm"))
    yield _asm(UNIT, d)
    shutil.rmtree(d, ignore_errors=True)


def test_no_vector_written_scalar_feeds_a_copy(assembly):
    assert valu_to_vmem_hazards(assembly) == []


def test_no_scalar_spills(assembly):
    assert "v_readlane_b32" not in assembly and "v_writelane_b32" not in assembly
