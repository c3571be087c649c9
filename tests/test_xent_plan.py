"""CPU tests of how the linear cross entropy is cut up: the sizes of
test_gpu_xent_large_batch.py take the kernels that they are meant for, and the
room for dX's sums and its grid hold for every number of live tokens."""
import json
import os
import shutil
import subprocess

import pytest

import thread_register_tile_amd as trt
from test_gpu_xent_large_batch import PIECES, WALKS, WIDE_DW

HEADER = os.path.join(os.path.dirname(trt.__file__), "csrc", "xent_plan.hpp")
UNITS = 256

pytestmark = pytest.mark.skipif(shutil.which("g++") is None, reason="g++ not installed")

SOURCE = r"""
#include <cstdio>
#include <cstdlib>
#include <initializer_list>
#include "%s"
using namespace trt;
static int plan(char** a) {
  const int64_t T = atoll(a[0]), V = atoll(a[1]), D = atoll(a[2]), piece = atoll(a[3]);
  const XentFwdPlan f = xent_fwd_plan(T, V);
  const XentBwdPlan b = xent_bwd_plan(T, V, D, piece);
  printf("{\"fwd\": %%d, \"g\": %%d, \"x\": %%d, \"w\": %%d, \"halves\": %%d, \"piece\": %%ld, \"pieces\": %%ld}\n",
         f.wide, b.wide_g, b.wide_x, b.wide_w, b.halves, (long)b.piece, (long)b.pieces);
  return 0;
}
// every live count of many sizes: sums and workgroups that dX's product may ask for
static int room() {
  long bad = 0, n = 0;
  for (int64_t T : {1, 2, 63, 64, 65, 100, 127, 128, 129, 192, 193, 255, 256, 257, 300, 1000, 4097})
    for (int64_t D : {1, 8, 128, 192, 193, 257, 1024, 4096})
      for (int64_t V : {1, 64, 500, 1000, 4096, 32003, 131072})
        for (int64_t piece : {0, 64, 1024}) {
          const XentBwdPlan p = xent_bwd_plan(T, V, D, piece);
          const int64_t k = p.piece < V ? p.piece : V, most = T << (p.halves ? 1 : 0), tile = p.wide_x ? 256 : 128;
          const int64_t have = (p.bytes - p.sums) / 4 / p.padded;
          for (int64_t live = 1; live <= most; ++live, ++n) {
            const int64_t slice = xent_slice(xent_slices(live, D, k, p.wide_x), k), s = (k + slice - 1) / slice;
            const int64_t tiles = s * ((live + tile - 1) / tile) * ((D + tile - 1) / tile);
            bad += s * xent_sum_rows(live) > have || tiles > p.most_tiles || s > kXentMostSlices || slice %% 64 != 0;
          }
        }
  printf("{\"checked\": %%ld, \"bad\": %%ld}\n", n, bad);
  return 0;
}
int main(int c, char** a) { return c == 5 ? plan(a + 1) : room(); }
"""


@pytest.fixture(scope="module")
def program(tmp_path_factory):
    d = tmp_path_factory.mktemp("plan")
    (d / "plan.cpp").write_text(SOURCE % HEADER)
    exe = str(d / "plan")
    subprocess.run(["g++", "-std=c++20", "-O2", str(d / "plan.cpp"), "-o", exe], check=True)
    return lambda *a: json.loads(subprocess.run([exe, *map(str, a)], check=True, capture_output=True, text=True).stdout)


def tiles(m, n, t=256):
    return -(-m // t) * -(-n // t)


def fewest_live(T, ignored):
    """A bound on how many tokens are live, for the tests' random targets."""
    return int(T * (1 - ignored) - 4 * (T * ignored * (1 - ignored)) ** 0.5)


@pytest.mark.parametrize("T,V,D,ignored", WALKS)
def test_sizes_that_walk(program, T, V, D, ignored):
    p, live = program(T, V, D, 0), fewest_live(T, ignored)
    assert p["fwd"] and p["g"] and p["pieces"] == 1
    assert tiles(live, V) > UNITS and live > 3 * 256


@pytest.mark.parametrize("T,V,D,ignored", WIDE_DW)
def test_sizes_with_wide_dw(program, T, V, D, ignored):
    assert program(T, V, D, 0)["w"]


@pytest.mark.parametrize("T,V,D,ignored,piece", PIECES)
def test_sizes_in_pieces(program, T, V, D, ignored, piece):
    p = program(T, V, D, piece)
    assert p["x"] and p["pieces"] > 1 and fewest_live(T, ignored) > 2 * 256


def test_one_of_the_pieces_has_wide_dw(program):
    assert [program(*c[:3], c[4])["w"] for c in PIECES] == [0, 1]


def test_room_for_every_number_of_live_tokens(program):
    r = program()
    assert r["checked"] > 100000 and r["bad"] == 0
