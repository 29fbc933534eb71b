"""How the embedding gradient divides its rows (csrc/embed_plan.cuh), compiled for
the host: every row in one tile, nothing beyond 32 bits up to the row limit."""
import ctypes
import os
import subprocess

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "atomistic_mlip_b200", "csrc")
MAX_ROWS = (1 << 31) - 4096

SRC = r"""
#include "embed_plan.cuh"
using namespace e2f::emb;
extern "C" void plans(int64_t N, int64_t V, int dv, int *o) {
  const SortPlan s = sort_plan(N, V);
  const RunPlan r = run_plan(N, V, dv);
  o[0] = s.tile; o[1] = s.tiles; o[2] = s.passes; o[3] = r.CL; o[4] = r.R; o[5] = r.tiles; o[6] = r.zero;
}
// Search among n keys of which the first `cut` are below v: the bound found, or -1
// for a read outside, -2 for no end.
extern "C" int bound(int n, int cut) {
  int lo = 0, hi = n;
  for (int it = 0; lo < hi; ++it) {
    if (it > 40) return -2;
    const int step = probe_step(lo, hi);
    int f = 32;
    for (int lane = 31; lane >= 0; --lane) {
      const int p = probe_at(lo, step, lane);
      if (p < 0 || (p < hi && p >= n)) return -1;
      if (p >= hi || p >= cut) f = lane;
    }
    narrow(lo, hi, step, f);
    if (lo < 0 || hi < lo || hi > n) return -1;
  }
  return lo;
}
"""


@pytest.fixture(scope="module")
def plan(tmp_path_factory):
    d = tmp_path_factory.mktemp("plan")
    (d / "plan.cpp").write_text(SRC)
    # (signed overflow ends the program)
    subprocess.check_call(["g++", "-std=c++17", "-O1", "-ftrapv", "-shared", "-fPIC", "-I", CSRC, str(d / "plan.cpp"),
                           "-o", str(d / "plan.so")])
    return ctypes.CDLL(str(d / "plan.so"))


def _plans(lib, N, V, dv):
    o = (ctypes.c_int * 7)()
    lib.plans(ctypes.c_int64(N), ctypes.c_int64(V), dv, o)
    return list(o)


@pytest.mark.parametrize("N", [1025, 2048, 2049, 100_002, 262_144, 262_145, 1 << 24, (1 << 31) - (1 << 24) - 1,
                               2_130_706_433, 2_147_000_000, MAX_ROWS - 1, MAX_ROWS])
@pytest.mark.parametrize("dv", [1, 9, 128, 1 << 20])
def test_every_row_is_in_one_tile(plan, N, dv):
    for V in (1, 255, 256, 65536, 1 << 24, MAX_ROWS):
        tile, tiles, passes, CL, R, rtiles, zero = _plans(plan, N, V, dv)
        assert tile % 2048 == 0 and 1 <= tiles <= 128
        assert (tiles - 1) * tile < N <= tiles * tile
        assert 1 << (8 * passes) > V >= 1 << (8 * (passes - 1)) or passes == 1
        assert CL in (8, 16, 32) and R % (256 // CL) == 0 and R // (256 // CL) <= 32 and R % 32 == 0
        assert (rtiles - 1) * R < N <= rtiles * R
        assert (zero - 1) * 64 < V <= zero * 64


@pytest.mark.parametrize("n", [1, 2, 31, 32, 33, 1000, 100_002, 2_000_000_000, 2_081_000_000, 2_147_000_000, MAX_ROWS])
def test_search_of_the_sorted_keys(plan, n):
    for cut in sorted({0, 1, 31, 32, n // 3, n // 2, n - n // 33, n - n // 32, n - 33, n - 2, n - 1, n}):
        if 0 <= cut <= n:
            assert plan.bound(n, cut) == cut
