"""Which tiles the products with many rows take, asked of the library's own host code (csrc/tile_plan.h) built by itself:
the exactness tests' sizes reach every kernel that any size reaches."""
import ctypes
import os
import random
import shutil
import subprocess

import pytest

from tests.test_block_exact import WHOLE_DXS, WHOLE_LINEARS

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "weight_only_int4_stats_amd", "csrc")
SOURCE = """
#include "tile_plan.h"
extern "C" void dx(int64_t M, int64_t N, int64_t K, int64_t cus, int64_t* o) {
  const awqk::TilePlan p = awqk::dx_plan(M, N, K, cus);
  o[0] = p.mb; o[1] = p.wm; o[2] = p.S; o[3] = 0;
}
extern "C" void linear(int64_t M, int64_t N, int64_t K, int64_t cus, int64_t* o) {
  const awqk::LinearPlan p = awqk::linear_plan(M, N, K, cus);
  o[0] = p.t.mb; o[1] = p.t.wm; o[2] = p.t.S; o[3] = p.wide;
}
extern "C" int64_t parts(int is_dx, int64_t M, int64_t cols, int64_t stages, int64_t cus) {
  return is_dx ? awqk::tile_parts(awqk::kDxShapes, M, cols, stages, cus) : awqk::tile_parts(awqk::kLinearShapes, M, cols, stages, cus);
}
"""


@pytest.fixture(scope="module")
def plan(tmp_path_factory):
    """kernel(op, M, N, K): what names the kernel that op takes on 256 compute units, and its number of slices."""
    cc = shutil.which("g++") or shutil.which("clang++")
    if cc is None:
        pytest.skip("no host compiler")
    d = tmp_path_factory.mktemp("plan")
    (d / "plan.cpp").write_text(SOURCE)
    subprocess.run([cc, "-std=c++17", "-O1", "-shared", "-fPIC", "-I", CSRC, str(d / "plan.cpp"), "-o", str(d / "plan.so")], check=True)
    lib = ctypes.CDLL(str(d / "plan.so"))
    i64 = ctypes.c_int64
    lib.parts.restype = i64
    lib.parts.argtypes = [ctypes.c_int] + [i64] * 4

    def kernel(op, M, N, K):
        out = (i64 * 4)()
        getattr(lib, op)(i64(M), i64(N), i64(K), i64(256), out)
        mb, wm, slices, wide = out
        return ("mixed" if wide else (mb, wm, slices > 1)), slices
    kernel.parts = lib.parts
    return kernel


def sizes(n, seed, rows):
    rng = random.Random(seed)
    log = lambda lo, hi: int(lo * (hi / lo) ** rng.random())  # noqa: E731
    return [(log(rows, 20000), log(1, 40000), 64 * log(1, 512)) for _ in range(n)]


def test_the_exactness_cases_reach_every_kernel_of_dx(plan):
    reached = {plan("dx", M, N, K)[0] for M, N, K, _ in WHOLE_DXS}
    assert reached == {plan("dx", *s)[0] for s in sizes(20000, 1, 1)}


def test_the_exactness_cases_reach_every_kernel_of_the_linear(plan):
    # above 64 rows every linear takes the tiles
    reached = {plan("linear", M, N, K)[0] for M, N, K, _ in WHOLE_LINEARS if M > 64}
    assert reached == {plan("linear", *s)[0] for s in sizes(20000, 2, 65)}


@pytest.mark.parametrize("op", ["dx", "linear"])
def test_slices_stay_within_what_the_workspace_query_counts(plan, op):
    for M, N, K in sizes(5000, 3, 1):
        slices = plan(op, M, N, K)[1]
        if slices > 1:
            cols, stages = (K, (N + 63) // 64) if op == "dx" else (N, K // 64)
            assert slices * M <= plan.parts(op == "dx", M, cols, stages, 256), (op, M, N, K)
