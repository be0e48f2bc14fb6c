"""The choice of kernel and tile rows of the linear operators (csrc/linear_plan.h), compiled for the
host: its tile counts against drawn loads, and its choices at sizes where two were measured."""

import ctypes
import os
import subprocess

import numpy as np
import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
SHIM = """
#include "linear_plan.h"
using namespace mxlinear;
extern "C" double tiles(int64_t rows, int64_t experts, int tm) {
  return expected_tiles(Sizes{rows, 2880, 2880, experts > 0 ? experts : 1, experts > 0, false}, tm);
}
// rows of a tile, 0 for the 16-row kernels
extern "C" int plan(int64_t rows, int64_t n, int64_t k, int64_t experts, int nv, int forward) {
  const Sizes s{rows, n, k, experts > 0 ? experts : 1, experts > 0, nv != 0};
  const int64_t cols = ((forward ? n : k) + 255) / 256;
  const TilePlan p = plan_tiles(s, forward != 0, 128, cols, (int)(((forward ? k : n) + 63) / 64), 256);
  return p.pays ? p.rows : 0;
}
extern "C" int stream(int64_t rows, int64_t n, int64_t k, int64_t experts, int nv) {
  return stream_tile_rows(Sizes{rows, n, k, experts > 0 ? experts : 1, experts > 0, nv != 0}, 256);
}
"""


@pytest.fixture(scope="module")
def plan(tmp_path_factory):
    d = tmp_path_factory.mktemp("plan")
    (d / "shim.cpp").write_text(SHIM)
    subprocess.run(["g++", "-O1", "-std=c++17", "-fPIC", "-shared", "-Wall", "-Werror",
                    "-I" + os.path.join(ROOT, "mxfp4_quantized_expert_amd", "csrc"), str(d / "shim.cpp"), "-o",
                    str(d / "shim.so")], check=True)
    lib = ctypes.CDLL(str(d / "shim.so"))
    i64 = ctypes.c_int64
    lib.tiles.argtypes, lib.tiles.restype = [i64, i64, ctypes.c_int], ctypes.c_double
    lib.plan.argtypes = [i64, i64, i64, i64, ctypes.c_int, ctypes.c_int]
    lib.stream.argtypes = [i64, i64, i64, i64, ctypes.c_int]
    return lib


@pytest.mark.parametrize("tm", [32, 64, 128])
@pytest.mark.parametrize("experts", [8, 32, 128])
def test_tiles_of_evenly_routed_rows(plan, experts, tm):
    """Against counted tiles.  An expert's last tile is uncertain by one where its count is near a
    multiple of tm; the mean of 200 draws over all experts is known to a few percent, the normal
    approximation of the counts and the half-full last tile to a tenth of a tile an expert."""
    rng = np.random.default_rng(experts + tm)
    for mean in (1, 3, 6.5, 12, 24, 31, 40, 56, 64, 100, 128, 200, 500):
        rows = int(mean * experts)
        counts = rng.multinomial(rows, np.full(experts, 1 / experts), 200)
        want = np.ceil(counts / tm).sum(1).mean()
        got = plan.tiles(rows, experts, tm)
        # rows that leave an expert empty: the estimate gives it a tile all the same
        slack = 0.2 * experts + experts * np.exp(-mean)
        assert abs(got - want) <= slack, (mean, got, want)
        assert got >= min(experts, rows)


def test_dense_tiles(plan):
    assert [plan.tiles(r, 0, 64) for r in (1, 64, 65, 640)] == [1, 1, 2, 10]


@pytest.mark.parametrize("rows,n,k,experts,forward,good", [
    # us in tiles of 32, 64 and 128 rows
    (832, 5760, 2880, 128, True, (32, 64)),      # 277, 279, 292
    (1536, 5760, 2880, 128, True, (32, 64)),     # 288, 291, 303
    (768, 5760, 2880, 32, True, (64,)),          # 88, 82, 94
    (1280, 5760, 2880, 32, True, (64, 128)),     # 121, 89, 94
    (1792, 5760, 2880, 32, False, (64,)),        # 149, 104, 117
    (1792, 2880, 2880, 32, False, (64,)),        # 79, 56, 61
    (7168, 2880, 736, 128, False, (64, 128)),    # 78, 59, 62
    (384, 2880, 2880, 8, True, (32,)),           # 20, 25, 25
    (800, 2880, 2880, 8, True, (64,)),           # 32, 26, 43
    (16384, 2880, 2880, 128, True, (128,)),
    (16384, 2880, 2880, 0, False, (128,)),
    (512, 2880, 2880, 0, True, (32,)),           # 19, 25, 42
    (32, 2880, 2880, 0, True, (0,)),             # the 16-row kernel
])
def test_choices_where_both_sides_were_measured(plan, rows, n, k, experts, forward, good):
    assert plan.plan(rows, n, k, experts, 0, forward) in good


@pytest.mark.parametrize("rows,n,k,experts,good", [
    # us in tiles of 4 and of 8 rows, and through the other kernels
    (1, 2880, 2880, 0, 0),       # 5.0, 6.0, 4.6
    (8, 5760, 2880, 0, 0),       # 8.1, 14.3, 7.7
    (8, 4096, 2880, 0, 0),       # 7.3, 9.9, 5.4
    (1, 12288, 2880, 0, 4),      # 7.4, 8.7, 10.0
    (1, 32768, 736, 0, 4),       # 6.8, 7.6, 9.2
    (8, 32768, 2880, 0, 8),      # 18.8, 17.8, 23.5
    (9, 32768, 2880, 0, 0),
    (2, 2880, 2880, 4, 0),       # two experts at most: 8.0, 11.6, 6.9
    (4, 2880, 2880, 4, 4),       # 7.9, 9.4, 10.8
    (32, 736, 736, 32, 0),       # 9.7, 7.9, 5.8
    (64, 736, 736, 64, 4),       # 9.2, 9.6, 10.0
    (16, 5760, 2880, 32, 4),     # 24, 27, 45
    (192, 2880, 2880, 32, 8),    # 46, 38, 48
    (320, 5760, 2880, 32, 0),    # 126, 94, 78
    (1, 736, 2880, 0, 4),        # 3.4, 4.3, 4.0: fewer row groups than CUs
    (1, 2880, 4096, 0, 4),       # 5.9, 8.0, 6.0: two rounds of the 16-row kernel
    (1, 736, 12288, 0, 4),       # 6.0, 7.2, 11.8
    (2, 1440, 8192, 0, 4),       # 9.2, 11.0, 9.6
    (8, 736, 4096, 0, 8),        # 6.2, 6.2, 7.0
    (16, 736, 736, 16, 0),       # 6.4, 7.5, 4.9
    (24, 1000, 736, 8, 0),       # 6.4, 7.0, 4.8
])
@pytest.mark.parametrize("nv", [0, 1])
def test_streaming_where_both_sides_were_measured(plan, rows, n, k, experts, good, nv):
    assert plan.stream(rows, n, k, experts, nv) == good
