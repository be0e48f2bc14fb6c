"""The choice of kernel and tile of the 8-bit products (csrc/fp8_plan.h), compiled for the host: its
choices at sizes where several were measured."""

import ctypes
import os
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
SHIM = """
#include "fp8_plan.h"
extern "C" int forward(int64_t rows, int64_t n, int64_t experts) {
  const mxfp8::Plan p = mxfp8::plan_forward(rows, n, experts, 256);
  return (p.few ? 1 : -1) * (1000 * p.rows + p.cols);
}
extern "C" int backward_few(int64_t rows, int64_t k, int64_t experts) {
  return mxfp8::backward_has_few(rows, k, experts, 256);
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
    lib.forward.argtypes = lib.backward_few.argtypes = [ctypes.c_int64] * 3

    def forward(rows, n, experts):
        v = lib.forward(rows, n, experts)
        return v > 0, abs(v) // 1000, abs(v) % 1000

    lib.choice = forward
    return lib


@pytest.mark.parametrize("rows,n,want", [
    (1, 2880, (True, 16, 16)), (32, 2880, (True, 16, 16)), (64, 2880, (True, 32, 32)), (128, 2880, (True, 32, 64)),
    (256, 2880, (False, 32, 128)), (512, 2880, (False, 64, 128)), (1024, 2880, (False, 64, 256)),
    (2048, 2880, (False, 128, 256)), (16384, 2880, (False, 128, 256)), (1000, 736, (False, 32, 128)),
    (4000, 736, (False, 64, 256)), (500, 100, (True, 16, 16)), (4000, 100, (True, 32, 64)),
])
def test_dense(plan, rows, n, want):
    assert plan.choice(rows, n, 1) == want


@pytest.mark.parametrize("rows,n,experts,want", [
    (4, 2880, 32, (True, 16, 16)), (16, 2880, 32, (True, 16, 16)), (64, 2880, 32, (False, 64, 128)),
    (64, 2880, 128, (False, 64, 128)), (1024, 2880, 128, (False, 64, 256)), (4096, 2880, 128, (False, 64, 256)),
    (16384, 2880, 128, (False, 128, 256)), (16384, 5760, 128, (False, 128, 256)), (4096, 2880, 32, (False, 128, 256)),
    (128, 1000, 8, (True, 16, 16)), (2048, 1000, 8, (False, 64, 128)), (8192, 1000, 8, (False, 128, 256)),
])
def test_per_expert(plan, rows, n, experts, want):
    assert plan.choice(rows, n, experts) == want


def test_every_size_has_a_kernel(plan):
    """Only tiles that are built; the largest sizes do not overflow."""
    built = {(True, 16, 16), (True, 32, 32), (True, 32, 64), (False, 32, 128), (False, 64, 128), (False, 64, 256),
             (False, 128, 256)}
    seen = set()
    for rows in (1, 2, 15, 16, 17, 40, 100, 250, 700, 2000, 5000, 100000, 2 ** 31 - 1):
        for n in (1, 16, 100, 736, 2880, 5760, 50000, 2 ** 31 - 1):
            for experts in (1, 2, 8, 32, 128, 4096):
                seen.add(plan.choice(rows, n, experts))
    assert seen == built


@pytest.mark.parametrize("rows,k,experts,few", [
    (1, 2880, 1, True), (256, 2880, 1, True), (512, 2880, 1, False), (16384, 2880, 1, False), (300, 736, 8, True),
    (512, 736, 8, True), (2048, 736, 8, False), (4, 2880, 32, True), (16, 2880, 32, False), (16, 736, 128, True),
    (64, 736, 128, False), (16384, 2880, 128, False),
])
def test_backward(plan, rows, k, experts, few):
    assert bool(plan.backward_few(rows, k, experts)) is few
