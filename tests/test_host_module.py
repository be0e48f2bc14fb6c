"""The native module of the short host path (csrc/host_calls.cpp) is optional: without it, or with one
that cannot be loaded, every call goes through ctypes."""

import os
import shutil
import subprocess
import sys

import pytest

from mxfp4_quantized_expert_amd import binding

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

CALLS = """
import warnings
import torch
from mxfp4_quantized_expert_amd import binding
for i in range(3):  # the same every time, the fused layer's calls and the separate operators' alike
    with warnings.catch_warnings(record=True) as seen:
        warnings.simplefilter("always")
        assert binding.workspace_bytes(4, 64, 64, 2, 1) > 0
        try:
            binding.moe_permute(torch.zeros((4, 8)), torch.zeros(4, dtype=torch.int32), 1)
            raise SystemExit("a host tensor was taken")
        except ValueError as e:
            assert "device" in str(e), e
    print(i, binding._host is None, len(seen))
"""


@pytest.fixture
def package(tmp_path):
    """A copy of the package, and the run of a program that imports it."""
    if not os.path.exists(binding.LIB_PATH):
        pytest.skip("the library is not built")
    pkg = tmp_path / "mxfp4_quantized_expert_amd"
    pkg.mkdir()
    for name in ("__init__.py", "binding.py", "libmxfp4moe.so"):
        shutil.copy(os.path.join(ROOT, "mxfp4_quantized_expert_amd", name), pkg / name)

    def run():
        r = subprocess.run([sys.executable, "-c", CALLS], cwd=tmp_path, capture_output=True, text=True, timeout=300)
        assert r.returncode == 0, r.stdout + r.stderr
        return r.stdout.split("\n")[:3]

    return pkg, run


def test_without_the_module(package):
    _, run = package
    assert run() == ["0 True 0", "1 True 0", "2 True 0"]


def test_a_module_that_cannot_be_loaded(package):
    """E.g. one left from another Python or torch: one warning, and the calls work from the first on."""
    pkg, run = package
    (pkg / "_host_calls.so").write_bytes(b"\x7fELF of something else")
    assert run() == ["0 True 1", "1 True 0", "2 True 0"]
