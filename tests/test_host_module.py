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


@pytest.fixture
def stale(tmp_path, monkeypatch):
    """A module of an earlier build at the place where the build puts a new one."""
    from mxfp4_quantized_expert_amd import build

    path = tmp_path / "_host_calls.so"
    path.write_bytes(b"of an earlier library")
    monkeypatch.setattr(build, "HOST_CALLS", str(path))
    return build, path


@pytest.mark.parametrize("compiler", ["false", "/nowhere/g++"])
def test_build_goes_on_without_a_compiler_for_the_module(stale, monkeypatch, capsys, compiler):
    """hipcc is enough for the library; a module that does not belong to it must not stay beside it."""
    build, path = stale
    monkeypatch.setenv("CXX", compiler)
    build._build_host_calls()
    assert not path.exists() and "ctypes" in capsys.readouterr().err


def test_build_goes_on_without_torch(stale, monkeypatch, capsys):
    build, path = stale
    monkeypatch.setitem(sys.modules, "torch", None)  # import torch raises ImportError
    build._build_host_calls()
    assert not path.exists() and "ctypes" in capsys.readouterr().err


REFUSED = """
import torch
from torch._subclasses.fake_tensor import FakeTensorMode
from torch.utils._python_dispatch import TorchDispatchMode
from mxfp4_quantized_expert_amd import binding
binding.load()
host = binding._host
assert host is not None

class Seen(TorchDispatchMode):
    names = []

    def __torch_dispatch__(self, func, types, args=(), kwargs=None):
        self.names.append(str(func))
        return func(*args, **(kwargs or {}))

x, pairs = torch.zeros((3, 8)), torch.zeros(3, dtype=torch.int32)
with Seen():  # the first call of the process that is left to the step-by-step path
    assert host.permute(x, pairs, 1) is None
print(len(Seen.names))
"""


def test_a_call_left_to_the_longer_way_makes_no_tensor_of_its_own():
    """What stands in for an unfit argument outlives the call, so no mode that happens to be on may make it."""
    if not os.path.exists(binding.HOST_PATH):
        pytest.skip("the module is not built")
    r = subprocess.run([sys.executable, "-c", REFUSED], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stdout + r.stderr
    assert r.stdout.split() == ["0"]
