"""What the expert layer's separate operators refuse, before any launch (CPU only)."""

import os

import pytest
import torch

from mxfp4_quantized_expert_amd import binding

A = 0x100000  # an aligned fake address: every call here fails, or has nothing to do, before use


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(binding.LIB_PATH):
        from mxfp4_quantized_expert_amd import build
        build.build(verbose=False)
    return binding.load()


def test_permute_checks(lib):
    f = lib.moe_permute
    for bad in [(-1, 8, 2, 8), (4, 0, 2, 8), (4, 8, 0, 8), (4, 8, 33, 8), (4, 8, 2, -1), (4, (1 << 28) + 1, 2, 8),
                (1 << 30, 8, 2, 8), (4, 8, 2, 1 << 31)]:
        assert f(A, 0, A, *bad, A, A, None) == -2, bad
    assert f(A, 3, A, 4, 8, 2, 8, A, A, None) == -1   # no such element type
    assert f(A, -1, A, 4, 8, 2, 8, A, A, None) == -1
    assert f(None, 0, A, 4, 8, 2, 8, A, A, None) == -1
    assert f(A, 0, None, 4, 8, 2, 8, A, A, None) == -1
    assert f(A, 0, A, 4, 8, 2, 8, None, A, None) == -1
    assert f(A, 0, A, 4, 8, 2, 8, A, None, None) == -1
    assert f(A + 1, 0, A, 4, 8, 2, 8, A, A, None) == -4
    assert f(A + 2, 2, A, 4, 8, 2, 8, A, A, None) == -4
    assert f(A, 0, A + 2, 4, 8, 2, 8, A, A, None) == -4
    assert f(A, 0, A, 4, 8, 2, 8, A, A + 1, None) == -4
    assert f(None, 0, None, 0, 8, 2, 0, None, None, None) == 0


def test_permute_backward_and_unpermute_checks(lib):
    f, g = lib.moe_permute_backward, lib.moe_unpermute
    assert f(A, 0, A, 4, 0, 2, 8, A, None) == -2 and g(A, 0, A, A, 4, 0, 2, 8, A, None) == -2
    assert f(A, 7, A, 4, 8, 2, 8, A, None) == -1 and g(A, 7, A, A, 4, 8, 2, 8, A, None) == -1
    for i in (0, 2, 7):
        args = [A, 0, A, 4, 8, 2, 8, A, None]
        args[i] = None
        assert f(*args) == -1
        args[i] = A + 1
        assert f(*args) == -4
    for i in (0, 2, 3, 8):
        args = [A, 0, A, A, 4, 8, 2, 8, A, None]
        args[i] = None
        assert g(*args) == -1
        args[i] = A + 1
        assert g(*args) == -4
    assert f(None, 0, None, 0, 8, 2, 0, None, None) == 0 and g(None, 0, None, None, 0, 8, 2, 0, None, None) == 0


def test_unpermute_backward_and_route_backward_checks(lib):
    f, g = lib.moe_unpermute_backward, lib.moe_route_backward
    for i in (0, 1, 3, 4, 5, 10, 11):
        args = [A, A, 0, A, A, A, 4, 8, 2, 8, A, A, None]
        args[i] = None
        assert f(*args) == -1
        args[i] = A + 1
        assert f(*args) == -4
    assert f(A, A, 0, A, A, A, 4, 8, 40, 8, A, A, None) == -2
    assert f(None, None, 0, None, None, None, 0, 8, 2, 0, None, None, None) == 0
    for bad in [(4, 0, 1), (4, 513, 1), (4, 8, 9), (-1, 8, 2), (4, 8, 0)]:
        assert g(A, A, A, *bad, A, None) == -2
    for i in (0, 1, 2, 6):
        args = [A, A, A, 4, 8, 2, A, None]
        args[i] = None
        assert g(*args) == -1
        args[i] = A + 2
        assert g(*args) == -4
    assert g(None, None, None, 0, 8, 2, None, None) == 0


def test_binding_refuses_host_tensors_and_wrong_types():
    x = torch.zeros((4, 8), dtype=torch.bfloat16)
    pairs = torch.zeros((8,), dtype=torch.int32)
    w = torch.zeros((4, 2))
    with pytest.raises(ValueError, match="device"):
        binding.moe_permute(x, pairs, 2)
    with pytest.raises(TypeError):
        binding.moe_permute(x.double(), pairs, 2)
    with pytest.raises(ValueError, match="dimension"):
        binding.moe_permute(x[0], pairs, 2)
    with pytest.raises(ValueError, match="top_k"):
        binding.moe_permute(x, pairs, 0)
    with pytest.raises(ValueError, match="multiple"):
        binding.moe_permute_backward(x, pairs, 3)
    with pytest.raises(ValueError, match="device"):
        binding.moe_unpermute(x, pairs, w)
    with pytest.raises(ValueError, match="device"):
        binding.moe_unpermute_backward(x, x, pairs, pairs, w)
    with pytest.raises(ValueError, match="device"):
        binding.moe_route_backward(pairs.view(4, 2), w, w, 8)


def _linear_calls(lib):
    """(call of the pointers and sizes by name, pointer names) of the four linear entry points."""
    for name in ("moe_mxfp4_linear", "moe_nvfp4_linear", "moe_mxfp4_linear_backward", "moe_nvfp4_linear_backward"):
        def call(x=A, blocks=A, scales=A, scale2=A, bias=A, offsets=A, y=A, R=8, K=64, N=40, E=4, name=name):
            args = [x, blocks, scales]
            args += [scale2] if "nvfp4" in name else []
            args += [] if "backward" in name else [bias]
            return getattr(lib, name)(*args, offsets, R, K, N, E, y, None)
        yield name, call


def test_linear_checks(lib):
    for name, call in _linear_calls(lib):
        for bad in [dict(R=-1), dict(R=1 << 31), dict(K=48), dict(K=0), dict(K=16), dict(N=0), dict(E=0), dict(E=513),
                    dict(K=(1 << 20) + 32), dict(N=(1 << 20) + 1), dict(K=1 << 18, N=1 << 14)]:
            assert call(**bad) == -2, (name, bad)
        assert call(offsets=None) == -1, name          # more than one expert need offsets
        for ptr in ("x", "blocks", "scales", "y"):
            assert call(**{ptr: None}) == -1, (name, ptr)
            assert call(**{ptr: A + 8}) == -4, (name, ptr)
        assert call(offsets=A + 2) == -4, name
        if "nvfp4" in name:
            assert call(scale2=None) == -1 and call(scale2=A + 2) == -4
        if "backward" not in name:
            assert call(bias=A + 1) == -4
        assert call(x=None, y=None, R=0) == 0


def test_linear_binding_refusals():
    x = torch.zeros((4, 64), dtype=torch.bfloat16)
    blocks, scales = torch.zeros((40, 32), dtype=torch.uint8), torch.zeros((40, 2), dtype=torch.uint8)
    with pytest.raises(ValueError, match="device"):
        binding.moe_mxfp4_linear(x, blocks, scales)
    with pytest.raises(ValueError, match="blocks has 2 dimensions"):
        binding.moe_mxfp4_linear(x, blocks, scales, None, torch.zeros(2, dtype=torch.int32))
    with pytest.raises(ValueError, match="blocks has 3 dimensions"):
        binding.moe_mxfp4_linear_backward(x, blocks[None], scales[None])
    with pytest.raises(ValueError, match="dimensions"):
        binding.moe_nvfp4_linear(x[0], blocks, scales, None)


def test_shared_memory_is_seen():
    flat = torch.zeros(32)
    binding._apart(flat[:16], "out", flat[16:], None, flat[:0])
    binding._apart(flat[:0], "out", flat)
    for a, b in ((flat, flat), (flat[:17], flat[16:]), (flat[16:], flat[:17]), (flat[4:8], flat)):
        with pytest.raises(ValueError, match="out shares memory"):
            binding._apart(a, "out", torch.zeros(3), b)
