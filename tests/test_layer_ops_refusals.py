"""What the operators around the expert products refuse, before any launch (CPU only)."""

import ctypes
import math
import os

import pytest
import torch

from mxfp4_quantized_expert_amd import binding

A = 0x100000  # an aligned fake address: every call here fails, or has nothing to do, before use
NAN, INF = math.nan, math.inf


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(binding.LIB_PATH):
        from mxfp4_quantized_expert_amd import build
        build.build(verbose=False)
    return binding.load()


def norm_args(x=A, residual=A, weight=A, dtype=0, wdtype=0, eps=1e-5, T=4, H=8, summed=A, out=(A,), rstd=A):
    return (x, residual, weight, dtype, wdtype, eps, T, H, summed, *out, rstd, None)


@pytest.mark.parametrize("fp8", [False, True])
def test_norm_checks(lib, fp8):
    f, outs = (lib.moe_rms_norm_fp8, (A, A)) if fp8 else (lib.moe_rms_norm, (A,))

    def call(**kw):
        return f(*norm_args(**{"out": outs, **kw}))

    for bad in (dict(T=-1), dict(T=1 << 31), dict(H=0), dict(H=32769)):
        assert call(**bad) == -2, bad
    for bad in (dict(dtype=3, wdtype=3), dict(dtype=-1, wdtype=-1), dict(wdtype=1), dict(dtype=2, wdtype=0),
                dict(eps=-1e-9), dict(eps=NAN), dict(eps=INF), dict(x=None), dict(weight=None), dict(rstd=None),
                dict(summed=None)):
        assert call(**bad) == -1, bad
    for i in range(len(outs)):
        assert call(out=outs[:i] + (None,) + outs[i + 1:]) == -1
    for bad in (dict(x=A + 1), dict(residual=A + 1), dict(summed=A + 1), dict(weight=A + 1), dict(rstd=A + 2),
                dict(wdtype=2, weight=A + 2), dict(dtype=2, wdtype=2, x=A + 2)):
        assert call(**bad) == -4, bad
    assert call(out=(A, A + 2) if fp8 else (A + 1,)) == -4
    assert call(T=0, x=None, weight=None, summed=None, rstd=None, out=(None,) * len(outs)) == 0


def test_norm_backward_checks(lib):
    f = lib.moe_rms_norm_backward
    n = ctypes.c_size_t(0)

    def call(dy=A, ds=A, s=A, w=A, dtype=0, wdtype=0, rstd=A, T=4, H=8, dx=A, dw=A, ws=A, have=1 << 40):
        n.value = have
        return f(dy, ds, s, w, dtype, wdtype, rstd, T, H, dx, dw, ws, ctypes.byref(n), None)

    assert call(ws=None) == 0 and n.value >= 8 * 4
    small = n.value
    assert call(ws=None, T=4096, H=2880) == 0 and n.value > small
    assert f(A, A, A, A, 0, 0, A, 4, 8, A, A, A, None, None) == -1
    assert call(have=small - 1) == -3
    for bad in (dict(T=-1), dict(H=0), dict(H=32769), dict(T=1 << 31)):
        assert call(**bad) == -2, bad
    for bad in (dict(dy=None), dict(s=None), dict(w=None), dict(rstd=None), dict(dx=None), dict(dw=None),
                dict(dtype=5), dict(wdtype=1)):
        assert call(**bad) == -1, bad
    for bad in (dict(dy=A + 1), dict(ds=A + 1), dict(s=A + 1), dict(w=A + 1), dict(dx=A + 1), dict(rstd=A + 2),
                dict(dw=A + 2), dict(ws=A + 2)):
        assert call(**bad) == -4, bad


def test_quantize_and_swiglu_checks(lib):
    q, s, s8, b = lib.moe_fp8_quantize, lib.moe_swiglu, lib.moe_swiglu_fp8, lib.moe_swiglu_backward
    for R, W, st in ((-1, 8, -2), (4, 0, -2), (4, (1 << 28) + 1, -2), (1 << 31, 8, -2), (1 << 30, 257, -2)):
        assert q(A, 0, R, W, A, A, None) == st
        assert s(A, 0, R, W, 1.0, 1.0, 1.0, 0, A, None) == st
        assert s8(A, 0, R, W, 1.0, 1.0, 1.0, 0, A, A, None) == st
        assert b(A, A, 0, R, W, 1.0, 1.0, 1.0, 0, A, None) == st
    assert s(A, 0, 4, (1 << 27) + 1, 1.0, 1.0, 1.0, 0, A, None) == -2
    for alpha, limit, offset in ((NAN, 1, 0), (INF, 1, 0), (1, 0, 0), (1, -1, 0), (1, NAN, 0), (1, 1, INF), (1, 1, NAN)):
        assert s(A, 0, 4, 8, alpha, limit, offset, 0, A, None) == -1
        assert s8(A, 0, 4, 8, alpha, limit, offset, 0, A, A, None) == -1
        assert b(A, A, 0, 4, 8, alpha, limit, offset, 0, A, None) == -1
    assert q(None, 0, 4, 8, A, A, None) == -1 and q(A, 0, 4, 8, None, A, None) == -1 and q(A, 0, 4, 8, A, None, None) == -1
    assert q(A, 9, 4, 8, A, A, None) == -1 and s(A, -1, 4, 8, 1.0, 1.0, 0.0, 0, A, None) == -1
    assert q(A + 1, 0, 4, 8, A, A, None) == -4 and q(A, 0, 4, 8, A, A + 2, None) == -4
    assert s(None, 0, 4, 8, 1.0, 1.0, 0.0, 0, A, None) == -1 and s(A, 0, 4, 8, 1.0, 1.0, 0.0, 0, None, None) == -1
    assert s(A + 1, 0, 4, 8, 1.0, 1.0, 0.0, 0, A, None) == -4 and s(A, 2, 4, 8, 1.0, 1.0, 0.0, 0, A + 2, None) == -4
    assert s8(A, 0, 4, 8, 1.0, 1.0, 0.0, 0, None, A, None) == -1 and s8(A, 0, 4, 8, 1.0, 1.0, 0.0, 0, A, A + 1, None) == -4
    for i in (0, 1, 9):
        args = [A, A, 0, 4, 8, 1.0, 1.0, 0.0, 0, A, None]
        args[i] = None
        assert b(*args) == -1
        args[i] = A + 1
        assert b(*args) == -4
    assert q(None, 0, 0, 8, None, None, None) == 0 and s(None, 0, 0, 8, 1.0, 1.0, 0.0, 0, None, None) == 0
    assert b(None, None, 0, 0, 8, 1.0, INF, 0.0, 0, None, None) == 0


@pytest.mark.parametrize("backward", [False, True])
def test_fp8_linear_checks(lib, backward):
    def call(x=A, xs=A, w=A, ws=A, bias=A, offsets=A, y=A, R=8, K=64, N=40, E=4):
        if backward:
            return lib.moe_fp8_linear_backward(x, w, ws, offsets, R, K, N, E, y, None)
        return lib.moe_fp8_linear(x, xs, w, ws, bias, offsets, R, K, N, E, y, None)

    for bad in (dict(R=-1), dict(R=1 << 31), dict(K=24), dict(K=0), dict(N=0), dict(E=0), dict(E=513),
                dict(K=(1 << 20) + 16), dict(N=(1 << 20) + 1), dict(K=1 << 16, N=1 << 15)):
        assert call(**bad) == -2, bad
    assert call(offsets=None) == -1  # more than one expert need offsets
    for ptr in ("x", "w", "y"):
        assert call(**{ptr: None}) == -1 and call(**{ptr: A + 8}) == -4, ptr
    assert call(ws=None) == -1 and call(ws=A + 2) == -4 and call(offsets=A + 2) == -4
    if not backward:
        assert call(xs=None) == -1 and call(xs=A + 2) == -4 and call(bias=A + 1) == -4
    assert call(x=None, y=None, R=0) == 0


def test_balance_checks(lib):
    f, g = lib.moe_balance_loss, lib.moe_balance_loss_backward
    n = ctypes.c_size_t(0)

    def call(lg=A, ids=A, mask=None, T=4096, E=8, k=2, loss=A, counts=A, density=A, ws=A, have=1 << 40):
        n.value = have
        return f(lg, ids, mask, T, E, k, loss, counts, density, ws, ctypes.byref(n), None)

    assert call(ws=None) == 0
    need = n.value
    assert need > 0 and call(have=need - 1) == -3
    assert call(ws=None, T=1) == 0 and n.value == 0  # one block joins its own sums
    for bad in (dict(T=-1), dict(E=0), dict(E=513), dict(k=0), dict(k=9), dict(k=33, E=64), dict(T=1 << 30, k=4)):
        assert call(**bad) == -2, bad
    for bad in (dict(lg=None), dict(ids=None), dict(loss=None), dict(counts=None), dict(density=None)):
        assert call(**bad) == -1, bad
    for bad in (dict(lg=A + 1), dict(ids=A + 2), dict(loss=A + 1), dict(counts=A + 2), dict(density=A + 2), dict(ws=A + 2)):
        assert call(**bad) == -4, bad
    assert f(A, A, None, 4, 8, 2, A, A, A, A, None, None) == -1
    for bad in ((-1, 8), (4, 0), (4, 513)):
        assert g(A, A, A, None, None, *bad, A, None) == -2
    for i in (0, 1, 2, 7):
        args = [A, A, A, None, None, 4, 8, A, None]
        args[i] = None
        assert g(*args) == -1
        args[i] = A + 2
        assert g(*args) == -4
    assert g(A, A, A, None, A + 1, 4, 8, A, None) == -4
    assert g(None, None, None, None, None, 0, 8, None, None) == 0


def test_binding_refuses_host_tensors_and_wrong_types():
    x, w = torch.zeros((4, 8)), torch.ones(8)
    codes, scales = torch.zeros((4, 16)).to(torch.float8_e4m3fn), torch.ones((4, 1))
    weight = torch.zeros((8, 16)).to(torch.float8_e4m3fn)
    for call in (lambda: binding.moe_rms_norm(x, w), lambda: binding.moe_rms_norm_fp8(x, w, x),
                 lambda: binding.moe_rms_norm_backward(x, x, w, torch.ones(4)),
                 lambda: binding.moe_fp8_quantize(x), lambda: binding.moe_swiglu(x), lambda: binding.moe_swiglu_fp8(x),
                 lambda: binding.moe_swiglu_backward(x, x),
                 lambda: binding.moe_fp8_linear(codes, scales, weight, torch.ones((1, 1))),
                 lambda: binding.moe_fp8_linear_backward(x.bfloat16(), weight, torch.ones((1, 1))),
                 lambda: binding.moe_balance_loss(x, torch.zeros((4, 2), dtype=torch.int32)),
                 lambda: binding.moe_balance_loss_backward(x, w, torch.ones(()))):
        with pytest.raises(ValueError, match="device"):
            call()
    for call in (lambda: binding.moe_rms_norm(x.double(), w), lambda: binding.moe_rms_norm(x, None),
                 lambda: binding.moe_fp8_quantize(x.to(torch.int32)), lambda: binding.moe_swiglu(None),
                 lambda: binding.moe_fp8_linear(x, scales, weight, scales), lambda: binding.moe_balance_loss(x.half(), w),
                 lambda: binding.moe_fp8_linear_backward(x, weight, scales)):
        with pytest.raises((TypeError, ValueError)):
            call()
    with pytest.raises(ValueError, match="gates and ups"):
        binding.moe_swiglu(x[:, :7])
    with pytest.raises(ValueError, match="weight has 2 dimensions"):
        binding.moe_fp8_linear(codes, scales, weight, scales, None, torch.zeros(2, dtype=torch.int32))
    with pytest.raises(ValueError, match="weight has 3 dimensions"):
        binding.moe_fp8_linear_backward(x.bfloat16(), weight[None], scales)
