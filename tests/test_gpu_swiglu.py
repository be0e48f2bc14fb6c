"""The experts' activation (moe_swiglu, moe_swiglu_fp8) and its gradient against the float64 oracle.

The sigmoid is 1 / (1 + 2^x), x = -alpha log2(e) g.  x is off by two roundings, 2^x
relatively by ln 2 times that and one step of the instruction, the reciprocal by one
step more: (1.4 |x| + 4) half steps u = 2^-24 of the sigmoid with the sum, 8 with the
products around it; 1 - sigmoid by as much of the sigmoid.
"""

import math

import numpy as np
import pytest
import torch

from oracle import layer_ops as L
from tests.op_helpers import TYPES, U, assert_codes_near, assert_near, f64, normal

pytestmark = pytest.mark.gpu

SHAPES = [(1, 1), (3, 5), (16, 2880), (2, 127), (5, 128), (7, 129), (300, 136), (33, 1001), (4100, 96), (1, 4096)]
CONSTANTS = [(1.702, 7.0, 1.0), (1.0, math.inf, 0.0), (0.9, 1.5, -0.25)]
LEAST = 2.0 ** -120  # results below come from a sigmoid under the smallest normal number


def rel(h, split, alpha, limit):
    g = np.minimum(L.halves(h, split)[0], limit)
    return (1.4 * np.abs(alpha * 1.4427 * g) + 12) * U


@pytest.mark.parametrize("dtype", TYPES, ids=str)
@pytest.mark.parametrize("split", [False, True])
@pytest.mark.parametrize("R,I", SHAPES)
def test_swiglu_and_gradient(gpu, R, I, split, dtype):
    alpha, limit, offset = CONSTANTS[(R + I) % 3]
    print(f"[swiglu] {R} x {I} {dtype} {alpha} {limit} {offset}", flush=True)
    h, da = normal(1, R, 2 * I, dtype=dtype, scale=4.0), normal(2, R, I, dtype=dtype)
    kw = dict(split=split, alpha=alpha, limit=limit, offset=offset)
    h64 = f64(h)
    want, r = L.swiglu(h64, split, alpha, limit, offset), rel(h64, split, alpha, limit)
    a = gpu.moe_swiglu(h, **kw)
    assert a.dtype == dtype
    assert_near(a, want, r * np.abs(want) + LEAST, dtype, "a")
    codes, scales = gpu.moe_swiglu_fp8(h, **kw)
    assert_codes_near(codes, scales, want, r.max() if r.size else 0.0)
    dh = gpu.moe_swiglu_backward(da, h, **kw)
    d, mag = L.swiglu_backward(f64(da), h64, split, alpha, limit, offset)
    wide = np.zeros_like(h64)
    for part in L.halves(wide, split):
        part[...] = r
    assert_near(dh, d, 2 * wide * mag + LEAST, dtype, "dh")


def test_defaults_are_the_layers(gpu):
    h = normal(1, 9, 96, dtype=torch.bfloat16, scale=6.0)
    assert_near(gpu.moe_swiglu(h), L.swiglu(f64(h), False, 1.702, 7.0, 1.0), 64 * U * 60, torch.bfloat16)
    assert torch.equal(gpu.moe_swiglu(h), gpu.moe_swiglu(h, False, 1.702, 7.0, 1.0))


def test_limits_and_special_values(gpu):
    inf, nan = math.inf, math.nan
    gates = [7.0, 7.0625, -100.0, inf, -inf, nan, 1.0, 1.0, 1.0, 1.0]
    ups = [1.0, 1.0, 1.0, 1.0, 0.0, 1.0, 7.0, 7.0625, -inf, nan]
    h = torch.tensor([v for p in zip(gates, ups) for v in p], device="cuda")[None]
    a, da = gpu.moe_swiglu(h)[0], torch.ones((1, 10), device="cuda")
    dh = gpu.moe_swiglu_backward(da, h)[0].view(10, 2)
    assert a[0] == a[1] == a[3] and a[2].abs() < 1e-30 and torch.isnan(a[5]) and a[6] == a[7] and torch.isnan(a[9])
    assert a[8] == -6 * a[6] / 8
    # a limit itself still has a slope, what lies past it none
    assert dh[0, 0] != 0 and torch.all(dh[[1, 3], 0] == 0) and dh[6, 1] != 0 and torch.all(dh[7:9, 1] == 0)


@pytest.mark.parametrize("dtype", TYPES, ids=str)
@pytest.mark.parametrize("split", [False, True])
@pytest.mark.parametrize("alpha,limit,offset", [(1.702, 7.0, 1.0), (1.702, math.inf, 0.0), (-3.0, math.inf, 0.5)])
def test_gradient_of_the_largest_and_smallest_gates(gpu, dtype, split, alpha, limit, offset):
    """Where alpha * gate overflows, the sigmoid is 0 or 1 and the gradient what the formula has there."""
    lo, hi = torch.finfo(dtype).min, torch.finfo(dtype).max
    gates = torch.tensor([lo, hi, lo / 2, hi / 2, lo, hi, -200.0, 200.0, -1.0, 0.0], dtype=dtype, device="cuda")
    ups = torch.tensor([0.5, 0.5, -2.0, 3.0, 0.0, 0.0, 1.0, 1.0, 2.0, 2.0], dtype=dtype, device="cuda")
    h = torch.stack([gates, ups], 0 if split else 1).reshape(1, -1)
    da = torch.full((1, 10), 0.5, dtype=dtype, device="cuda")
    dh = gpu.moe_swiglu_backward(da, h, split, alpha, limit, offset)
    want, mag = L.swiglu_backward(f64(da), f64(h), split, alpha, limit, offset)
    # past |alpha gate| = 128 the sigmoid is 0 or 1 in fp32 and its slope 0: the products' roundings alone are left
    x, bound = np.abs(alpha * np.minimum(f64(gates), limit)), np.zeros_like(want)
    for part, m, v in zip(L.halves(bound, split), L.halves(mag, split), L.halves(np.abs(want), split)):
        part[...] = np.where(x <= 128, 2 * (1.4 * 1.4427 * x + 12) * m, 12 * v) * U
    assert_near(dh, want, bound + LEAST, dtype, "dh")


def test_rows_at_any_element(gpu):
    R, I = 6, 261
    flat, da = normal(1, R * 2 * I + 1, dtype=torch.float16), normal(2, R * I + 1, dtype=torch.float16)
    h, d = flat[1:].view(R, 2 * I), da[1:].view(R, I)
    for split in (False, True):
        assert torch.equal(gpu.moe_swiglu(h, split), gpu.moe_swiglu(h.clone(), split))
        assert torch.equal(gpu.moe_swiglu_backward(d, h, split), gpu.moe_swiglu_backward(d.clone(), h.clone(), split))
        a, b = gpu.moe_swiglu_fp8(h, split), gpu.moe_swiglu_fp8(h.clone(), split)
        assert torch.equal(a[0].view(torch.uint8), b[0].view(torch.uint8)) and torch.equal(a[1], b[1])


def test_no_rows_outputs_and_refusals(gpu):
    e = torch.zeros((0, 20), device="cuda")
    assert gpu.moe_swiglu(e).shape == (0, 10) and gpu.moe_swiglu_backward(e[:, :10], e).shape == (0, 20)
    h = normal(1, 3, 20)
    out = torch.empty((3, 10), device="cuda")
    assert gpu.moe_swiglu(h, out=out).data_ptr() == out.data_ptr() and torch.equal(out, gpu.moe_swiglu(h))
    with pytest.raises(ValueError, match="shares memory"):
        gpu.moe_swiglu(h, out=h.view(-1)[:30].view(3, 10))
    with pytest.raises(ValueError, match="shape"):
        gpu.moe_swiglu_backward(h, h)
    with pytest.raises(TypeError):
        gpu.moe_swiglu_backward(out.half(), h)
    with pytest.raises(gpu.MXFP4MoEError):
        gpu.moe_swiglu(h, limit=0.0)
    with pytest.raises(gpu.MXFP4MoEError):
        gpu.moe_swiglu(h, alpha=math.nan)
