"""More rows than a launch of the norm (2^20 blocks), of the activation and of the quantizer (2^22) has
blocks for: the loops past that, against the same rows in calls that need none."""

import pytest
import torch

from tests.op_helpers import bytes_of

pytestmark = pytest.mark.gpu


def rows_of(R, width, seed):
    return torch.randn((R, width), device="cuda", dtype=torch.bfloat16, generator=torch.Generator("cuda").manual_seed(seed))


def pieces(R):
    """The first rows, and the last ones, which the launch's blocks come to in their second round."""
    return slice(0, 1000), slice(R - 1000, R)


@pytest.mark.parametrize("T,H", [(4 * 2 ** 20 + 37, 8), (2 ** 20 + 501, 1032)])  # four rows a block, and one
def test_norm(gpu, T, H):
    x, res, w = rows_of(T, H, 1), rows_of(T, H, 2), rows_of(1, H, 3)[0].contiguous()
    y, s, r = gpu.moe_rms_norm(x, w, res)
    for p in pieces(T):
        a = gpu.moe_rms_norm(x[p], w, res[p])
        assert torch.equal(y[p], a[0]) and torch.equal(s[p], a[1]) and torch.equal(r[p], a[2])
    del y, s
    codes, scales, s, r = gpu.moe_rms_norm_fp8(x, w, res)
    for p in pieces(T):
        a = gpu.moe_rms_norm_fp8(x[p], w, res[p])
        assert (bytes_of(codes[p]) == bytes_of(a[0])).all() and torch.equal(scales[p], a[1])
        assert torch.equal(s[p], a[2]) and torch.equal(r[p], a[3])


@pytest.mark.parametrize("split", [False, True])
def test_activation(gpu, split):
    R = 2 ** 26 + 555
    h, da = rows_of(R, 2, 1), rows_of(R, 1, 2)
    a, dh = gpu.moe_swiglu(h, split), gpu.moe_swiglu_backward(da, h, split)
    codes, scales = gpu.moe_swiglu_fp8(h, split)
    for p in pieces(R):
        assert torch.equal(a[p], gpu.moe_swiglu(h[p], split))
        assert torch.equal(dh[p], gpu.moe_swiglu_backward(da[p], h[p], split))
        c, s = gpu.moe_swiglu_fp8(h[p], split)
        assert (bytes_of(codes[p]) == bytes_of(c)).all() and torch.equal(scales[p], s)


def test_quantizer(gpu):
    R = 2 ** 26 + 555
    x = rows_of(R, 1, 1)
    codes, scales = gpu.moe_fp8_quantize(x)
    for p in pieces(R):
        c, s = gpu.moe_fp8_quantize(x[p])
        assert (bytes_of(codes[p]) == bytes_of(c)).all() and torch.equal(scales[p], s)
