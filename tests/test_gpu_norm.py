"""The norm ahead of the layer (moe_rms_norm, moe_rms_norm_fp8) and its gradients, and rows in
8 bits (moe_fp8_quantize), against the float64 oracle.

u = 2^-24 is half a step of fp32.  A sum of a row goes through at most 64 additions of a
lane, 6 of a wave's tree and 16 of a block's waves, so it is off by at most 86 u of its
terms' magnitudes; the norm's factor r = 1 / sqrt(sum / H + eps) by half of that and
4 u, and a product with it by 2 u more: 64 u in all are allowed.  The gradient's dot
product has 2 u more a term and multiplies r three times: 160 u.  A sum over T rows: T u
and what each term has.
"""

import ctypes

import numpy as np
import pytest
import torch

from oracle import layer_ops as L
from tests.op_helpers import TYPES, U, assert_codes_near, assert_near, bytes_of, f64, normal

pytestmark = pytest.mark.gpu

SHAPES = [(1, 1), (3, 7), (4, 8), (5, 127), (2, 128), (9, 129), (4, 2880), (1, 1001), (33, 512), (1030, 264),
          (1025, 1003), (1024, 4096), (3, 4104), (1100, 8200), (2, 16384), (3, 20001), (1, 32768), (1027, 2050)]


@pytest.mark.parametrize("dtype", TYPES, ids=str)
@pytest.mark.parametrize("T,H", SHAPES)
def test_norm_and_gradients(gpu, T, H, dtype):
    print(f"[norm] {T} x {H} {dtype}", flush=True)
    x, res = normal(1, T, H, dtype=dtype), normal(2, T, H, dtype=dtype, scale=3.0)
    dy, ds = normal(3, T, H, dtype=dtype), normal(4, T, H, dtype=dtype)
    eps = 1e-5
    for wtype, residual, stream_grad in ((dtype, res, ds), (torch.float32, None, None)):
        w = (1 + 0.3 * normal(5, H)).to(wtype)
        y, s, r = gpu.moe_rms_norm(x, w, residual, eps)
        codes, scales, s8, r8 = gpu.moe_rms_norm_fp8(x, w, residual, eps)
        if residual is None:
            assert s is x and s8 is x
        else:
            assert_near(s, f64(x) + f64(residual), U * (np.abs(f64(x)) + np.abs(f64(residual))), dtype, "s")
            assert torch.equal(s, s8)
        assert torch.equal(r, r8)
        want, factor = L.rms_norm(f64(s), f64(w), eps)
        assert_near(r, factor, 64 * U * factor, torch.float32, "rstd")
        assert_near(y, want, 64 * U * np.abs(want), dtype, "y")
        assert codes.dtype == torch.float8_e4m3fn and scales.shape == (T, L.blocks(H))
        assert_codes_near(codes, scales, want, 64 * U)
        dx, dw = gpu.moe_rms_norm_backward(dy, s, w, r, stream_grad)
        d, mag, wsum, wmag = L.rms_norm_backward(f64(dy), f64(s), f64(w), eps,
                                                 None if stream_grad is None else f64(stream_grad))
        assert dx.dtype == dtype and dw.dtype == torch.float32
        assert_near(dx, d, 160 * U * mag, dtype, "dx")
        assert_near(dw, wsum, (T + 80) * U * wmag, torch.float32, "d_weight")
        again = gpu.moe_rms_norm_backward(dy, s, w, r, stream_grad)
        assert torch.equal(again[0], dx) and torch.equal(again[1], dw)


def test_rows_at_any_element(gpu):
    """Slices of a buffer that start at an odd element, and outputs that do."""
    T, H = 5, 387
    flat, out = normal(1, T * H + 3, dtype=torch.bfloat16), torch.zeros(T * H + 3, device="cuda", dtype=torch.bfloat16)
    bytes_, w = torch.zeros(T * H + 5, device="cuda", dtype=torch.uint8), normal(2, H + 1, dtype=torch.bfloat16)[1:]
    x = flat[3:].view(T, H)
    y, _, r = gpu.moe_rms_norm(x, w, out=out[3:].view(T, H))
    base = gpu.moe_rms_norm(x.clone(), w.clone())
    assert torch.equal(y, base[0]) and torch.equal(r, base[2]) and torch.all(out[:3] == 0)
    codes, scales, _, _ = gpu.moe_rms_norm_fp8(x, w, codes=bytes_[5:].view(T, H).view(torch.float8_e4m3fn))
    want = gpu.moe_rms_norm_fp8(x.clone(), w.clone())
    assert torch.equal(codes.view(torch.uint8), want[0].view(torch.uint8)) and torch.equal(scales, want[1])
    assert torch.all(bytes_[:5] == 0)


def test_no_rows(gpu):
    x, w = torch.zeros((0, 40), device="cuda"), torch.ones(40, device="cuda")
    y, s, r = gpu.moe_rms_norm(x, w, x)
    assert y.shape == (0, 40) and r.shape == (0,)
    dx, dw = gpu.moe_rms_norm_backward(x, s, w, r)
    assert dx.shape == (0, 40) and torch.equal(dw, torch.zeros_like(w))
    codes, scales = gpu.moe_fp8_quantize(x)
    assert codes.shape == (0, 40) and scales.shape == (0, 1)


def test_zeros_and_extremes(gpu):
    w = torch.ones(300, device="cuda")
    x = torch.zeros((4, 300), device="cuda")
    x[1] = 1e-30
    x[2] = 1e18
    x[3, 5] = float("nan")
    y, _, r = gpu.moe_rms_norm(x, w, eps=1e-6)
    assert torch.all(y[0] == 0) and torch.all(torch.isnan(y[3])) and torch.isnan(r[3])
    assert torch.allclose(y[2], torch.ones(300, device="cuda")) and torch.allclose(y[1], x[1] * 1e3)
    codes, scales, _, _ = gpu.moe_rms_norm_fp8(x, w, eps=1e-6)
    assert torch.all(codes[0].float() == 0) and torch.all(torch.isnan(scales[3]))
    zero = gpu.moe_rms_norm(x[:1], w, eps=0.0)[0]
    assert torch.all(torch.isnan(zero))  # 0 / 0, as the formula has it


def quantized(v):
    """moe_fp8_quantize in fp32 steps on the host: IEEE operations alone, so the same bits."""
    rows, width = v.shape
    scales = np.zeros((rows, L.blocks(width)), np.float32)
    codes = np.zeros((rows, width), np.uint8)
    with np.errstate(all="ignore"):
        for j in range(scales.shape[1]):
            part = v[:, 128 * j: 128 * (j + 1)]
            largest = np.maximum(np.max(np.abs(part), axis=1), np.float32(2.0 ** -100))  # (NaN stays NaN)
            scales[:, j] = largest / np.float32(448)
            up = part * (np.float32(448) / largest)[:, None]
            codes[:, 128 * j: 128 * (j + 1)] = torch.from_numpy(up).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    return codes, scales


def assert_same_codes(got, want):
    nan = (want & 127) == 127
    assert np.array_equal((got & 127) == 127, nan) and np.array_equal(got[~nan], want[~nan])


@pytest.mark.parametrize("dtype", TYPES, ids=str)
@pytest.mark.parametrize("R,K", [(1, 1), (3, 8), (2, 127), (17, 128), (5, 129), (4, 2880), (700, 1001), (2049, 96)])
def test_quantize_to_the_bit(gpu, R, K, dtype):
    x = normal(R + K, R, K, dtype=dtype)
    x *= torch.exp2(torch.randint(-12, 9, (R, 1), device="cuda")).to(dtype)
    codes, scales = gpu.moe_fp8_quantize(x)
    want, s = quantized(x.float().cpu().numpy())
    assert np.array_equal(scales.cpu().numpy(), s)
    assert_same_codes(bytes_of(codes), want)


def test_quantize_every_code_and_tie(gpu):
    """A block whose largest is 448 has scale 1: every code comes back, every middle between two
    goes to the even one, and the smallest values round to zero or the first subnormal."""
    v = np.sort(L.E4M3[:127])
    mid = (v[1:] + v[:-1]) / 2
    vals = np.concatenate([v, mid, np.nextafter(mid, 0), np.nextafter(mid, 1e9), [2.0 ** -10, 2.0 ** -11, 1e-30]])
    vals = np.concatenate([vals, -vals]).astype(np.float32)
    rows = np.zeros((len(vals) // 127 + 1, 128), np.float32)
    rows[:, 0] = 448
    rows[:, 1:].flat[: len(vals)] = vals
    codes, scales = gpu.moe_fp8_quantize(torch.from_numpy(rows).cuda())
    assert torch.all(scales == 1)
    assert_same_codes(bytes_of(codes), torch.from_numpy(rows).to(torch.float8_e4m3fn).view(torch.uint8).numpy())


def test_quantize_infinity_nan_zero_and_tiny(gpu):
    x = torch.ones((6, 256), device="cuda")
    x[0, 7], x[1, 200], x[2] = float("inf"), float("nan"), 0.0
    x[3], x[4, :128] = 1e-38, 2.0 ** -101
    x[5, 3] = 3e38
    codes, scales = gpu.moe_fp8_quantize(x)
    want, s = quantized(x.cpu().numpy())
    assert np.array_equal(scales.cpu().numpy(), s, equal_nan=True)
    assert_same_codes(bytes_of(codes), want)
    c = codes.float()
    assert torch.isnan(c[0, 7]) and c[0, 8] == 0 and torch.isinf(scales[0, 0]) and scales[0, 1] == 1 / 448
    assert torch.all(torch.isnan(c[1, 128:])) and torch.all(c[2] == 0) and torch.all(c[3] == 0)


@pytest.mark.parametrize("H", [5, 300, 1001, 1500, 2050, 9001, 20001])
def test_norm_to_8_bits_is_the_norm_then_the_quantizer(gpu, H):
    """To the bit, in every form of the kernel, also where r is infinite (eps = 0 and squares that
    underflow): what lies behind a row's end has no part in its last block."""
    x, w = normal(H, 5, H), 1 + 0.3 * normal(1, H)
    x[1], x[2, -1], x[3, 0] = 1e-30, 1e19, float("inf")
    for eps in (1e-5, 0.0):
        y, _, r = gpu.moe_rms_norm(x, w, eps=eps)
        assert torch.isinf(r[1]) == (eps == 0.0)
        codes, scales, _, _ = gpu.moe_rms_norm_fp8(x, w, eps=eps)
        want, s = gpu.moe_fp8_quantize(y)
        assert np.array_equal(scales.cpu().numpy(), s.cpu().numpy(), equal_nan=True)
        assert_same_codes(bytes_of(codes), bytes_of(want))


def test_streams_and_graph(gpu):
    """Two streams at once, a stream passed in, and a captured step replayed on other inputs."""
    T, H = 600, 2880
    w = 1 + 0.1 * normal(0, H, dtype=torch.bfloat16)
    x, res, dy = (normal(i, T, H, dtype=torch.bfloat16) for i in (1, 2, 3))

    def step(a, b, **kw):
        y, s, r = gpu.moe_rms_norm(a, w, b, **kw)
        c, sc, _, _ = gpu.moe_rms_norm_fp8(a, w, b, **kw)
        return [y, s, r, c.view(torch.uint8), sc, *gpu.moe_rms_norm_backward(dy, s, w, r, a, **kw)]

    want, swapped = step(x, res), step(res, x)
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(3):
        got1, got2 = step(x, res, stream=s1), step(res, x, stream=s2)
    torch.cuda.synchronize()
    for a, b in zip(want + swapped, got1 + got2):
        assert torch.equal(a, b)

    a, b = x.clone(), res.clone()
    with torch.cuda.stream(s1):
        step(a, b)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = step(a, b)
    for i in range(4):
        first, second = (x, res) if i % 2 == 0 else (res, x)
        a.copy_(first)
        b.copy_(second)
        g.replay()
        eager = step(first, second)
        torch.cuda.synchronize()
        for p, q in zip(out, eager):
            assert torch.equal(p, q)


def test_refusals_of_the_binding(gpu):
    x, w = torch.zeros((4, 64), device="cuda"), torch.ones(64, device="cuda")
    with pytest.raises(ValueError, match="contiguous"):
        gpu.moe_rms_norm(x.t(), torch.ones(4, device="cuda"))
    with pytest.raises(ValueError, match="shape"):
        gpu.moe_rms_norm(x, w[:63])
    with pytest.raises(TypeError):
        gpu.moe_rms_norm(x, w.bfloat16())
    with pytest.raises(TypeError):
        gpu.moe_rms_norm(x, w, x.bfloat16())
    with pytest.raises(ValueError, match="shares memory"):
        gpu.moe_rms_norm(x, w, out=x)
    with pytest.raises(ValueError, match="only with a residual"):
        gpu.moe_rms_norm(x, w, summed=torch.empty_like(x))
    with pytest.raises(gpu.MXFP4MoEError):
        gpu.moe_rms_norm(x, w, eps=-1.0)
    with pytest.raises(gpu.MXFP4MoEError):
        gpu.moe_rms_norm(torch.zeros((1, 32769), device="cuda"), torch.zeros(32769, device="cuda"))
    with pytest.raises(ValueError, match="shape"):
        gpu.moe_rms_norm_backward(x, x, w, torch.ones(5, device="cuda"))
    with pytest.raises(ValueError, match="shares memory"):
        gpu.moe_rms_norm_backward(x, x.clone(), w, torch.ones(4, device="cuda"), dx=x)
    n = ctypes.c_size_t(0)
    f = gpu.load().moe_rms_norm_backward
    args = [x.data_ptr(), None, x.data_ptr(), w.data_ptr(), 2, 2, x.data_ptr(), 4, 64, x.data_ptr(), w.data_ptr()]
    assert f(*args, x.data_ptr(), ctypes.byref(n), None) == -3


@pytest.mark.parametrize("dtype", TYPES, ids=str)
def test_several_wide_rows_a_block(gpu, dtype):
    """Sixteen waves a row, more rows than the gradient's launch has blocks."""
    test_norm_and_gradients(gpu, 1030, 16500, dtype)
