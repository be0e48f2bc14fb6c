"""The kernels of the 8-bit products with tiles in LDS, at sizes where the choice of kernel
(csrc/fp8_plan.h) takes them: what test_gpu_fp8_linear.py asks of small calls, which have kernels of
their own.  Each test names the kernels that it is for and asserts that its sizes reach them."""

import numpy as np
import pytest
import torch

from oracle import expert_ops as X
from oracle import layer_ops as L
from tests.op_helpers import bytes_of, f64, normal
from tests.test_fp8_plan import plan  # noqa: F401  (a fixture)
from tests.test_gpu_fp8_linear import (E4M3, Weights, assert_sums, check_both, largest_of_eights, offsets_of, random_codes)
from tests.test_gpu_fp8_linear import test_a_layer_of_8_bit_experts as check_layer

pytestmark = pytest.mark.gpu


def reaches(plan, R, N, K, E, tile, gradient=True):  # noqa: F811
    assert plan.choice(R, N, E) == (False, *tile)
    assert not gradient or not plan.backward_few(R, K, E)


# R, N, K, E of equal shares, the product's tile
NAN = [(1100, 1100, 1040, 1, (64, 128)), (1400, 1100, 1040, 2, (64, 128)), (1900, 1100, 1040, 4, (64, 256)),
       (2800, 1500, 528, 4, (128, 256)), (2100, 2600, 528, 1, (128, 256)), (1000, 1000, 1040, 1, (32, 128))]


@pytest.mark.parametrize("R,N,K,E,tile", NAN)
def test_nan_codes_stay_in_their_places(gpu, plan, R, N, K, E, tile):  # noqa: F811
    """A NaN weight reaches its output column (its k in the gradient) of its expert's rows, a NaN in a
    row that row.  A wave of the gradient reads past K into the next weight row, one of the product
    past its rows into zeros: neither reaches an output."""
    reaches(plan, R, N, K, E, tile)
    part, rng = R // E, np.random.default_rng(1)
    off = offsets_of([part] * E) if E > 1 else None
    x, xs = random_codes(rng, R, K), torch.ones((R, L.blocks(K)), device="cuda")
    dy = normal(1, R, N, dtype=torch.bfloat16)
    e = E - 1
    rows = slice(e * part, (e + 1) * part)
    for n, k in ((5, 7), (6, 0), (N - 1, K - 1), (64, K - 1), (0, 0), (N - 1, 0)):
        w = Weights(E, N, K, seed=3, dense=E == 1)
        w.codes.view(torch.uint8).view(E, N, K)[e, n, k] = 0xFF
        y = gpu.moe_fp8_linear(x, xs, w.codes, w.scales, None, off)
        bad = torch.zeros_like(y, dtype=torch.bool)
        bad[rows, n] = True
        assert torch.equal(torch.isnan(y), bad), (n, k)
        dx = gpu.moe_fp8_linear_backward(dy, w.codes, w.scales, off)
        bad = torch.zeros_like(dx, dtype=torch.bool)
        bad[rows, k] = True
        assert torch.equal(torch.isnan(dx), bad), (n, k)
    w = Weights(E, N, K, seed=3, dense=E == 1)
    for r in (0, part - 1, R - 1):
        x2, dy2 = x.clone(), dy.clone()
        x2.view(torch.uint8)[r, K - 1], dy2[r, N - 1] = 0x7F, float("nan")
        bad = torch.zeros(R, dtype=torch.bool, device="cuda")
        bad[r] = True
        y, dx = gpu.moe_fp8_linear(x2, xs, w.codes, w.scales, None, off), gpu.moe_fp8_linear_backward(dy2, w.codes, w.scales, off)
        for got in (y, dx):
            assert torch.equal(torch.isnan(got), bad[:, None].expand(got.shape))


@pytest.mark.parametrize("R,tile", [(2500, (32, 128)), (5000, (64, 128)), (10000, (64, 256)), (20000, (128, 256))])
def test_every_code_is_exact(gpu, plan, R, tile):  # noqa: F811
    """One product an output: each pair of codes, and each code with dy, comes out rounded once."""
    reaches(plan, R, 256, 256, 1, tile, R > 4096)
    codes = torch.arange(256, dtype=torch.uint8, device="cuda")
    eye = torch.zeros((256, 256), dtype=torch.uint8, device="cuda")
    eye[torch.arange(256), torch.arange(256)] = codes
    eye[127, 127] = eye[255, 255] = 0  # the NaN codes have a test of their own
    w, s = eye.view(E4M3), torch.ones((2, 2), device="cuda")
    x = torch.randint(0, 127, (R, 256), dtype=torch.uint8, device="cuda", generator=torch.Generator("cuda").manual_seed(1)).view(E4M3)
    v = torch.where((codes & 127) == 127, 0.0, codes.view(E4M3).float())
    assert torch.equal(gpu.moe_fp8_linear(x, torch.ones((R, 2), device="cuda"), w, s), (x.float() * v).bfloat16())
    dy = normal(2, R, 256, dtype=torch.bfloat16)
    assert torch.equal(gpu.moe_fp8_linear_backward(dy, w, s), (dy.float() * v).bfloat16())


def uneven(E, R, seed):
    """Counts of R rows: empty experts and a large one on both sides of the 64th, the first and the last empty."""
    rng = np.random.default_rng(seed)
    share = rng.dirichlet(np.full(E, 1.5))
    share[[0, 3, 62, 63, 64, E - 1]] = 0
    share[[20, E - 20]] += 0.05
    return rng.multinomial(R, share / share.sum())


@pytest.mark.parametrize("E,R,N,K,tile", [(200, 700, 400, 272, (64, 128)), (200, 4000, 300, 272, (64, 256)),
                                          (200, 13000, 300, 144, (128, 256)), (130, 9000, 264, 272, (128, 256)),
                                          (512, 3000, 264, 144, (64, 256)), (65, 1000, 1100, 528, (64, 256))])
def test_more_experts_than_a_wave_has_lanes(gpu, plan, E, R, N, K, tile):  # noqa: F811
    reaches(plan, R, N, K, E, tile)
    check_both(gpu, Weights(E, N, K, seed=E), R, offsets_of(uneven(E, R, R)), label=f"{E} experts")


@pytest.mark.parametrize("counts,R,first,N,K,tile", [
    ([300, 0, 450], 900, 37, 1100, 656, (64, 128)), ([0, 0, 0], 900, 4, 1100, 656, (64, 128)),
    ([700, 0, 33, 900, 5], 1900, 129, 2600, 272, (128, 256)), ([64, 640], 720, 3, 1000, 720, (32, 128)),
    ([5] * 70 + [0] * 30 + [9] * 50, 1200, 111, 500, 400, (64, 256))])
def test_rows_of_no_expert_are_left(gpu, plan, counts, R, first, N, K, tile):  # noqa: F811
    """A rank's share: rows before the first and from the last offset on keep what they held."""
    reaches(plan, R, N, K, len(counts), tile)
    check_both(gpu, Weights(len(counts), N, K), R, offsets_of(counts, first), label="share")


@pytest.mark.parametrize("R,N,K,tile", [(1200, 1100, 528, (64, 128)), (2800, 1500, 144, (128, 256))])
def test_offsets_past_the_rows_are_clamped(gpu, plan, R, N, K, tile):  # noqa: F811
    reaches(plan, R, N, K, 3, tile)
    w = Weights(3, N, K)
    off = torch.tensor([-5, R // 3, R - 7, 1 << 30], dtype=torch.int32, device="cuda")
    bounds = np.array([0, R // 3, R - 7, R])
    x, xs, dy = random_codes(np.random.default_rng(0), R, K), torch.ones((R, L.blocks(K)), device="cuda"), normal(1, R, N, dtype=torch.bfloat16)
    x64, w64 = L.values(bytes_of(x), f64(xs)), w.f64
    want, mag, _ = X.linear(x64, w64, bounds, None)
    assert_sums(gpu.moe_fp8_linear(x, xs, w.codes, w.scales, None, off), want, mag, K, "clamped", largest_of_eights(x64, w64, bounds))
    want, mag, _ = X.linear_backward(f64(dy), w64, bounds)
    assert_sums(gpu.moe_fp8_linear_backward(dy, w.codes, w.scales, off), want, mag, N, "clamped dx")


@pytest.mark.parametrize("counts,N,K,tile", [([500, 0, 200, 800], 1300, 656, (64, 256)), ([9] * 90, 800, 400, (64, 256)),
                                             ([700, 800, 750, 700], 1500, 400, (128, 256))])
def test_same_bits_on_streams_and_in_a_graph(gpu, plan, counts, N, K, tile):  # noqa: F811
    R, E = sum(counts), len(counts)
    reaches(plan, R, N, K, E, tile)
    w, off = Weights(E, N, K, seed=1), offsets_of(counts)
    x, x2 = normal(1, R, K, dtype=torch.bfloat16), normal(2, R, K, dtype=torch.bfloat16)

    def step(v, **kw):
        c, s = gpu.moe_fp8_quantize(v, **kw)
        y = gpu.moe_fp8_linear(c, s, w.codes, w.scales, w.bias, off, **kw)
        return [y, gpu.moe_fp8_linear_backward(y, w.codes, w.scales, off, **kw)]

    want, other = step(x), step(x2)
    assert not torch.equal(want[0], other[0])
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(5):
        got, got2 = step(x, stream=s1), step(x2, stream=s2)
    torch.cuda.synchronize()
    for a, b in zip(want + other, got + got2):
        assert torch.equal(a, b)
    v = x.clone()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = step(v)
    for i in range(4):
        v.copy_(x if i % 2 else x2)
        g.replay()
        step(x if i % 2 else x2)
        torch.cuda.synchronize()
        for a, b in zip(out, want if i % 2 else other):
            assert torch.equal(a, b)


def test_a_layer_of_8_bit_experts(gpu, plan):  # noqa: F811
    """All steps together, with as many rows an expert as take the tiles."""
    reaches(plan, 12000, 288, 256, 6, (128, 256))
    reaches(plan, 12000, 256, 144, 6, (64, 256))
    check_layer(gpu, 6000)
