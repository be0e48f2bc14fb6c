"""Rows in 8 bits times 8-bit weights with a scale for each block of 128, dense and per expert, and
the gradient to the rows (moe_fp8_linear, moe_fp8_linear_backward) against the float64 oracle, and
runs of the operators as a layer of 8-bit experts makes them.

Every product is exact, so a sum of n terms with its blocks' scales (two roundings each), the
bias and the addition of K parts is off by at most (n + 8) * 2^-23 of the sum of the terms'
magnitudes (one step of fp32 an addition, whichever way the matrix core rounds), then the
result is rounded once to bf16 (half a step, 2^-8 relative).

The FP8 matrix instruction adds eight neighbouring products as integers, in steps of 2^-13 of
the power of two of the largest, and cuts off what lies below: 65536 + 7 * 4 gives 65536 where the
eight are neighbours and 65564 where they are not, 65536 + 8 gives 65544.  So each of eight
products loses less than 2^-13 of the largest of them, and the largest itself nothing that is not
in its own eight bits (two codes of four): 7 * 2^-13 of the largest, summed over the eights.  The
gradient's bf16 instruction adds exact products in fp32.
"""

import numpy as np
import pytest
import torch

from oracle import expert_ops as X
from oracle import layer_ops as L
from tests.op_helpers import bytes_of, f64, normal

pytestmark = pytest.mark.gpu

BF16 = torch.finfo(torch.bfloat16)
E4M3 = torch.float8_e4m3fn


def random_codes(rng, *shape):
    """Every code but the two NaN."""
    b = rng.integers(0, 254, shape, dtype=np.uint8)
    return torch.from_numpy(np.where(b >= 127, b + 1, b)).cuda().view(E4M3)


class Weights:
    def __init__(self, E, N, K, seed=0, dense=False):
        rng = np.random.default_rng(seed)
        lead = () if dense else (E,)
        self.codes = random_codes(rng, *lead, N, K)
        self.scales = torch.from_numpy(rng.uniform(0.5, 2, (*lead, L.blocks(N), L.blocks(K))).astype(np.float32)).cuda()
        self.bias = torch.from_numpy(rng.standard_normal((*lead, N)).astype(np.float32) * 100).bfloat16().cuda()

    @property
    def f64(self):
        return L.weights(bytes_of(self.codes), f64(self.scales))


def offsets_of(counts, first=0):
    return torch.tensor(np.concatenate([[first], first + np.cumsum(counts)]).astype(np.int32)).cuda()


def largest_of_eights(x, w, off):
    """Sum over the eights of k of the largest product, for every output."""
    out = np.zeros((x.shape[0], w.shape[-2]))
    bounds = [0, len(x)] if off is None else np.clip(off, 0, len(x))
    for e, (a, b) in enumerate(zip(bounds, bounds[1:])):
        p = torch.from_numpy(np.abs(x[a:b])).cuda()
        q = torch.from_numpy(np.abs(w if w.ndim == 2 else w[e])).cuda()
        total = torch.zeros((len(p), len(q)), dtype=torch.float64, device="cuda")
        for k in range(0, x.shape[1], 8):
            most = torch.zeros_like(total)
            for j in range(k, min(k + 8, x.shape[1])):
                torch.maximum(most, p[:, j, None] * q[None, :, j], out=most)
            total += most
        out[a:b] = total.cpu().numpy()
    return out


def assert_sums(got, want, mag, terms, label, cut=0.0):
    slack = (terms + 8) * 2.0 ** -23 * mag + 7 * 2.0 ** -13 * cut
    bound = slack + (np.abs(want) + slack) * BF16.eps / 2 + BF16.tiny * BF16.eps / 2
    g = f64(got)
    assert np.all(np.isfinite(g)), f"{label}: {np.argwhere(~np.isfinite(g))[:4].tolist()} not finite"
    off = np.abs(g - want) - bound
    assert off.size == 0 or off.max() <= 0, \
        f"{label}: {off.max():.3e} over its bound, first at {np.argwhere(off > 0)[:4].tolist()} of {off.shape}"


def check_both(gpu, w, R, offsets=None, bias=True, seed=1, label=""):
    rng = np.random.default_rng(seed)
    N, K = w.codes.shape[-2:]
    x, dy = random_codes(rng, R, K), normal(seed, R, N, dtype=torch.bfloat16)
    xs = torch.from_numpy(rng.uniform(0.5, 2, (R, L.blocks(K))).astype(np.float32)).cuda()
    off = None if offsets is None else offsets.cpu().numpy()
    w64 = w.f64
    print(f"[fp8 linear] {label} R={R} N={N} K={K}", flush=True)
    for forward in (True, False):
        out = torch.full((R, N if forward else K), 7.0, dtype=torch.bfloat16, device="cuda")
        if forward:
            x64 = L.values(bytes_of(x), f64(xs))
            want, mag, written = X.linear(x64, w64, off, f64(w.bias) if bias else None)
            cut = largest_of_eights(x64, w64, off)
            got = gpu.moe_fp8_linear(x, xs, w.codes, w.scales, w.bias if bias else None, offsets, out=out)
        else:
            want, mag, written = X.linear_backward(f64(dy), w64, off)
            cut = np.zeros_like(want)
            got = gpu.moe_fp8_linear_backward(dy, w.codes, w.scales, offsets, out=out)
        assert got.data_ptr() == out.data_ptr()
        want[~written] = 7.0  # rows of no expert keep what they held
        mag[~written] = cut[~written] = 0.0
        assert_sums(got, want, mag, K if forward else N, f"{label} {'y' if forward else 'dx'}", cut)


DENSE = [  # R, N, K
    (1, 1, 16), (1, 3, 32), (2, 66, 144), (1, 2880, 2880), (1, 64, 4096), (3, 17, 112), (16, 100, 160), (17, 130, 736),
    (4, 131, 2592), (40, 257, 288), (64, 256, 512), (100, 1000, 736), (129, 203, 608), (200, 513, 320),
    (300, 96, 2880), (257, 5, 32), (5, 7, 9216), (130, 640, 1088), (1, 50000, 96), (31, 33, 16), (65, 300, 1040),
    (1000, 700, 400), (520, 1500, 272), (33, 129, 128), (700, 255, 1168), (128, 256, 256), (96, 64, 11008),
]


@pytest.mark.parametrize("R,N,K", DENSE)
def test_dense(gpu, R, N, K):
    check_both(gpu, Weights(1, N, K, seed=R + N, dense=True), R, bias=N % 2 == 0, label="dense")


GROUPED = [  # rows of every expert, N, K
    ([1, 0, 4, 0, 0, 3, 0, 0, 2], 1440, 2880),
    ([0, 9, 0, 0, 0, 0, 0, 0, 0, 0, 1, 0], 67, 1184),
    ([0] * 200 + [5] + [0] * 50, 130, 512),
    ([1], 32, 32),
    ([0, 0, 0], 32, 32),
    ([4, 0, 1, 0, 0, 11], 96, 128),
    ([16, 17, 0, 33, 1, 64], 200, 336),
    ([100, 0, 130, 7], 515, 272),
    ([300, 1, 0, 129, 128, 127], 384, 640),
    ([31, 32, 33, 63, 65, 95, 97] * 3, 256, 208),
    ([700, 20], 1001, 144),
    ([40] * 64, 300, 256),
]


@pytest.mark.parametrize("counts,N,K", GROUPED)
def test_per_expert(gpu, counts, N, K):
    check_both(gpu, Weights(len(counts), N, K, seed=N), sum(counts), offsets_of(counts), label=f"{len(counts)} experts")


# Sizes that reach each of the tiles of 32, 64 and 128 rows (csrc/fp8_plan.h), with one block of 128
# and several, whole and cut ones, and counts of weight rows that leave waves with little or nothing.
DENSE_TILES = [(R, N, K) for R, N in ((60, 2222), (120, 2500), (250, 2600), (500, 2564), (1000, 2690), (2100, 2600))
               for K in (16, 128, 144, 256, 400, 768)]
# ... and the split of K over eight waves, in one round, several and a cut last one
DENSE_TILES += [(60, 2222, 1168), (60, 2222, 4112), (120, 2500, 1040), (120, 2500, 2592), (250, 2600, 2064)]


@pytest.mark.parametrize("R,N,K", DENSE_TILES)
def test_dense_tiles(gpu, R, N, K):
    check_both(gpu, Weights(1, N, K, seed=R + N, dense=True), R, bias=K % 128 != 0, label="dense")


# ... and each path of the gradient's: N that 8 divides and not, shorter than a chunk of 64, with whole
# periods of six of them and not, last row tiles of one block of 32 rows and two, K that leaves waves idle.
@pytest.mark.parametrize("R,N,K", [(1040, 8, 1040), (1057, 64, 1040), (1040, 131, 1040), (2000, 72, 544), (1500, 384, 720),
                                   (1100, 1096, 1008), (1090, 1150, 1008), (1040, 8200, 1040)])
def test_dense_gradient_tiles(gpu, R, N, K):
    w = Weights(1, N, K, seed=N, dense=True)
    dy = normal(R, R, N, dtype=torch.bfloat16)
    want, mag, _ = X.linear_backward(f64(dy), w.f64, None)
    assert_sums(gpu.moe_fp8_linear_backward(dy, w.codes, w.scales), want, mag, N, "dx")


@pytest.mark.parametrize("mean", [1, 20, 70])
@pytest.mark.parametrize("K", [112, 272, 512])
def test_tiles_of_many_experts(gpu, mean, K):
    """Uneven counts, an expert without rows and one with rows for several tiles among them."""
    E = 64
    counts = np.random.default_rng(mean + K).multinomial(mean * E, np.random.default_rng(mean).dirichlet(np.full(E, 2.0)))
    counts[3], counts[17] = 0, counts[17] + counts[3]
    for N in (1100, 1128):
        check_both(gpu, Weights(E, N, K, seed=K), int(counts.sum()), offsets_of(counts), label=f"mean {mean}")


@pytest.mark.parametrize("R,N,K", [(3, 96, 128), (60, 2222, 128), (250, 2600, 128), (500, 2564, 272), (1000, 2690, 128),
                                   (2100, 2600, 128), (2100, 2600, 144)])
def test_scales_that_are_not_finite_stay_in_their_places(gpu, R, N, K):
    """An infinite or NaN scale of a row reaches that row, of a block of weights its outputs; nothing
    else, blocks of zeros behind K included."""
    w = Weights(1, N, K, seed=5, dense=True)
    x, xs = torch.full((R, K), 0x38, dtype=torch.uint8, device="cuda").view(E4M3), torch.ones((R, L.blocks(K)), device="cuda")
    w.codes.view(torch.uint8).fill_(0x38)
    xs[R // 2, 0], xs[R - 1, -1] = float("nan"), float("inf")
    y = gpu.moe_fp8_linear(x, xs, w.codes, w.scales)
    bad = torch.zeros_like(y, dtype=torch.bool)
    bad[R // 2], bad[R - 1] = True, True
    assert torch.equal(~torch.isfinite(y), bad)
    xs.fill_(1.0)
    w.scales[-1, 0] = float("nan")
    y = gpu.moe_fp8_linear(x, xs, w.codes, w.scales)
    bad.fill_(False)
    bad[:, (N - 1) // 128 * 128:] = True
    assert torch.equal(torch.isnan(y), bad)


def test_rows_of_no_expert_are_left(gpu):
    """A rank's share: rows before the first and from the last offset on keep what they held."""
    for counts, R, first in (([5, 0, 20], 60, 11), ([0, 0, 0], 9, 4), ([150, 90], 300, 33)):
        check_both(gpu, Weights(3 if len(counts) == 3 else 2, 96, 160), R, offsets_of(counts, first), label="share")


def test_offsets_past_the_rows_are_clamped(gpu):
    w = Weights(3, 64, 64)
    off = torch.tensor([-5, 10, 40, 1 << 30], dtype=torch.int32, device="cuda")
    x, xs = random_codes(np.random.default_rng(0), 30, 64), torch.ones((30, 1), device="cuda")
    got = gpu.moe_fp8_linear(x, xs, w.codes, w.scales, None, off)
    x64, bounds = L.values(bytes_of(x), f64(xs)), np.array([0, 10, 30, 30])
    want, mag, _ = X.linear(x64, w.f64, bounds, None)
    assert_sums(got, want, mag, 64, "clamped", largest_of_eights(x64, w.f64, bounds))


def test_no_rows(gpu):
    w = Weights(2, 40, 48)
    off = torch.zeros(3, dtype=torch.int32, device="cuda")
    x = torch.zeros((0, 48), device="cuda").to(E4M3)
    assert gpu.moe_fp8_linear(x, torch.zeros((0, 1), device="cuda"), w.codes, w.scales, w.bias, off).shape == (0, 40)
    assert gpu.moe_fp8_linear_backward(torch.zeros((0, 40), device="cuda").bfloat16(), w.codes, w.scales, off).shape == (0, 48)


@pytest.mark.parametrize("R", [1, 40, 300])
def test_nan_codes_stay_in_their_rows(gpu, R):
    """A NaN weight reaches its output column (its k in the gradient), a NaN in a row that row, and
    what lies behind a row, a tile or a matrix reaches nothing."""
    N, K = 136, 144
    w = Weights(3, N, K, seed=3)
    off = offsets_of([R, 0, R])
    rng = np.random.default_rng(1)
    x, xs = random_codes(rng, 2 * R, K), torch.ones((2 * R, 2), device="cuda")
    dy = normal(1, 2 * R, N, dtype=torch.bfloat16)
    w.codes.view(torch.uint8)[1] = 0x7F  # of an expert without rows
    w.codes.view(torch.uint8)[2, 5, 7] = 0xFF
    y = gpu.moe_fp8_linear(x, xs, w.codes, w.scales, None, off)
    dx = gpu.moe_fp8_linear_backward(dy, w.codes, w.scales, off)
    bad = torch.zeros_like(y, dtype=torch.bool)
    bad[R:, 5] = True
    assert torch.equal(torch.isnan(y), bad)
    bad = torch.zeros_like(dx, dtype=torch.bool)
    bad[R:, 7] = True
    assert torch.equal(torch.isnan(dx), bad)
    w = Weights(3, N, K, seed=3)
    x.view(torch.uint8)[R - 1, 3] = 0x7F
    dy[R, 2] = float("nan")
    assert torch.equal(torch.isnan(gpu.moe_fp8_linear(x, xs, w.codes, w.scales, None, off)).all(1).nonzero(),
                       torch.tensor([[R - 1]], device="cuda"))
    assert torch.equal(torch.isnan(gpu.moe_fp8_linear_backward(dy, w.codes, w.scales, off)).any(1).nonzero(),
                       torch.tensor([[R]], device="cuda"))


@pytest.mark.parametrize("R", [3, 200])
def test_every_code_is_exact(gpu, R):
    """One product an output: each pair of codes, and each code with dy, comes out rounded once."""
    codes = torch.arange(256, dtype=torch.uint8, device="cuda")
    eye = torch.zeros((256, 256), dtype=torch.uint8, device="cuda")
    eye.fill_diagonal_(0)
    eye[torch.arange(256), torch.arange(256)] = codes
    eye[127, 127] = eye[255, 255] = 0  # the NaN codes have a test of their own
    w, s = eye.view(E4M3), torch.ones((2, 2), device="cuda")
    x = torch.randint(0, 127, (R, 256), dtype=torch.uint8, device="cuda", generator=torch.Generator("cuda").manual_seed(1)).view(E4M3)
    v = torch.where((codes & 127) == 127, 0.0, codes.view(E4M3).float())
    y = gpu.moe_fp8_linear(x, torch.ones((R, 2), device="cuda"), w, s)
    assert torch.equal(y, (x.float() * v).bfloat16())
    dy = normal(2, R, 256, dtype=torch.bfloat16)
    assert torch.equal(gpu.moe_fp8_linear_backward(dy, w, s), (dy.float() * v).bfloat16())


def test_far_offsets(gpu):
    """An expert whose weights start past 2^31 bytes."""
    N, K, E = 8192, 8192, 34
    codes = torch.zeros((E, N, K), dtype=torch.uint8, device="cuda")
    rng = np.random.default_rng(0)
    part = random_codes(rng, N, 64).view(torch.uint8)
    codes[E - 1, :, -64:] = part
    w, s = codes.view(E4M3), torch.ones((E, 64, 64), device="cuda")
    for R in (3, 300):
        off = torch.zeros(E + 1, dtype=torch.int32, device="cuda")
        off[E] = R
        x = random_codes(rng, R, K)
        y = gpu.moe_fp8_linear(x, torch.ones((R, 64), device="cuda"), w, s, None, off)
        a, b = L.E4M3[bytes_of(x)[:, -64:]], L.E4M3[part.cpu().numpy()]
        assert_sums(y, a @ b.T, np.abs(a) @ np.abs(b).T, 64, "far", largest_of_eights(a, b, None))
        dy = normal(1, R, N, dtype=torch.bfloat16)
        dx = gpu.moe_fp8_linear_backward(dy, w, s, off)
        assert torch.all(dx[:, :-64] == 0)
        assert_sums(dx[:, -64:], f64(dy) @ b, np.abs(f64(dy)) @ np.abs(b), N, "far dx")


def test_same_bits_on_streams_and_in_a_graph(gpu):
    w = Weights(4, 520, 656, seed=1)
    counts = [70, 0, 200, 30]
    rng = np.random.default_rng(0)
    x, off = normal(1, 300, 656, dtype=torch.bfloat16), offsets_of(counts)
    x2 = normal(2, 300, 656, dtype=torch.bfloat16)

    def step(v, **kw):
        c, s = gpu.moe_fp8_quantize(v, **kw)
        y = gpu.moe_fp8_linear(c, s, w.codes, w.scales, w.bias, off, **kw)
        return [y, gpu.moe_fp8_linear_backward(y, w.codes, w.scales, off, **kw)]

    want, other = step(x), step(x2)
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
        eager = step(x if i % 2 else x2)
        torch.cuda.synchronize()
        for a, b in zip(out, eager):
            assert torch.equal(a, b)


def layer(gpu, x, ids, weights, w13, w2, res, norm_w, train=None):
    """The norm, the experts in 8 bits and the weighted sum, as a user runs them; with train (a
    gradient of the output) the gradients too."""
    T, E = x.shape[0], w13.codes.shape[0]
    k = ids.shape[1]
    flat = ids.reshape(-1).long()
    order = torch.argsort(flat, stable=True).to(torch.int32)
    off = torch.zeros(E + 1, dtype=torch.int32, device="cuda")
    off[1:] = torch.bincount(flat, minlength=E).cumsum(0)
    codes, scales, s, rstd = gpu.moe_rms_norm_fp8(x, norm_w, res)
    rows, pair_rows = gpu.moe_permute(codes.view(torch.float16), order, k)
    row_scales, _ = gpu.moe_permute(scales, order, k)
    h = gpu.moe_fp8_linear(rows.view(E4M3), row_scales, w13.codes, w13.scales, w13.bias, off)
    a, a_scales = gpu.moe_swiglu_fp8(h)
    z = gpu.moe_fp8_linear(a, a_scales, w2.codes, w2.scales, w2.bias, off)
    y = gpu.moe_unpermute(z, pair_rows, weights)
    if train is None:
        return y, s
    dz, dwt = gpu.moe_unpermute_backward(train, z, order, pair_rows, weights)
    da = gpu.moe_fp8_linear_backward(dz, w2.codes, w2.scales, off)
    dh = gpu.moe_swiglu_backward(da, h)
    drows = gpu.moe_fp8_linear_backward(dh, w13.codes, w13.scales, off)
    dn = gpu.moe_permute_backward(drows, pair_rows, k)
    dx, dw = gpu.moe_rms_norm_backward(dn, s, norm_w, rstd, train)
    return y, s, dx, dw, dwt


@pytest.mark.parametrize("T", [5, 150])
def test_a_layer_of_8_bit_experts(gpu, T):
    """All steps together against float64, with the roundings to 8 bits taken from the steps
    themselves: the relative error of the whole (2-norm) is that of its bf16 roundings (each of the
    four stored tensors 2^-8 at most) plus those to 8 bits, 2^-4 at most an element and not
    correlated over the sums: 2^-4 for each of the two products of the forward pass."""
    H, I, E, k = 256, 144, 6, 2
    rng = np.random.default_rng(T)
    w13, w2 = Weights(E, 2 * I, H, seed=1), Weights(E, H, I, seed=2)
    w13.codes = (normal(1, E, 2 * I, H) * 100).clamp(-448, 448).to(E4M3)
    w2.codes = (normal(2, E, H, I) * 100).clamp(-448, 448).to(E4M3)
    w13.scales *= 1e-3
    w2.scales *= 1e-3
    w13.bias, w2.bias = (w13.bias / 1000).contiguous(), (w2.bias / 1000).contiguous()
    x, res, g = (normal(i, T, H, dtype=torch.bfloat16) for i in (3, 4, 5))
    norm_w = 1 + 0.1 * normal(6, H, dtype=torch.bfloat16)
    ids, wts, _, _ = gpu.moe_mxfp4_route(normal(7, T, E), k)
    y, s, dx, dw, dwt = layer(gpu, x, ids, wts, w13, w2, res, norm_w, g)
    assert torch.equal(layer(gpu, x, ids, wts, w13, w2, res, norm_w)[0], y)

    leaves = [torch.from_numpy(f64(t)).requires_grad_() for t in (s, norm_w, wts)]
    s64, w64, p64 = leaves
    a13, a2 = torch.from_numpy(w13.f64), torch.from_numpy(w2.f64)
    n = s64 * torch.rsqrt((s64 * s64).mean(1, keepdim=True) + 1e-5) * w64
    out = torch.zeros((T, H), dtype=torch.float64)
    for e in range(E):
        t, j = (ids.cpu() == e).nonzero(as_tuple=True)
        h = n[t] @ a13[e].t() + torch.from_numpy(f64(w13.bias[e]))
        gate, up = h[:, 0::2].clamp(max=7), h[:, 1::2].clamp(-7, 7)
        z = (gate * torch.sigmoid(1.702 * gate) * (up + 1)) @ a2[e].t() + torch.from_numpy(f64(w2.bias[e]))
        out = out.index_add(0, t, p64[t, j, None] * z)
    g64 = torch.from_numpy(f64(g))
    ((out + s64) * g64).sum().backward()
    allowed = 2 * 2.0 ** -4 + 4 * 2.0 ** -8
    for got, want, name in ((y, out, "y"), (dx, s64.grad, "dx"), (dw, w64.grad, "d_weight"), (dwt, p64.grad, "d_weights")):
        want = want.detach().numpy()
        rel = np.linalg.norm(f64(got) - want) / np.linalg.norm(want)
        assert rel <= allowed, (name, rel)


def test_refusals_of_the_binding(gpu):
    w = Weights(2, 40, 48)
    off = torch.zeros(3, dtype=torch.int32, device="cuda")
    x, xs = torch.zeros((4, 48), device="cuda").to(E4M3), torch.ones((4, 1), device="cuda")
    with pytest.raises(ValueError, match="rows of"):
        gpu.moe_fp8_linear(x[:, :32].contiguous(), xs, w.codes, w.scales, None, off)
    with pytest.raises(ValueError, match="shape"):
        gpu.moe_fp8_linear(x, xs[:3], w.codes, w.scales, None, off)
    with pytest.raises(ValueError, match="shape"):
        gpu.moe_fp8_linear(x, xs, w.codes, w.scales[:, :, :0], None, off)
    with pytest.raises(ValueError, match="shape"):
        gpu.moe_fp8_linear(x, xs, w.codes, w.scales, w.bias[:1], off)
    with pytest.raises(ValueError, match="contiguous"):
        gpu.moe_fp8_linear(x, xs, w.codes.transpose(1, 2), w.scales, None, off)
    with pytest.raises(ValueError, match="without expert_offsets"):
        gpu.moe_fp8_linear(x, xs, w.codes, w.scales)
    with pytest.raises(TypeError):
        gpu.moe_fp8_linear(x.view(torch.uint8), xs, w.codes, w.scales, None, off)
    with pytest.raises(TypeError):
        gpu.moe_fp8_linear_backward(torch.zeros((4, 40), device="cuda"), w.codes, w.scales, off)
    with pytest.raises(gpu.MXFP4MoEError):  # K no multiple of 16
        gpu.moe_fp8_linear(x[:, :40].contiguous(), xs, w.codes[0, :, :40].contiguous(), w.scales[0])
    flat = torch.zeros(4 * 40 + 8, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(gpu.MXFP4MoEError):  # an output that is not aligned
        gpu.moe_fp8_linear(x, xs, w.codes, w.scales, None, off, out=flat[1:161].view(4, 40))
    with pytest.raises(ValueError, match="shares memory"):
        gpu.moe_fp8_linear_backward(flat[:160].view(4, 40), w.codes, w.scales, off,
                                    out=torch.as_strided(flat, (4, 48), (48, 1)) if flat.numel() >= 192 else
                                    w.codes.view(torch.uint8).view(-1)[:384].view(torch.bfloat16).view(4, 48))
