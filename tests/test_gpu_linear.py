"""Rows times 4-bit weights, dense and per expert, and the gradient to the rows
(moe_mxfp4_linear, moe_nvfp4_linear, moe_mxfp4_linear_backward,
moe_nvfp4_linear_backward) against the float64 oracle, and a run of the layer's
separate operators against the fused layer and float64 gradients.

Every product is exact, so a sum of n terms (and the bias, the second-level scale and
the addition of K parts) is off by at most (n + 4) * 2^-23 of the sum of the terms'
magnitudes (one step of fp32 an addition, whichever way the matrix core rounds), then
the result is rounded once to bf16 (half a step, 2^-8 relative).
"""

import numpy as np
import pytest
import torch

from mxfp4_quantized_expert_amd import workloads as W
from oracle import expert_ops as X
from oracle import mxfp4_moe as O

pytestmark = pytest.mark.gpu

BF16 = torch.finfo(torch.bfloat16)


def f64(t):
    return t.detach().double().cpu().numpy()


def bf16(rng, *shape):
    return torch.from_numpy(rng.standard_normal(shape).astype(np.float32)).bfloat16().cuda()


class Weights:
    def __init__(self, fmt, E, N, K, seed=0, dense=False, scales=None):
        rng = np.random.default_rng(seed)
        self.fmt, self.dense, self.group = fmt, dense, 32 if fmt == "mxfp4" else 16
        lead = () if dense else (E,)
        self.b = np.frombuffer(rng.bytes(E * N * K // 2), dtype=np.uint8).reshape(*lead, N, K // 2).copy()
        lo, hi = scales or ((118, 133) if fmt == "mxfp4" else (0x30, 0x49))
        self.s = rng.integers(lo, hi, (*lead, N, K // self.group), dtype=np.uint8)
        self.s2 = None if fmt == "mxfp4" else rng.uniform(1 / 16, 1 / 4, E).astype(np.float32)
        self.bias = torch.from_numpy(rng.standard_normal((*lead, N)).astype(np.float32)).bfloat16().cuda()
        self.upload()

    def upload(self):
        self.blocks, self.scales = torch.from_numpy(self.b).cuda(), torch.from_numpy(self.s).cuda()
        self.scale2 = None if self.s2 is None else torch.from_numpy(self.s2).cuda()

    @property
    def f64(self):
        return X.weights_of(self.b, self.s, self.s2)

    def linear(self, gpu, x, bias=None, offsets=None, **kw):
        if self.fmt == "mxfp4":
            return gpu.moe_mxfp4_linear(x, self.blocks, self.scales, bias, offsets, **kw)
        return gpu.moe_nvfp4_linear(x, self.blocks, self.scales, self.scale2, bias, offsets, **kw)

    def backward(self, gpu, dy, offsets=None, **kw):
        if self.fmt == "mxfp4":
            return gpu.moe_mxfp4_linear_backward(dy, self.blocks, self.scales, offsets, **kw)
        return gpu.moe_nvfp4_linear_backward(dy, self.blocks, self.scales, self.scale2, offsets, **kw)


def offsets_of(counts, first=0):
    return torch.tensor(np.concatenate([[first], first + np.cumsum(counts)]).astype(np.int32)).cuda()


def assert_sums(got, want, mag, terms, label):
    slack = (terms + 4) * 2.0 ** -23 * mag
    bound = slack + (np.abs(want) + slack) * BF16.eps / 2 + BF16.tiny * BF16.eps / 2
    g = f64(got)
    assert np.all(np.isfinite(g)), f"{label}: {np.argwhere(~np.isfinite(g))[:4].tolist()} not finite"
    off = np.abs(g - want) - bound
    assert off.size == 0 or off.max() <= 0, \
        f"{label}: {off.max():.3e} over its bound, first at {np.argwhere(off > 0)[:4].tolist()} of {off.shape}"


def check_both(gpu, w, R, offsets=None, bias=True, seed=1, label=""):
    rng = np.random.default_rng(seed)
    N, K = w.b.shape[-2], 2 * w.b.shape[-1]
    x, dy = bf16(rng, R, K), bf16(rng, R, N)
    off = None if offsets is None else offsets.cpu().numpy()
    w64 = w.f64
    print(f"[linear] {label} R={R} N={N} K={K}", flush=True)
    for forward in (True, False):
        out = torch.full((R, N if forward else K), 7.0, dtype=torch.bfloat16, device="cuda")
        if forward:
            want, mag, written = X.linear(f64(x), w64, off, f64(w.bias) if bias else None)
            got = w.linear(gpu, x, w.bias if bias else None, offsets, out=out)
        else:
            want, mag, written = X.linear_backward(f64(dy), w64, off)
            got = w.backward(gpu, dy, offsets, out=out)
        assert got.data_ptr() == out.data_ptr()
        want[~written] = 7.0  # rows of no expert keep what they held
        mag[~written] = 0.0
        assert_sums(got, want, mag, K if forward else N, f"{label} {'y' if forward else 'dx'}")


DENSE = [  # R, N, K
    (1, 4, 512), (1, 3, 544), (2, 66, 3104), (4, 131, 2592), (3, 1030, 7 * 512 + 96), (4, 65, 30 * 512 + 64),
    (1, 50000, 96), (4, 9, 49 * 512),
    (1, 1, 32), (1, 2880, 2880), (1, 64, 4096), (2, 33, 64), (3, 17, 96), (16, 100, 160), (17, 130, 736),
    (40, 257, 288), (64, 256, 512), (100, 1000, 736), (129, 203, 608), (200, 513, 320), (300, 96, 2880),
    (257, 5, 32), (5, 7, 9 * 128 * 8), (130, 640, 1088),
]


@pytest.mark.parametrize("fmt", ["mxfp4", "nvfp4"])
@pytest.mark.parametrize("R,N,K", DENSE)
def test_dense(gpu, fmt, R, N, K):
    check_both(gpu, Weights(fmt, 1, N, K, seed=R + N, dense=True), R, bias=N % 2 == 0, label=f"dense {fmt}")


GROUPED = [  # rows of every expert, N, K
    ([1, 0, 4, 0, 0, 3, 0, 0, 2], 2880, 2880),
    ([0, 9, 0, 0, 0, 0, 0, 0, 0, 0, 1, 0], 67, 1184),
    ([0] * 200 + [5] + [0] * 50, 130, 4096),
    ([1], 32, 32),
    ([0, 0, 0], 32, 32),
    ([4, 0, 1, 0, 0, 11], 96, 128),
    ([1] * 40, 72, 160),
    ([0, 300, 2, 0, 17, 16, 15, 1], 260, 736),
    ([128, 129, 127, 0, 1], 130, 320),
    ([33, 64, 65, 32, 31, 0, 48], 1000, 96),
    ([513, 3], 384, 512),
    ([0] * 63 + [5, 9] + [0] * 100 + [130], 48, 64),
    ([1, 0] * 256, 16, 32),
]


@pytest.mark.parametrize("fmt", ["mxfp4", "nvfp4"])
@pytest.mark.parametrize("counts,N,K", GROUPED, ids=[str(i) for i in range(len(GROUPED))])
def test_grouped(gpu, fmt, counts, N, K):
    w = Weights(fmt, len(counts), N, K, seed=N + K)
    check_both(gpu, w, sum(counts), offsets_of(counts), bias=K % 64 == 0, label=f"grouped {fmt}")


@pytest.mark.parametrize("fmt", ["mxfp4", "nvfp4"])
@pytest.mark.parametrize("first,behind", [(0, 9), (5, 0), (70, 200)])
def test_rows_of_no_expert_are_left_alone(gpu, fmt, first, behind):
    counts = [20, 0, 130, 3]
    w = Weights(fmt, 4, 136, 96, seed=first)
    check_both(gpu, w, first + sum(counts) + behind, offsets_of(counts, first), label="share")


@pytest.mark.parametrize("fmt,scales", [("mxfp4", (0, 40)), ("mxfp4", (1, 253)), ("nvfp4", (0, 0x7F)),
                                        ("nvfp4", (0x80, 0xFF))])
def test_scale_bytes(gpu, fmt, scales):
    """Scales over the formats' range: subnormal ones, signs, large ones (a row's scales spread over
    few octaves here, so that the fp32 sums stay in range)."""
    N, K, R = 96, 256, 40
    w = Weights(fmt, 1, N, K, dense=True, scales=scales)
    if scales == (1, 253):
        w.s[:] = (np.arange(N)[:, None] * 2 % 190 + 20 + w.s % 8).astype(np.uint8)
        w.upload()
    rng = np.random.default_rng(5)
    x = bf16(rng, R, K)
    w64 = w.f64
    want, mag, _ = X.linear(f64(x), w64)
    # products below the fp32 normal range may be lost to zero
    assert_sums(w.linear(gpu, x), want, mag + K * 2.0 ** -126, K, f"{fmt} {scales}")
    if scales != (1, 253):
        dy = bf16(rng, R, N)
        want, mag, _ = X.linear_backward(f64(dy), w64)
        assert_sums(w.backward(gpu, dy), want, mag + N * 2.0 ** -126, N, f"{fmt} {scales} dx")


@pytest.mark.parametrize("fmt,nan", [("mxfp4", 0xFF), ("nvfp4", 0x7F), ("nvfp4", 0xFF)])
@pytest.mark.parametrize("R", [3, 40, 300])
def test_nan_scales_reach_their_rows_and_groups_only(gpu, fmt, nan, R):
    N, K = 70, 192
    counts = [R, R + 1, 2]
    w = Weights(fmt, 3, N, K, seed=R)
    w.s[1, 69, -1] = nan  # the last group of the last row of the middle expert
    w.upload()
    rng = np.random.default_rng(6)
    off = offsets_of(counts)
    rows = np.zeros(sum(counts), bool)
    rows[R:2 * R + 1] = True
    y, dx = f64(w.linear(gpu, bf16(rng, len(rows), K), None, off)), f64(w.backward(gpu, bf16(rng, len(rows), N), off))
    bad = np.zeros(y.shape, bool)
    bad[np.ix_(rows, [69])] = True
    assert np.array_equal(np.isnan(y), bad)
    bad = np.zeros(dx.shape, bool)
    bad[np.ix_(rows, np.arange(K - w.group, K))] = True
    assert np.array_equal(np.isnan(dx), bad)


@pytest.mark.parametrize("fmt", ["mxfp4", "nvfp4"])
@pytest.mark.parametrize("R,N,K", [(2, 33, 96), (40, 97, 160), (150, 130, 224), (300, 64, 96)])
def test_infinite_inputs_stay_in_their_rows(gpu, fmt, R, N, K):
    """A row of infinities and one of NaN (the last) make only their own outputs non-finite: nothing
    past K, N or a tile's rows is multiplied in."""
    w = Weights(fmt, 2, N, K, seed=3)
    rng = np.random.default_rng(7)
    off = offsets_of([R, 1])
    for width, call in ((K, lambda v: w.linear(gpu, v, None, off)), (N, lambda v: w.backward(gpu, v, off))):
        v = bf16(rng, R + 1, width)
        clean = call(v).clone()
        v[0] = float("inf")
        v[R] = float("nan")
        got = call(v)
        assert torch.equal(got[1:R], clean[1:R])
        assert not bool(torch.isfinite(got[0]).any()) and bool(torch.isnan(got[R]).all())


# Batches whose size takes the 128-row tiles, at sizes that end inside a chunk, a block of rows or a tile.
def _many(seed, E=128, mean=40):
    rng = np.random.default_rng(seed)
    counts = rng.poisson(mean, E)
    counts[:12] = [0, 1, 31, 32, 33, 64, 97, 127, 128, 129, 256, 300]
    return [int(c) for c in rng.permutation(counts)]


@pytest.mark.parametrize("fmt", ["mxfp4", "nvfp4"])
@pytest.mark.parametrize("N,K", [(1, 32), (8, 64), (33, 96), (64, 160), (72, 544), (130, 288), (200, 256), (256, 320),
                                 (257, 32), (321, 224), (264, 1056)])
def test_many_rows_grouped(gpu, fmt, N, K):
    counts = _many(N + K)
    w = Weights(fmt, len(counts), N, K, seed=N)
    check_both(gpu, w, sum(counts) + 11, offsets_of(counts, 7), bias=N % 2 == 1, label=f"many {fmt}")


@pytest.mark.parametrize("fmt", ["mxfp4", "nvfp4"])
@pytest.mark.parametrize("mean,N,K", [(900, 64, 160), (900, 72, 544), (900, 130, 288), (700, 200, 256),
                                      (600, 256, 320), (900, 257, 96), (500, 321, 224), (150, 264, 1056),
                                      (900, 97, 160), (900, 40, 1088), (300, 129, 640), (700, 520, 64)])
def test_long_batches_grouped(gpu, fmt, mean, N, K):
    """Enough rows that small matrices take the 128-row tiles too."""
    counts = _many(N + K, mean=mean)
    w = Weights(fmt, len(counts), N, K, seed=N)
    check_both(gpu, w, sum(counts) + 11, offsets_of(counts, 7), bias=N % 2 == 1, label=f"long {fmt}")


@pytest.mark.parametrize("fmt", ["mxfp4", "nvfp4"])
@pytest.mark.parametrize("N,K", [(97, 288), (200, 224), (264, 544)])
def test_long_batches_infinite_inputs(gpu, fmt, N, K):
    counts = _many(5, mean=700)
    R = sum(counts)
    w = Weights(fmt, len(counts), N, K, seed=3)
    rng = np.random.default_rng(7)
    off = offsets_of(counts)
    at = np.sort(rng.permutation(R)[:2000])
    rest = np.setdiff1d(np.arange(R), at)
    for width, call in ((K, lambda v: w.linear(gpu, v, None, off)), (N, lambda v: w.backward(gpu, v, off))):
        v = bf16(rng, R, width)
        clean = call(v).clone()
        v[at[::2]] = float("inf")
        v[at[1::2]] = float("nan")
        got = call(v)
        assert torch.equal(got[rest], clean[rest])
        assert not bool(torch.isfinite(got[at]).any())


@pytest.mark.parametrize("fmt,nan", [("mxfp4", 0xFF), ("nvfp4", 0xFF)])
def test_long_batches_nan_scales(gpu, fmt, nan):
    N, K = 198, 352
    counts = _many(3, mean=700)
    off = offsets_of(counts)
    e = int(np.argmax(counts))
    w = Weights(fmt, len(counts), N, K, seed=4)
    w.s[e, N - 1, -1] = nan
    w.s[e, 3, 0] = nan
    w.upload()
    rng = np.random.default_rng(6)
    R, first = sum(counts), int(np.sum(counts[:e]))
    y, dx = w.linear(gpu, bf16(rng, R, K), None, off), w.backward(gpu, bf16(rng, R, N), off)
    bad = torch.zeros(y.shape, dtype=torch.bool, device="cuda")
    bad[first:first + counts[e], 3] = bad[first:first + counts[e], N - 1] = True
    assert torch.equal(torch.isnan(y), bad)
    bad = torch.zeros(dx.shape, dtype=torch.bool, device="cuda")
    bad[first:first + counts[e], :w.group] = bad[first:first + counts[e], K - w.group:] = True
    assert torch.equal(torch.isnan(dx), bad)


@pytest.mark.parametrize("fmt", ["mxfp4", "nvfp4"])
@pytest.mark.parametrize("R,N,K", [(17_000, 40, 96), (2500, 2050, 1568), (4000, 1030, 1088)])
def test_many_rows_dense(gpu, fmt, R, N, K):
    w = Weights(fmt, 1, N, K, dense=True, seed=R)
    check_both(gpu, w, R, label=f"many dense {fmt}")


@pytest.mark.parametrize("fmt,nan", [("mxfp4", 0xFF), ("nvfp4", 0x7F)])
def test_many_rows_nan_scales(gpu, fmt, nan):
    N, K = 70, 192
    counts = _many(3)
    off = offsets_of(counts)
    e = int(np.argmax(counts))
    w = Weights(fmt, len(counts), N, K, seed=4)
    w.s[e, 69, -1] = nan
    w.s[e, 3, 0] = nan
    w.upload()
    rng = np.random.default_rng(6)
    R, first = sum(counts), int(np.sum(counts[:e]))
    y, dx = f64(w.linear(gpu, bf16(rng, R, K), None, off)), f64(w.backward(gpu, bf16(rng, R, N), off))
    bad = np.zeros(y.shape, bool)
    bad[first:first + counts[e], [[3], [69]]] = True
    assert np.array_equal(np.isnan(y), bad)
    bad = np.zeros(dx.shape, bool)
    bad[first:first + counts[e], :w.group] = bad[first:first + counts[e], K - w.group:] = True
    assert np.array_equal(np.isnan(dx), bad)


@pytest.mark.parametrize("fmt", ["mxfp4", "nvfp4"])
@pytest.mark.parametrize("N,K", [(97, 160), (72, 96), (64, 64)])
def test_many_rows_infinite_inputs(gpu, fmt, N, K):
    counts = _many(5)
    R = sum(counts)
    w = Weights(fmt, len(counts), N, K, seed=3)
    rng = np.random.default_rng(7)
    off = offsets_of(counts)
    at = np.sort(rng.permutation(R)[:200])
    rest = np.setdiff1d(np.arange(R), at)
    for width, call in ((K, lambda v: w.linear(gpu, v, None, off)), (N, lambda v: w.backward(gpu, v, off))):
        v = bf16(rng, R, width)
        clean = call(v).clone()
        v[at[::2]] = float("inf")
        v[at[1::2]] = float("nan")
        got = call(v)
        assert torch.equal(got[rest], clean[rest])
        assert not bool(torch.isfinite(got[at]).any())


def test_offsets_out_of_range_are_clamped(gpu):
    w = Weights("mxfp4", 4, 64, 64, seed=9)
    rng = np.random.default_rng(8)
    x = bf16(rng, 50, 64)
    off = torch.tensor([-7, 10, 10, 45, 2 ** 31 - 1], dtype=torch.int32).cuda()
    want, mag, _ = X.linear(f64(x), w.f64, [0, 10, 10, 45, 50])
    assert_sums(w.linear(gpu, x, None, off), want, mag, 64, "clamped")
    for scale in (1, 100):  # descending in places: in bounds all the same
        down = torch.tensor([40, 10, 30, 20, 50], dtype=torch.int32).cuda() * scale
        x = bf16(rng, 50 * scale, 64)
        w.linear(gpu, x, None, down), w.backward(gpu, x, down)
    torch.cuda.synchronize()


def test_layer_shapes(gpu):
    """A 20b prefill batch through one projection of gpt-oss sizes, with an uneven load."""
    counts = [200, 0, 37, 3, 130, 1, 64, 77]
    w = Weights("mxfp4", 8, 2880, 2880, seed=10)
    check_both(gpu, w, sum(counts), offsets_of(counts), label="20b")


def test_by_differences(gpu):
    """<dy, linear(x)> is linear in x: its step along u is <dx, u> up to the roundings."""
    for fmt in ("mxfp4", "nvfp4"):
        w = Weights(fmt, 2, 200, 256, seed=12)
        rng = np.random.default_rng(13)
        off = offsets_of([21, 150])
        x, u, dy = bf16(rng, 171, 256), bf16(rng, 171, 256), bf16(rng, 171, 200)
        y1, y0 = f64(w.linear(gpu, x + u, None, off)), f64(w.linear(gpu, x, None, off))
        step = f64(x + u) - f64(x)
        dx = f64(w.backward(gpu, dy, off))
        mag1, mag0 = (X.linear(f64(v), w.f64, off.cpu().numpy())[1] for v in (x + u, x))
        magx = X.linear_backward(f64(dy), w.f64, off.cpu().numpy())[1]
        tol = (np.abs(f64(dy)) * ((np.abs(y1) + np.abs(y0)) * 2.0 ** -8 + 260 * 2.0 ** -23 * (mag0 + mag1))).sum()
        tol += (np.abs(step) * (np.abs(dx) * 2.0 ** -8 + 204 * 2.0 ** -23 * magx)).sum()
        lhs, rhs = (f64(dy) * (y1 - y0)).sum(), (dx * step).sum()
        scale = np.abs(f64(dy) * (y1 - y0)).sum()
        assert abs(lhs - rhs) <= tol and tol <= 0.05 * scale


@pytest.mark.parametrize("counts", [[3, 0, 1], [40, 17, 0], [300, 129, 5], [7000, 5000, 5000]])
def test_captured_and_replayed(gpu, counts):
    w = Weights("nvfp4", 3, 200, 256, seed=14)
    R = sum(counts)
    off = offsets_of(counts)
    gen = torch.Generator().manual_seed(15)
    x, dy = torch.zeros((R, 256), dtype=torch.bfloat16).cuda(), torch.zeros((R, 200), dtype=torch.bfloat16).cuda()

    def run():
        return w.linear(gpu, x, w.bias, off), w.backward(gpu, dy, off)

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        run()
    torch.cuda.current_stream().wait_stream(s)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        kept = run()
    for rep in range(4):
        x.copy_(torch.randn(x.shape, generator=gen)), dy.copy_(torch.randn(dy.shape, generator=gen))
        off.copy_(offsets_of(counts[rep % 3:] + counts[:rep % 3]))  # the loads move between the experts
        eager = [t.clone() for t in run()]
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        for a, b in zip(kept, eager):
            assert torch.equal(a, b), rep


def test_on_another_stream(gpu):
    w = Weights("mxfp4", 1, 300, 512, seed=16, dense=True)
    rng = np.random.default_rng(17)
    x, dy = bf16(rng, 200, 512), bf16(rng, 200, 300)
    want = w.linear(gpu, x, w.bias), w.backward(gpu, dy)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    for stream in (s, s.cuda_stream):
        got = w.linear(gpu, x, w.bias, stream=stream), w.backward(gpu, dy, stream=stream)
        s.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_many_rows_past_32_bit_offsets(gpu):
    """R * K and R * N above 2^31 elements; the weights pass each row's values through (one code per row)."""
    R, N, K = 1_100_000, 2048, 2048
    blocks = torch.zeros((N, K // 2), dtype=torch.uint8, device="cuda")
    n = torch.arange(N, device="cuda")
    blocks[n, n // 2] = torch.where(n % 2 == 0, 2, 0x20).to(torch.uint8)  # W[n, n] = 1
    scales = torch.full((N, K // 32), 127, dtype=torch.uint8, device="cuda")
    x = torch.empty((R, K), dtype=torch.bfloat16, device="cuda")
    x.copy_((torch.arange(K, device="cuda") % 200)[None])
    x[-1] = x[-1].flip(0)
    y = gpu.moe_mxfp4_linear(x, blocks, scales)
    assert torch.equal(y[-300:], x[-300:]) and torch.equal(y[::100_003], x[::100_003])
    dx = gpu.moe_mxfp4_linear_backward(x, blocks, scales, out=y)
    assert torch.equal(dx[-300:], x[-300:]) and torch.equal(dx[::100_003], x[::100_003])


# ---------------------------------------------------------------- the operators as they are used together

def _swiglu(h):
    gate, up = h[:, 0::2].clamp(max=7), h[:, 1::2].clamp(-7, 7)
    return gate * torch.sigmoid(1.702 * gate) * (up + 1)


@pytest.mark.parametrize("fmt,T", [("mxfp4", 4), ("mxfp4", 200), ("nvfp4", 33)])
def test_layer_from_its_operators_and_its_gradients(gpu, fmt, T):
    spec = W.LAYERS["tiny"].with_(T=T, H=192, I=96, E=8, top_k=3, scale_lo=118, scale_hi=122)
    L = W.make_layer(spec, seed=20) if fmt == "mxfp4" else W.make_nvfp4_layer(spec, seed=20)
    if fmt == "nvfp4":
        L["w13_scales"], L["w2_scales"] = L["w13_scales"] // 4, L["w2_scales"] // 4  # inside the clamps
    d = gpu.layer_to_device(L)
    k = spec.top_k
    rng = np.random.default_rng(21)
    dy = bf16(rng, T, spec.H)

    class Lin(torch.autograd.Function):  # a user's wrapper of the two entry points
        @staticmethod
        def forward(ctx, x, name, offsets):
            ctx.name, ctx.offsets = name, offsets
            w = (d[name + "_blocks"], d[name + "_scales"])
            if fmt == "mxfp4":
                return gpu.moe_mxfp4_linear(x, *w, d[name + "_bias"], offsets)
            return gpu.moe_nvfp4_linear(x, *w, d[name + "_scale2"], d[name + "_bias"], offsets)

        @staticmethod
        def backward(ctx, g):
            w = (d[ctx.name + "_blocks"], d[ctx.name + "_scales"])
            g = g.contiguous()
            if fmt == "mxfp4":
                return gpu.moe_mxfp4_linear_backward(g, *w, ctx.offsets), None, None
            return gpu.moe_nvfp4_linear_backward(g, *w, d[ctx.name + "_scale2"], ctx.offsets), None, None

    ids, weights, offsets, pairs = gpu.moe_mxfp4_route(d["router_logits"], k)
    rows, pair_rows = gpu.moe_permute(d["x"], pairs, k)
    xin = rows.requires_grad_()
    a = _swiglu(Lin.apply(xin, "w13", offsets).float()).bfloat16()
    z = Lin.apply(a, "w2", offsets)
    y = gpu.moe_unpermute(z.detach(), pair_rows, weights)
    ref = (O.moe_forward if fmt == "mxfp4" else O.moe_forward_nvfp4)(L, k)
    rel, mx = O.parity_errors(f64(y), ref)
    assert rel <= 1e-2 and mx <= 2e-2, (rel, mx)  # the fused layer's own bar

    dz, dw = gpu.moe_unpermute_backward(dy, z.detach(), pairs, pair_rows, weights)
    z.backward(dz)
    dx = gpu.moe_permute_backward(xin.grad, pair_rows, k)
    dlogits = gpu.moe_route_backward(ids, weights, dw, spec.E)

    # the same in float64 on the host, with torch's own gradients
    x64 = d["x"].double().cpu().requires_grad_()
    lg = d["router_logits"].double().cpu().requires_grad_()
    scale2 = {n: None if fmt == "mxfp4" else L[n + "_scale2"] for n in ("w13", "w2")}
    w64 = {n: torch.from_numpy(X.weights_of(L[n + "_blocks"], L[n + "_scales"], scale2[n])) for n in ("w13", "w2")}
    b64 = {n: d[n + "_bias"].double().cpu() for n in ("w13", "w2")}
    pick = ids.long().cpu()
    p = torch.softmax(lg.gather(1, pick), 1)
    out = torch.zeros((T, spec.H), dtype=torch.float64)
    for j in range(k):
        e = pick[:, j]
        h = torch.einsum("th,tnh->tn", x64, w64["w13"][e]) + b64["w13"][e]
        out = out + p[:, j:j + 1] * (torch.einsum("ti,tni->tn", _swiglu(h), w64["w2"][e]) + b64["w2"][e])
    out.backward(dy.double().cpu())
    # about six bf16 roundings on the way, each 2^-9 or less on average: under 1e-2 normwise
    for got, want, name in ((dx, x64.grad, "dx"), (dlogits, lg.grad, "dlogits")):
        rel = float((got.double().cpu() - want).norm() / want.norm())
        print(f"[layer] {fmt} T={T} {name}: {rel:.2e}", flush=True)
        assert rel <= 1e-2, (name, rel)


# experts, rows of an expert on average, N, K: where each of the kernels and of its variants is taken, with loops over
# K (the gradient: over N) that pass through every stage of a ring more than once and end in each of them
VARIANTS = [
    (16, 5, 100, 704), (32, 7, 530, 2112), (128, 7, 180, 2112), (32, 24, 2002, 800), (32, 24, 1998, 832),
    (20, 70, 850, 1184), (6, 400, 1057, 1600), (5, 900, 834, 1504), (8, 37, 1001, 736), (3, 12, 2050, 96),
    (128, 130, 1606, 1568),
]


@pytest.mark.parametrize("fmt", ["mxfp4", "nvfp4"])
@pytest.mark.parametrize("E,mean,N,K", VARIANTS)
def test_kernel_variants(gpu, fmt, E, mean, N, K):
    counts = np.random.default_rng(E + N).poisson(mean, E)
    counts[E // 3] = 0
    w = Weights(fmt, E, N, K, seed=N + K)
    check_both(gpu, w, int(counts.sum()) + 3, offsets_of(counts, 2), label=f"variants {fmt}")


@pytest.mark.parametrize("fmt", ["mxfp4", "nvfp4"])
@pytest.mark.parametrize("E,mean,N,K", VARIANTS)
def test_same_bits_every_time(gpu, fmt, E, mean, N, K):
    """A product that read a stage before its loads were there would differ from call to call, most of all while
    another one keeps the caches cold."""
    counts = np.random.default_rng(E + K).poisson(mean, E)
    w, other = Weights(fmt, E, N, K, seed=3), Weights(fmt, E, N, K, seed=4)
    off = offsets_of(counts)
    rng = np.random.default_rng(5)
    R = int(counts.sum())
    x, dy = bf16(rng, R, K), bf16(rng, R, N)
    spill = torch.empty(300 << 20, dtype=torch.uint8, device="cuda")
    y, dx = w.linear(gpu, x, None, off), w.backward(gpu, dy, off)
    for i in range(12):
        if i % 3 == 0:
            spill.fill_(i)
        other.linear(gpu, x, None, off), other.backward(gpu, dy, off)
        assert torch.equal(w.linear(gpu, x, None, off), y)
        assert torch.equal(w.backward(gpu, dy, off), dx)


def test_two_streams_at_once(gpu):
    """Calls on two streams share nothing: each gives what it gives alone."""
    rng = np.random.default_rng(11)
    jobs = []
    for i, (fmt, E, mean, N, K) in enumerate([("mxfp4", 32, 24, 2002, 800), ("nvfp4", 64, 100, 1606, 1568)]):
        counts = rng.poisson(mean, E)
        w, off, R = Weights(fmt, E, N, K, seed=i), offsets_of(counts), int(counts.sum())
        x, dy = bf16(rng, R, K), bf16(rng, R, N)
        jobs.append((w, off, x, dy, w.linear(gpu, x, None, off), w.backward(gpu, dy, off), torch.cuda.Stream()))
    torch.cuda.synchronize()
    for _ in range(6):
        got = []
        for w, off, x, dy, _, _, stream in jobs:
            with torch.cuda.stream(stream):
                got.append((w.linear(gpu, x, None, off), w.backward(gpu, dy, off)))
        torch.cuda.synchronize()
        for (_, _, _, _, y, dx, _), (a, b) in zip(jobs, got):
            assert torch.equal(a, y) and torch.equal(b, dx)


# Calls with enough weights (13 MB and more) for few rows that they are streamed past them, in tiles of 4 rows and of 8:
# every number of units of 512 k a wave and of waves a block, N that ends inside a row group.
STREAMED = [  # rows of every expert (an int: dense), N, K
    (1, 100_001, 256), (4, 50_003, 544), (3, 22_010, 1184), (7, 17_003, 1568), (8, 10_013, 2592), (2, 8_001, 3104),
    (6, 7_002, 3680), (5, 5_003, 5152), (1, 4_007, 7200), (4, 3_001, 9888), (8, 2_501, 12_288), (3, 2_050, 12_256),
    ([1, 0] * 256, 300, 352), ([0] * 20 + [3, 1, 0, 7] * 3 + [1] * 30, 515, 1184), ([2, 0, 0, 9, 4, 0, 1, 5], 1441, 3104),
    ([0, 30] + [0, 1, 5, 8, 9] * 12, 290, 2112), ([4] * 64, 736, 736), ([17, 1], 3001, 9888),
]
STREAMED_IDS = [f"{c if isinstance(c, int) else len(c)}-{n}-{k}" for c, n, k in STREAMED]


def streamed(fmt, counts, N, K, seed):
    dense = isinstance(counts, int)
    w = Weights(fmt, 1 if dense else len(counts), N, K, seed=seed, dense=dense)
    return w, (counts if dense else sum(counts)), None if dense else offsets_of(counts)


@pytest.mark.parametrize("fmt", ["mxfp4", "nvfp4"])
@pytest.mark.parametrize("counts,N,K", STREAMED, ids=STREAMED_IDS)
def test_streamed_weights(gpu, fmt, counts, N, K):
    w, R, off = streamed(fmt, counts, N, K, seed=N + K)
    used = 1 if off is None else min(len(counts), R)
    assert used * N * K * 0.53125 >= 13e6
    rng = np.random.default_rng(1)
    x, bias = bf16(rng, R, K), w.bias if N % 2 else None
    print(f"[streamed] {fmt} R={R} N={N} K={K}", flush=True)
    want, mag, written = X.linear(f64(x), w.f64, None if off is None else off.cpu().numpy(),
                                  None if bias is None else f64(bias))
    assert written.all()
    y = w.linear(gpu, x, bias, off)
    assert_sums(y, want, mag, K, f"streamed {fmt}")
    assert torch.equal(w.linear(gpu, x, bias, off), y)


@pytest.mark.parametrize("fmt", ["mxfp4", "nvfp4"])
@pytest.mark.parametrize("counts,N,K", [(4, 50_003, 544), (8, 10_013, 2592), ([2, 0, 0, 9, 4, 0, 1, 5], 1441, 3104)],
                         ids=["4-rows", "8-rows", "experts"])
def test_streamed_weights_keep_rows_apart(gpu, fmt, counts, N, K):
    """Infinities and NaN of a row, and a NaN scale of a weight row, reach their own outputs only."""
    w, R, off = streamed(fmt, counts, N, K, seed=3)
    x = bf16(np.random.default_rng(7), R, K)
    clean = w.linear(gpu, x, None, off)
    x[0], x[R - 1] = float("inf"), float("nan")
    got = w.linear(gpu, x, None, off)
    assert torch.equal(got[1:R - 1], clean[1:R - 1])
    assert not bool(torch.isfinite(got[0]).any()) and bool(torch.isnan(got[R - 1]).all())
    x = bf16(np.random.default_rng(7), R, K)
    w.s.reshape(-1, *w.s.shape[-2:])[-1, N - 1, -1] = 0xFF
    w.upload()
    bad = torch.zeros((R, N), dtype=torch.bool, device="cuda")
    bad[0 if off is None else int(off[-2]):, N - 1] = True
    got = w.linear(gpu, x, None, off)
    assert torch.equal(torch.isnan(got), bad) and torch.equal(got[~bad], clean[~bad])


def test_streamed_weights_in_a_graph(gpu):
    counts, N, K = [2, 0, 0, 9, 4, 0, 1, 5], 1441, 3104
    w, R, off = streamed("mxfp4", counts, N, K, seed=4)
    x = torch.zeros((R, K), dtype=torch.bfloat16, device="cuda")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        w.linear(gpu, x, w.bias, off)
    torch.cuda.current_stream().wait_stream(s)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        kept = w.linear(gpu, x, w.bias, off)
    gen = torch.Generator().manual_seed(15)
    for rep in range(4):
        x.copy_(torch.randn(x.shape, generator=gen))
        off.copy_(offsets_of(counts[rep:] + counts[:rep]))
        eager = w.linear(gpu, x, w.bias, off).clone()
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(kept, eager), rep
