"""Token rows by expert and back, their gradients and the routing softmax's gradient
(moe_permute, moe_permute_backward, moe_unpermute, moe_unpermute_backward,
moe_route_backward) against the float64 oracle.

Copies and row numbers must be equal.  A sum of k fp32 terms fma(w, z, s) is off by at
most k * 2^-24 of the sum of the terms' magnitudes, then the result is rounded once to
its type (half a step, eps / 2 relative); a dot product of H terms summed in fp32 in any
order by at most (H + 1) * 2^-24 of the sum of the products' magnitudes.
"""

import numpy as np
import pytest
import torch

from oracle import expert_ops as X

pytestmark = pytest.mark.gpu

U32 = 2.0 ** -24
DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


def f64(t):
    return t.detach().double().cpu().numpy()


def assert_rounded(got, want, slack, dtype, label):
    """|got - want| at most the fp32 slack plus half a step of dtype at the largest value that slack allows."""
    info = torch.finfo(dtype)
    bound = slack + (np.abs(want) + slack) * info.eps / 2 + info.tiny * info.eps / 2
    off = np.abs(f64(got) - want) - bound
    assert np.all(np.isfinite(f64(got))), f"{label}: non-finite"
    assert off.size == 0 or off.max() <= 0, f"{label}: {off.max():.3e} over its bound at {np.argmax(off)}"


class Batch:
    """Seeded routing of T tokens to k of E experts, of which the first `local` are held here;
    `pad` empty rows are mixed in, and the rows without a pair hold NaN."""

    def __init__(self, T, H, E, k, dtype, local=None, pad=0, seed=0, shift=0):
        rng = np.random.default_rng(seed)
        local = E if local is None else local
        ids = np.argsort(rng.standard_normal((T, E)), axis=1)[:, :k].reshape(-1) if T else np.zeros(0, int)
        order = np.argsort(ids, kind="stable")
        here = order[ids[order] < local]
        pairs = np.full(len(here) + pad, -1, dtype=np.int64)
        pairs[np.sort(rng.permutation(len(pairs))[:len(here)])] = here
        bad = np.flatnonzero(pairs < 0)
        pairs[bad[1::2]] = T * k + 5 + np.arange(len(bad[1::2]))  # empty rows: -1 and past the last pair
        self.T, self.H, self.k, self.R, self.dtype = T, H, k, len(pairs), DTYPES[dtype]
        self.pairs_host = pairs
        self.pairs = torch.from_numpy(pairs.astype(np.int32)).cuda()

        def rows(n, fill=None):
            v = torch.from_numpy(rng.standard_normal((n, H)))
            if fill is not None:
                v[torch.from_numpy(fill)] = float("nan")
            flat = torch.empty(n * H + shift, dtype=self.dtype, device="cuda")  # shift: off the 16-byte grid
            t = flat[shift:].view(n, H)
            t.copy_(v)
            return t

        self.x, self.dy = rows(T), rows(T)
        self.z, self.dz = rows(self.R, bad), rows(self.R, bad)
        w = rng.random((T, k)) + 0.01
        self.w = torch.from_numpy((w / w.sum(1, keepdims=True)).astype(np.float32)).cuda()
        self.pair_rows_host = X.permute(np.zeros((T, 1)), pairs, k)[1]
        self.pair_rows = torch.from_numpy(self.pair_rows_host.astype(np.int32)).cuda()


CASES = [
    # T, H, E, k, dtype, local, pad, shift
    (1, 1, 1, 1, "bf16", None, 0, 0),
    (1, 2880, 32, 4, "bf16", None, 0, 0),
    (4, 2880, 32, 4, "bf16", None, 0, 0),
    (3, 7, 5, 5, "f16", None, 2, 0),
    (17, 64, 8, 2, "f32", 3, 4, 0),
    (65, 1001, 8, 2, "f32", 5, 3, 0),
    (33, 1001, 16, 3, "bf16", None, 1, 0),
    (64, 2142, 17, 3, "f16", None, 0, 0),
    (129, 88, 128, 8, "bf16", 40, 70, 0),
    (40, 72, 40, 32, "bf16", None, 0, 0),
    (50, 72, 8, 2, "bf16", None, 5, 1),      # rows off the 16-byte grid, by one element
    (50, 72, 8, 2, "f32", None, 5, 1),
    (50, 72, 8, 2, "f16", None, 5, 2),
    (20, 40, 4, 2, "bf16", 0, 3, 0),         # no pair is held here
    (20, 40, 4, 2, "bf16", 0, 0, 0),         # ... and no row at all
    (0, 40, 4, 2, "bf16", None, 3, 0),       # no tokens, rows of padding
    (700, 256, 8, 4, "bf16", None, 0, 0),    # more pairs than one block inverts
    (300, 6000, 8, 2, "f32", 7, 9, 0),
]
IDS = ["-".join(map(str, c)) for c in CASES]


@pytest.mark.parametrize("case", CASES, ids=IDS)
def test_permute_and_gradient(gpu, case):
    T, H, E, k, dtype, local, pad, shift = case
    b = Batch(T, H, E, k, dtype, local, pad, seed=T + H, shift=shift)
    print(f"[permute] {case}", flush=True)
    rows, pair_rows = gpu.moe_permute(b.x, b.pairs, k)
    want, want_rows = X.permute(f64(b.x), b.pairs_host, k)
    assert np.array_equal(f64(rows), want)
    assert np.array_equal(pair_rows.cpu().numpy(), want_rows)
    dx = gpu.moe_permute_backward(b.dz, pair_rows, k)
    want, mag = X.unpermute(f64(b.dz), want_rows, np.ones((T, k)))
    assert_rounded(dx, want, k * U32 * mag, b.dtype, "dx")


@pytest.mark.parametrize("case", CASES, ids=IDS)
def test_unpermute_and_gradients(gpu, case):
    T, H, E, k, dtype, local, pad, shift = case
    b = Batch(T, H, E, k, dtype, local, pad, seed=T + 2 * H, shift=shift)
    print(f"[unpermute] {case}", flush=True)
    y = gpu.moe_unpermute(b.z, b.pair_rows, b.w)
    want, mag = X.unpermute(f64(b.z), b.pair_rows_host, f64(b.w))
    assert_rounded(y, want, k * U32 * mag, b.dtype, "y")
    d_rows, d_w = gpu.moe_unpermute_backward(b.dy, b.z, b.pairs, b.pair_rows, b.w)
    want, want_w, mag = X.unpermute_backward(f64(b.dy), f64(b.z), b.pairs_host, b.pair_rows_host, f64(b.w))
    held = np.zeros(b.R, dtype=bool)
    held[b.pair_rows_host[b.pair_rows_host >= 0]] = True
    assert not f64(d_rows)[~held].any()
    want[~held] = 0
    assert_rounded(d_rows, want, U32 * np.abs(want), b.dtype, "d_rows")
    assert_rounded(d_w, want_w, (H + 1) * U32 * mag, torch.float32, "d_weights")


def test_pair_listed_twice_belongs_to_its_later_row(gpu):
    b = Batch(12, 24, 4, 2, "f32", seed=5)
    pairs = b.pairs_host.copy()
    pairs[3] = pairs[20]  # one pair twice, another nowhere
    d = torch.from_numpy(pairs.astype(np.int32)).cuda()
    rows, pair_rows = gpu.moe_permute(b.x, d, 2)
    want, want_rows = X.permute(f64(b.x), pairs, 2)
    assert np.array_equal(f64(rows), want) and np.array_equal(pair_rows.cpu().numpy(), want_rows)
    d_rows, d_w = gpu.moe_unpermute_backward(b.dy, b.z, d, pair_rows, b.w)
    want, want_w, mag = X.unpermute_backward(f64(b.dy), f64(b.z), pairs, want_rows, f64(b.w))
    assert not d_rows[3].any()
    assert_rounded(d_rows, want, U32 * np.abs(want), b.dtype, "d_rows")
    assert_rounded(d_w, want_w, 25 * U32 * mag, torch.float32, "d_weights")


@pytest.mark.parametrize("seed", [1, 2])
def test_pairs_past_those_that_blocks_invert(gpu, seed):
    """More pairs than kInvertInBlocks: the rows are entered into a cleared pair_rows."""
    b = Batch(22000, 3, 16, 3, "bf16", local=11, pad=100, seed=seed)
    assert b.T * b.k > 65536
    for _ in range(2):
        rows, pair_rows = gpu.moe_permute(b.x, b.pairs, 3)
        want, want_rows = X.permute(f64(b.x), b.pairs_host, 3)
        assert np.array_equal(f64(rows), want) and np.array_equal(pair_rows.cpu().numpy(), want_rows)
    none = torch.empty((0,), dtype=torch.int32, device="cuda")
    rows, pair_rows = gpu.moe_permute(b.x, none, 3)
    assert rows.shape == (0, 3) and bool((pair_rows == -1).all())


@pytest.mark.parametrize("T,H,k,dtype", [(4000, 2880, 2, "bf16"), (1500, 2881, 4, "f32"), (13000, 2047, 1, "f16"),
                                         (70000, 512, 1, "bf16")])
def test_large_batches_by_token(gpu, T, H, k, dtype):
    """Rows of 32 MiB and more are written token by token; a pair listed twice among them."""
    b = Batch(T, H, 8, k, dtype, local=6, pad=37, seed=T)
    pairs = b.pairs_host.copy()
    twice = np.flatnonzero((pairs >= 0) & (pairs < T * k))[[5, -3]]
    pairs[twice[0]] = pairs[twice[1]]
    d = torch.from_numpy(pairs.astype(np.int32)).cuda()
    assert b.R * H * b.x.element_size() >= 32 << 20
    rows, pair_rows = gpu.moe_permute(b.x, d, k, out=torch.full((b.R, H), 9.0, dtype=b.dtype, device="cuda"))
    ok = (pairs >= 0) & (pairs < T * k)
    want = torch.where(torch.from_numpy(ok).cuda()[:, None], b.x[torch.from_numpy(np.where(ok, pairs, 0) // k).cuda()],
                       torch.zeros((), dtype=b.dtype, device="cuda"))
    assert torch.equal(rows, want)
    assert np.array_equal(pair_rows.cpu().numpy(), X.permute(np.zeros((T, 1)), pairs, k)[1])


def test_infinite_rows_reach_their_tokens_only(gpu):
    b = Batch(9, 16, 4, 2, "bf16", seed=7)
    b.z[int(b.pair_rows_host[5])] = float("inf")
    y = gpu.moe_unpermute(b.z, b.pair_rows, b.w)
    assert bool(torch.isinf(y[2]).all()) and bool(torch.isfinite(y[torch.arange(9) != 2]).all())


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_infinite_element_is_counted_once(gpu, dtype):
    """An infinity among the elements that the last two pieces of a row share (H no multiple of a
    piece): its dot product with positive values is infinite, not NaN."""
    H = 13 if dtype == "bf16" else 7
    b = Batch(6, H, 4, 2, dtype, seed=9)
    b.dy.copy_(b.dy.abs() + 0.1)
    b.z[int(b.pair_rows_host[3]), H - 6 if dtype == "f32" else 6] = float("inf")
    d_rows, d_w = gpu.moe_unpermute_backward(b.dy, b.z, b.pairs, b.pair_rows, b.w)
    want = f64(b.dy)[:, None] * f64(b.z)[b.pair_rows_host].reshape(6, 2, H)
    assert bool(torch.isposinf(d_w[1, 1])) and np.array_equal(np.isfinite(f64(d_w)), np.isfinite(want.sum(2)))


def test_out_of_range_rows_are_no_rows(gpu):
    b = Batch(9, 16, 4, 2, "f32", seed=8)
    host = b.pair_rows_host.copy()
    host[[0, 7, 11]] = [-2 ** 31, b.R, 2 ** 31 - 1]
    pr = torch.from_numpy(host.astype(np.int32)).cuda()
    want, mag = X.unpermute(f64(b.z), host, f64(b.w))
    assert_rounded(gpu.moe_unpermute(b.z, pr, b.w), want, 2 * U32 * mag, b.dtype, "y")
    d_rows, d_w = gpu.moe_unpermute_backward(b.dy, b.z, b.pairs, pr, b.w)
    want, want_w, mag = X.unpermute_backward(f64(b.dy), f64(b.z), b.pairs_host, host, f64(b.w))
    assert_rounded(d_rows, want, U32 * np.abs(want), b.dtype, "d_rows")
    assert_rounded(d_w, want_w, 17 * U32 * mag, torch.float32, "d_weights")


@pytest.mark.parametrize("T,E,k", [(1, 1, 1), (1, 32, 4), (5, 7, 3), (64, 32, 4), (33, 128, 8), (9, 512, 32),
                                   (1000, 66, 6), (3, 300, 2), (4097, 128, 4)])
def test_route_backward(gpu, T, E, k):
    rng = np.random.default_rng(T + E)
    ids = np.argsort(rng.standard_normal((T, E)), axis=1)[:, :k].astype(np.int32)
    w = rng.random((T, k)).astype(np.float32)
    w /= w.sum(1, keepdims=True)
    dw = rng.standard_normal((T, k)).astype(np.float32)
    got = gpu.moe_route_backward(*(torch.from_numpy(a).cuda() for a in (ids, w, dw)), E)
    w64, dw64 = w.astype(np.float64), dw.astype(np.float64)
    want = X.route_backward(ids, w64, dw64, E)
    # the mean is off by k roundings of its terms; then a difference and a product
    terms = (w64 * np.abs(dw64)).sum(1, keepdims=True)
    slack = np.zeros((T, E))
    np.put_along_axis(slack, ids.astype(np.int64), w64 * (k + 3) * U32 * (terms + np.abs(dw64)), 1)
    assert_rounded(got, want, slack, torch.float32, "d_logits")


def test_route_backward_skips_and_adds_ids(gpu):
    ids = torch.tensor([[3, -1, 3], [9, 2, 5]], dtype=torch.int32, device="cuda")
    w = torch.tensor([[0.5, 0.25, 0.25], [0.2, 0.3, 0.5]], device="cuda")
    dw = torch.tensor([[1.0, 2.0, -1.0], [0.5, -2.0, 4.0]], device="cuda")
    got = f64(gpu.moe_route_backward(ids, w, dw, 6))
    want = X.route_backward(ids.cpu().numpy(), f64(w), f64(dw), 6)
    assert np.abs(got - want).max() <= 16 * U32 and not got[0, :3].any()


def test_gradients_by_differences(gpu):
    """Along random directions: unpermute is linear in the rows and in the weights, so a step of any
    size gives its gradient up to the fp32 sums; the softmax's by a small central difference."""
    b = Batch(21, 50, 8, 3, "f32", local=6, seed=11)
    rng = np.random.default_rng(12)
    z = torch.where(torch.isnan(b.z), torch.zeros_like(b.z), b.z)
    dy64 = f64(b.dy)
    d_rows, d_w = gpu.moe_unpermute_backward(b.dy, z, b.pairs, b.pair_rows, b.w)

    def loss(rows, w):
        return (dy64 * f64(gpu.moe_unpermute(rows, b.pair_rows, w))).sum()

    uw = torch.from_numpy(rng.standard_normal((b.T, b.k)).astype(np.float32)).cuda()
    uz = torch.from_numpy(rng.standard_normal((b.R, b.H)).astype(np.float32)).cuda()
    big_w, big_z = b.w.abs() + uw.abs(), z.abs() + uz.abs()
    mag = X.unpermute(f64(big_z), b.pair_rows_host, f64(big_w))[1]
    tol = 2 * (b.k + 4) * U32 * (np.abs(dy64) * mag).sum()
    got = (loss(z, b.w + uw) - loss(z, b.w - uw)) / 2
    assert abs(got - (f64(d_w) * f64(uw)).sum()) <= tol
    got = (loss(z + uz, b.w) - loss(z - uz, b.w)) / 2
    assert abs(got - (f64(d_rows) * f64(uz)).sum()) <= tol

    # permute: <d_rows, permute(x)> is linear in x
    rows, pair_rows = gpu.moe_permute(b.x, b.pairs, b.k)
    dz = torch.where(torch.isnan(b.dz), torch.zeros_like(b.dz), b.dz)
    dx = gpu.moe_permute_backward(dz, pair_rows, b.k)
    lhs, rhs = (f64(dz) * f64(rows)).sum(), (f64(dx) * f64(b.x)).sum()
    mag = X.unpermute(f64(dz), b.pair_rows_host, np.ones((b.T, b.k)))[1]
    assert abs(lhs - rhs) <= (b.k + 1) * U32 * (mag * np.abs(f64(b.x))).sum()

    # routing: logits whose picks are far apart, so that the steps keep the choice
    T, E, k, h = 16, 12, 4, 2.0 ** -7
    logits = np.stack([rng.permutation(E) * 0.25 for _ in range(T)]).astype(np.float32)
    u = rng.uniform(-1, 1, (T, E)).astype(np.float32)
    g = torch.from_numpy(rng.standard_normal((T, k)).astype(np.float32)).cuda()
    ids, w, _, _ = gpu.moe_mxfp4_route(torch.from_numpy(logits).cuda(), k)
    d = gpu.moe_route_backward(ids, w, g, E)

    def f(sign):
        i2, w2, _, _ = gpu.moe_mxfp4_route(torch.from_numpy(logits + np.float32(sign * h) * u).cuda(), k)
        assert torch.equal(i2, ids)
        return f64(g) * f64(w2)

    got = ((f(1) - f(-1)) / (2 * h)).sum(1)
    want = (f64(d) * u).sum(1)
    # third derivatives of a softmax weight along |u| <= 1 are below 6; route's weights are good to 1e-6
    tol = np.abs(f64(g)).sum(1) * (h * h + 1e-6 / h)
    assert np.all(np.abs(got - want) <= tol), np.abs(got - want) / tol


def _calls(gpu, b):
    ids = torch.arange(b.T * b.k, dtype=torch.int32, device="cuda").view(b.T, b.k) % 16
    def run():
        rows, pair_rows = gpu.moe_permute(b.x, b.pairs, b.k)
        dx = gpu.moe_permute_backward(b.dz, pair_rows, b.k)
        y = gpu.moe_unpermute(b.z, pair_rows, b.w)
        d_rows, d_w = gpu.moe_unpermute_backward(b.dy, b.z, b.pairs, pair_rows, b.w)
        return rows, pair_rows, dx, y, d_rows, d_w, gpu.moe_route_backward(ids, b.w, d_w, 16)
    return run


@pytest.mark.parametrize("T", [4, 300, 33000])
def test_captured_and_replayed(gpu, T):
    b = Batch(T, 96 if T < 1000 else 8, 8, 2, "bf16", seed=3)
    b.z.nan_to_num_(), b.dz.nan_to_num_()
    run = _calls(gpu, b)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        run()
    torch.cuda.current_stream().wait_stream(s)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        kept = run()
    for rep in range(4):
        for t in (b.x, b.z, b.dz, b.dy):
            t.copy_(torch.randn(t.shape, generator=torch.Generator().manual_seed(rep)))
        b.pairs.copy_(b.pairs.flip(0))
        eager = [t.clone() for t in run()]
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        for a, c in zip(kept, eager):
            assert torch.equal(a, c), rep


def test_on_another_stream(gpu):
    b = Batch(500, 512, 8, 4, "bf16", seed=4)
    want = _calls(gpu, b)()
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    for stream in (s, s.cuda_stream):
        rows, pair_rows = gpu.moe_permute(b.x, b.pairs, b.k, stream=stream)
        dx = gpu.moe_permute_backward(b.dz, pair_rows, b.k, stream=stream)
        y = gpu.moe_unpermute(b.z, pair_rows, b.w, stream=stream)
        d_rows, d_w = gpu.moe_unpermute_backward(b.dy, b.z, b.pairs, pair_rows, b.w, stream=stream)
        s.synchronize()
        for a, c in zip((rows, pair_rows, dx, y, d_rows, d_w), want):
            assert torch.equal(a, c)


def test_rows_past_32_bit_offsets(gpu):
    """R * H above 2^31 elements: the last rows are found."""
    T, H, k = 600_000, 4096, 1
    x = torch.zeros((T, H), dtype=torch.bfloat16, device="cuda")
    x[:, 0] = torch.arange(T, device="cuda") % 251
    x[:, -1] = torch.arange(T, device="cuda") % 241
    pairs = torch.arange(T - 1, -1, -1, dtype=torch.int32, device="cuda")
    rows, pair_rows = gpu.moe_permute(x, pairs, k)
    assert torch.equal(pair_rows, pairs)
    assert torch.equal(rows[:, 0], x[:, 0].flip(0)) and torch.equal(rows[:, -1], x[:, -1].flip(0))
    w = torch.full((T, 1), 0.5, device="cuda")
    y = gpu.moe_unpermute(rows, pair_rows, w)
    assert torch.equal(y, x * 0.5)
    d_rows, d_w = gpu.moe_unpermute_backward(x, rows, pairs, pair_rows, w, d_rows=y)
    assert torch.equal(d_rows[:, -1], (x[:, -1] * 0.5).flip(0))
    assert torch.equal(d_w[:, 0], x[:, 0].float() ** 2 + x[:, -1].float() ** 2)


def unpermute_f64(b, dy=None):
    """y, or with dy the gradients, in float64 on the GPU, each with the sum of its terms' magnitudes."""
    at = torch.from_numpy(b.pair_rows_host).cuda()
    here = (at >= 0)[:, None]
    z = torch.where(here, b.z.double()[at.clamp_min(0)], 0.0).view(b.T, b.k, b.H)
    w = b.w.double()[..., None]
    if dy is None:
        return (w * z).sum(1), (w * z).abs().sum(1)
    d_rows = torch.zeros((b.R, b.H), dtype=torch.float64, device="cuda")
    d_rows[at[here[:, 0]]] = (w * dy.double()[:, None]).reshape(-1, b.H)[here[:, 0]]
    p = z * dy.double()[:, None]
    return d_rows, p.sum(2), p.abs().sum(2)


WIDE = [  # T, H, E, k, dtype, local, pad
    (200, 2881, 16, 8, "f32", 11, 9),      # four waves a token, two rounds of four pairs
    (200, 2881, 40, 32, "bf16", 29, 9),    # ... eight rounds
    (63, 2880, 40, 32, "f16", None, 0),
    (130, 1030, 12, 5, "bf16", 7, 3),      # ... the second round holds one pair
    (4096, 2880, 32, 4, "bf16", None, 0),  # a wave a token, several pieces a lane, four pairs
    (4100, 2883, 32, 4, "bf16", 20, 50),
    (4100, 1001, 16, 6, "f32", 9, 70),     # ... two rounds
    (5000, 2880, 16, 3, "f16", 5, 0),
]


@pytest.mark.parametrize("case", WIDE, ids=["-".join(map(str, c)) for c in WIDE])
def test_unpermute_and_gradients_of_wide_rows(gpu, case):
    T, H, E, k, dtype, local, pad = case
    b = Batch(T, H, E, k, dtype, local, pad, seed=T + H + k)
    print(f"[unpermute wide] {case}", flush=True)
    want, mag = (v.cpu().numpy() for v in unpermute_f64(b))
    assert_rounded(gpu.moe_unpermute(b.z, b.pair_rows, b.w), want, k * U32 * mag, b.dtype, "y")
    d_rows, d_w = gpu.moe_unpermute_backward(b.dy, b.z, b.pairs, b.pair_rows, b.w)
    want, want_w, mag = (v.cpu().numpy() for v in unpermute_f64(b, b.dy))
    assert_rounded(d_rows, want, U32 * np.abs(want), b.dtype, "d_rows")
    assert_rounded(d_w, want_w, (H + 1) * U32 * mag, torch.float32, "d_weights")
    again = gpu.moe_unpermute_backward(b.dy, b.z, b.pairs, b.pair_rows, b.w)
    assert torch.equal(again[0], d_rows) and torch.equal(again[1], d_w)
