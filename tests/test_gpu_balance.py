"""The router's balance loss with the experts' counts (moe_balance_loss) and its gradient against the
float64 oracle.

u = 2^-24.  A logit less the row's largest has one rounding, its exponential log2(e)
times that and one step, and a product and a step more: with logits within 30 of the
largest (64 + 4) u; the sum over E adds E / 16 + 5 additions, the division and product 3:
(80 + E / 16) u a probability.  Sums over tokens: one u an addition.
"""

import math

import numpy as np
import pytest
import torch

from oracle import layer_ops as L
from tests.op_helpers import U, f64

pytestmark = pytest.mark.gpu


def case(T, E, k, seed=0, masked=False):
    rng = np.random.default_rng(seed)
    logits = rng.standard_normal((T, E)) - 0.5 * np.log(np.arange(1, E + 1))
    ids = np.argsort(-logits, axis=1, kind="stable")[:, :k].astype(np.int32)
    mask = rng.random(T) < 0.7 if masked else None
    lg = torch.from_numpy(logits).float().cuda()
    return lg, torch.from_numpy(ids.copy()).cuda(), None if mask is None else torch.from_numpy(mask).cuda()


def check(gpu, lg, ids, mask, g=0.37):
    T, E = lg.shape
    m = None if mask is None else mask.cpu().numpy()
    loss, counts, density = gpu.moe_balance_loss(lg, ids, mask)
    want, c, d = L.balance_loss(f64(lg), ids.cpu().numpy(), m)
    assert loss.shape == () and counts.dtype == torch.int32 and np.array_equal(counts.cpu().numpy(), c)
    assert np.all(np.abs(f64(density) - d) <= 8 * U * d)
    assert abs(float(loss) - want) <= (100 + E / 16 + min(T, 2048) + 300) * U * want + 1e-30
    base = torch.from_numpy(np.random.default_rng(9).standard_normal((T, E))).float().cuda()
    d_loss = torch.tensor(g, device="cuda")
    dl, mag = L.balance_loss_backward(f64(lg), f64(density), float(d_loss), m)
    slack = 3 * (100 + E / 8) * U * mag
    got = gpu.moe_balance_loss_backward(lg, density, d_loss, mask)
    assert np.all(np.abs(f64(got) - dl) <= slack + U * np.abs(dl) + 1e-37)
    added = gpu.moe_balance_loss_backward(lg, density, d_loss, mask, base)
    assert np.all(np.abs(f64(added) - dl - f64(base)) <= slack + U * (np.abs(dl) + np.abs(f64(base))))
    if mask is not None:
        assert torch.all(got[~mask] == 0) and torch.equal(added[~mask], base[~mask])
    inplace = base.clone()
    assert gpu.moe_balance_loss_backward(lg, density, d_loss, mask, inplace, out=inplace) is inplace
    assert torch.equal(inplace, added)
    again = gpu.moe_balance_loss(lg, ids, mask)
    assert torch.equal(again[0], loss) and torch.equal(again[1], counts) and torch.equal(again[2], density)


SIZES = [(1, 1, 1), (1, 8, 2), (5, 3, 3), (64, 32, 4), (65, 33, 4), (256, 32, 4), (1000, 64, 8), (777, 65, 3),
         (512, 31, 4), (513, 32, 4), (9, 5, 2), (256, 66, 4), (257, 128, 4), (70, 500, 3), (17000, 1, 1),
         (300, 127, 4), (4096, 128, 4), (130, 129, 2), (515, 512, 32), (33000, 10, 2), (20000, 200, 1)]


@pytest.mark.parametrize("masked", [False, True])
@pytest.mark.parametrize("T,E,k", SIZES)
def test_balance(gpu, T, E, k, masked):
    print(f"[balance] {T} {E} {k} {masked}", flush=True)
    check(gpu, *case(T, E, k, seed=T + E, masked=masked))


def test_nothing_counts(gpu):
    lg, ids, _ = case(300, 16, 2)
    none = torch.zeros(300, dtype=torch.bool, device="cuda")
    loss, counts, density = gpu.moe_balance_loss(lg, ids, none)
    assert float(loss) == 0 and torch.all(counts == 0) and torch.all(density == 0)
    one = torch.ones((), device="cuda")
    assert torch.all(gpu.moe_balance_loss_backward(lg, density, one, none) == 0)
    loss, counts, density = gpu.moe_balance_loss(lg, torch.full_like(ids, -1))  # no pick
    assert float(loss) == 0 and torch.all(counts == 0) and torch.all(density == 0)
    empty = torch.zeros((0, 16), device="cuda")
    loss, counts, density = gpu.moe_balance_loss(empty, torch.zeros((0, 2), dtype=torch.int32, device="cuda"))
    assert float(loss) == 0 and torch.all(counts == 0)
    assert gpu.moe_balance_loss_backward(empty, density, one).shape == (0, 16)


def test_masked_logits(gpu):
    """Experts of -infinity have no probability and no gradient, a token of them alone neither; a NaN
    stays with its token in the gradient, and does not pass where the mask leaves its token out."""
    lg, ids, _ = case(200, 24, 2)
    lg[3:9, 4:] = -math.inf
    lg[11] = -math.inf
    check(gpu, lg, ids, None)
    mask = torch.ones(200, dtype=torch.bool, device="cuda")
    mask[20] = mask[21] = False
    clean = gpu.moe_balance_loss(lg, ids, mask)
    lg[20], lg[21] = math.nan, math.inf
    for a, b in zip(gpu.moe_balance_loss(lg, ids, mask), clean):
        assert torch.equal(a, b)
    d = gpu.moe_balance_loss_backward(lg, clean[2], torch.ones((), device="cuda"), mask)
    assert torch.all(d[20:22] == 0) and torch.all(torch.isfinite(d))
    d = gpu.moe_balance_loss_backward(lg, clean[2], torch.ones((), device="cuda"))
    assert torch.all(torch.isnan(d[20:22])) and torch.all(torch.isfinite(d[:20])) and torch.all(torch.isfinite(d[22:]))


def test_picks_outside_count_for_none(gpu):
    lg, ids, mask = case(500, 12, 3, masked=True)
    ids[::7, 1] = -1
    ids[::5, 2] = 12
    ids[1] = 4  # the same expert three times
    check(gpu, lg, ids, mask)


def test_gradient_against_differences(gpu):
    """Central differences of the loss itself, with the counts held fixed."""
    lg, ids, mask = case(40, 8, 2, masked=True)
    _, _, density = gpu.moe_balance_loss(lg, ids, mask)
    d = f64(gpu.moe_balance_loss_backward(lg, density, torch.ones((), device="cuda"), mask))
    h, m = 1e-2, mask.cpu().numpy()
    for t, e in ((0, 0), (3, 5), (17, 2), (39, 7)):
        hi, lo = lg.clone(), lg.clone()
        hi[t, e] += h
        lo[t, e] -= h
        step = float((hi[t, e] - lo[t, e]).double())
        diff = (L.balance_loss(f64(hi), ids.cpu().numpy(), m)[0] - L.balance_loss(f64(lo), ids.cpu().numpy(), m)[0]) / step
        # the difference's own error: h^2 / 6 of the third derivative, at most the density's range
        assert abs(diff - d[t, e]) <= h * h * float(density.max()) + 1e-6


def test_streams_and_graph(gpu):
    lg, ids, mask = case(9000, 128, 4, masked=True)
    lg2, ids2, _ = case(9000, 128, 4, seed=5)
    g = torch.tensor(0.01, device="cuda")

    def step(a, b, **kw):
        loss, counts, density = gpu.moe_balance_loss(a, b, mask, **kw)
        return [loss, counts, density, gpu.moe_balance_loss_backward(a, density, g, mask, a, **kw)]

    want, other = step(lg, ids), step(lg2, ids2)
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(3):
        got, got2 = step(lg, ids, stream=s1), step(lg2, ids2, stream=s2)
    torch.cuda.synchronize()
    for a, b in zip(want + other, got + got2):
        assert torch.equal(a, b)
    a, b = lg.clone(), ids.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step(a, b)
    for i in range(4):
        a.copy_(lg if i % 2 else lg2)
        b.copy_(ids if i % 2 else ids2)
        graph.replay()
        eager = step(lg, ids) if i % 2 else step(lg2, ids2)
        torch.cuda.synchronize()
        for p, q in zip(out, eager):
            assert torch.equal(p, q)


def test_refusals(gpu):
    lg, ids, mask = case(10, 8, 2, masked=True)
    with pytest.raises(ValueError, match="shape"):
        gpu.moe_balance_loss(lg, ids[:9])
    with pytest.raises(TypeError):
        gpu.moe_balance_loss(lg, ids.long())
    with pytest.raises(TypeError):
        gpu.moe_balance_loss(lg, ids, mask.float())
    with pytest.raises(gpu.MXFP4MoEError):
        gpu.moe_balance_loss(lg, torch.zeros((10, 9), dtype=torch.int32, device="cuda"))
    d = torch.ones(8, device="cuda")
    with pytest.raises(ValueError, match="one element"):
        gpu.moe_balance_loss_backward(lg, d, d)
    with pytest.raises(ValueError, match="shares memory"):
        gpu.moe_balance_loss_backward(lg, d, d[0], out=lg)
    flat = torch.zeros(90, device="cuda")
    with pytest.raises(ValueError, match="shares memory"):
        gpu.moe_balance_loss_backward(lg, d, d[0], None, flat[:80].view(10, 8), out=flat[8:88].view(10, 8))
