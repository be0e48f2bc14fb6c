"""Pins of oracle/layer_ops.py: torch's own operators in float64, differences, closed forms."""

import numpy as np
import pytest
import torch

from oracle import layer_ops as L


def differences(f, x, at, step=1e-6):
    """d f / d x[i] for the indices in `at`, by central differences."""
    out = []
    for i in at:
        hi, lo = x.copy(), x.copy()
        hi[i] += step
        lo[i] -= step
        out.append((f(hi) - f(lo)) / (2 * step))
    return np.array(out)


def some(rng, shape, n=12):
    return [tuple(rng.integers(0, s) for s in shape) for _ in range(n)]


def test_e4m3_is_torchs():
    t = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(L.E4M3, t, equal_nan=True)


def test_norm_is_torchs_and_its_gradient_the_differences():
    rng = np.random.default_rng(0)
    s, w, dy, ds = rng.standard_normal((5, 9)), rng.standard_normal(9), rng.standard_normal((5, 9)), rng.standard_normal((5, 9))
    y, r = L.rms_norm(s, w, 1e-3)
    want = torch.nn.functional.rms_norm(torch.tensor(s), (9,), torch.tensor(w), 1e-3)
    assert np.allclose(y, want.numpy(), rtol=1e-13)
    dx, mag, dw, wmag = L.rms_norm_backward(dy, s, w, 1e-3, ds)
    at = some(rng, s.shape)
    got = differences(lambda v: np.sum(L.rms_norm(v, w, 1e-3)[0] * dy) + np.sum(v * ds), s, at)
    assert np.allclose(got, [dx[i] for i in at], atol=1e-8)
    got = differences(lambda v: np.sum(L.rms_norm(s, v, 1e-3)[0] * dy), w, [(i,) for i in range(9)])
    assert np.allclose(got, dw, atol=1e-8)
    assert np.all(mag >= np.abs(dx) - 1e-12) and np.all(wmag >= np.abs(dw) - 1e-12)


@pytest.mark.parametrize("split", [False, True])
@pytest.mark.parametrize("alpha,limit,offset", [(1.702, 7.0, 1.0), (1.0, np.inf, 0.0), (0.7, 0.5, -0.3)])
def test_swiglu_and_its_gradient(split, alpha, limit, offset):
    rng = np.random.default_rng(1)
    h, da = 4 * rng.standard_normal((3, 10)), rng.standard_normal((3, 5))
    gate, up = L.halves(h, split)
    assert np.shares_memory(gate, h)
    a = L.swiglu(h, split, alpha, limit, offset)
    if limit == np.inf:
        want = torch.nn.functional.silu(torch.tensor(gate.copy())) * torch.tensor(up.copy())
        assert np.allclose(a, want.numpy(), rtol=1e-13)
    dh, mag = L.swiglu_backward(da, h, split, alpha, limit, offset)
    at = [(i, j) for i in range(3) for j in range(10)]
    got = differences(lambda v: np.sum(L.swiglu(v, split, alpha, limit, offset) * da), h, at)
    assert np.allclose(got, [dh[i] for i in at], atol=1e-7)
    assert np.all(mag >= np.abs(dh) - 1e-12)


def test_swiglu_is_the_layers():
    """The defaults are the fused layer's activation."""
    from oracle import mxfp4_moe as O

    h = 5 * np.random.default_rng(2).standard_normal((4, 12))
    assert np.allclose(L.swiglu(h, False, 1.702, 7.0, 1.0), O.swiglu_clamped(h[:, 0::2], h[:, 1::2]), rtol=1e-13)


def test_balance_loss_closed_forms_and_gradient():
    rng = np.random.default_rng(3)
    logits, ids = rng.standard_normal((7, 5)), rng.integers(0, 5, (7, 2))
    mask = np.array([1, 0, 1, 1, 1, 0, 1], bool)
    loss, counts, density = L.balance_loss(logits, ids, mask)
    p = torch.softmax(torch.tensor(logits[mask]), 1).mean(0).numpy()
    share = np.bincount(ids[mask].reshape(-1), minlength=5) / (2 * mask.sum())
    assert np.isclose(loss, 5 * np.sum(p * share)) and counts.sum() == 2 * mask.sum()
    # even shares: 1 whatever the probabilities are
    assert np.isclose(L.balance_loss(rng.standard_normal((4, 4)), np.arange(4)[:, None])[0], 1.0)
    d, mag = L.balance_loss_backward(logits, density, 0.3, mask)
    at = some(rng, logits.shape)
    got = differences(lambda v: 0.3 * np.sum(L.probabilities(v)[mask] * density), logits, at)
    assert np.allclose(got, [d[i] for i in at], atol=1e-9) and np.all(d[~mask] == 0) and np.all(mag >= np.abs(d))
    # no token, no pick, no finite logit
    assert L.balance_loss(logits, ids, np.zeros(7, bool))[0] == 0 and L.balance_loss(logits, ids + 9)[0] == 0
    assert np.all(L.probabilities(np.full((1, 3), -np.inf)) == 0)


def test_blocks_of_128():
    v = np.zeros((2, 300))
    v[0, 130], v[1, 299] = -896.0, 2.0
    s = L.block_scales(v)
    assert s.shape == (2, 3) and s[0, 1] == 2.0 and s[1, 2] == 2.0 / 448 and s[0, 0] == 2.0 ** -100 / 448
    codes = np.full((2, 300), 0x38)  # 1.0
    assert np.all(L.values(codes, s)[0, 128:256] == 2.0)
    w = L.weights(np.full((200, 300), 0xB8), np.arange(6.0).reshape(2, 3))  # -1.0
    assert w[127, 127] == 0 and w[127, 128] == -1 and w[128, 299] == -5
