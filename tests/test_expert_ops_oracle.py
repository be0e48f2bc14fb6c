"""Pins of oracle/expert_ops.py against facts fixed outside it (CPU only): torch's own
operations and autograd in float64, central differences, hand-written cases, and the
fused layer's oracle."""

import numpy as np
import pytest
import torch

from mxfp4_quantized_expert_amd import workloads as W
from oracle import expert_ops as X
from oracle import mxfp4_moe as O


def routed(rng, T, E, k):
    ids = np.stack([rng.permutation(E)[:k] for _ in range(T)])
    order = np.argsort(ids.reshape(-1), kind="stable")
    return ids, rng.random((T, k)), order, np.concatenate([[0], np.cumsum(np.bincount(ids.reshape(-1), minlength=E))])


def test_permute_by_hand():
    x = np.array([[1.0, 2.0], [3.0, 4.0]])
    rows, at = X.permute(x, [3, -1, 0, 4, 3], 2)  # -1 and 4 are no pairs, pair 3 is listed twice
    assert rows.tolist() == [[3, 4], [0, 0], [1, 2], [0, 0], [3, 4]]
    assert at.tolist() == [2, -1, -1, 4]


def test_permute_is_an_index_and_unpermute_its_adjoint():
    rng = np.random.default_rng(0)
    T, E, k, H = 13, 5, 3, 7
    _, w, order, _ = routed(rng, T, E, k)
    x = rng.standard_normal((T, H))
    rows, at = X.permute(x, order, k)
    assert np.array_equal(rows, x[order // k]) and np.array_equal(at[order], np.arange(T * k))
    g = rng.standard_normal(rows.shape)
    back, _ = X.unpermute(g, at, np.ones((T, k)))
    assert np.isclose(np.vdot(back, x), np.vdot(g, rows), rtol=1e-13)
    y, mag = X.unpermute(rows, at, w)  # rows of a token are its x
    assert np.allclose(y, x * w.sum(1, keepdims=True), rtol=1e-14)
    assert np.allclose(mag, np.abs(x) * w.sum(1, keepdims=True), rtol=1e-14)


def test_unpermute_backward_against_autograd_and_differences():
    rng = np.random.default_rng(1)
    T, E, k, H = 9, 4, 2, 6
    ids, w, order, _ = routed(rng, T, E, k)
    order = order[ids.reshape(-1)[order] < 3]            # a share of the experts
    pairs = np.concatenate([order, [-1, T * k]])         # and rows of padding
    _, at = X.permute(np.zeros((T, H)), pairs, k)
    rows, dy = rng.standard_normal((len(pairs), H)), rng.standard_normal((T, H))
    d_rows, d_w, _ = X.unpermute_backward(dy, rows, pairs, at, w)
    r, v = torch.from_numpy(rows).requires_grad_(), torch.from_numpy(w).requires_grad_()
    picked = torch.cat([r, torch.zeros(1, H, dtype=torch.float64)])[torch.from_numpy(at)]  # -1: the zero row
    y = (picked.reshape(T, k, H) * v[..., None]).sum(1)
    assert np.allclose(X.unpermute(rows, at, w)[0], y.detach().numpy(), rtol=1e-13)
    y.backward(torch.from_numpy(dy))
    assert np.allclose(d_rows, r.grad.numpy(), rtol=1e-13) and np.allclose(d_w, v.grad.numpy(), rtol=1e-12)
    assert not d_rows[-2:].any() and not d_w.reshape(-1)[at < 0].any()
    h = 1e-5
    for p in (0, 7, 11):
        up, down = w.copy(), w.copy()
        up.flat[p] += h
        down.flat[p] -= h
        slope = np.vdot(dy, X.unpermute(rows, at, up)[0] - X.unpermute(rows, at, down)[0]) / (2 * h)
        assert abs(slope - d_w.flat[p]) < 1e-8


def test_route_backward_against_autograd():
    rng = np.random.default_rng(2)
    logits = torch.from_numpy(rng.standard_normal((11, 7))).requires_grad_()
    top, ids = logits.topk(3, dim=1)
    w = torch.softmax(top, 1)
    dw = rng.standard_normal((11, 3))
    w.backward(torch.from_numpy(dw))
    got = X.route_backward(ids.numpy(), w.detach().numpy(), dw, 7)
    assert np.allclose(got, logits.grad.numpy(), rtol=1e-12, atol=1e-15)
    assert np.allclose(got.sum(1), 0, atol=1e-15)  # a softmax does not see a shift


@pytest.mark.parametrize("nv", [False, True])
def test_linear_against_autograd(nv):
    rng = np.random.default_rng(3)
    E, N, K = 3, 5, 64
    blocks = rng.integers(0, 256, (E, N, K // 2), dtype=np.uint8)
    scales = rng.integers(0x30, 0x49, (E, N, K // 16), dtype=np.uint8) if nv else \
        rng.integers(120, 131, (E, N, K // 32), dtype=np.uint8)
    s2 = np.array([0.5, 0.25, 2.0], np.float32) if nv else None
    w = X.weights_of(blocks, scales, s2)
    if nv:
        assert np.array_equal(w, O.nvfp4_dequantize_f64(blocks, scales) * np.array([0.5, 0.25, 2.0])[:, None, None])
    else:
        assert np.array_equal(w, O.dequantize_f64(blocks, scales))
    off, bias = [1, 4, 4, 9], rng.standard_normal((E, N))
    x = torch.from_numpy(rng.standard_normal((10, K))).requires_grad_()
    dy = rng.standard_normal((10, N))
    y, mag, written = X.linear(x.detach().numpy(), w, off, bias)
    dx, _, also = X.linear_backward(dy, w, off)
    owner = torch.tensor([0, 0, 0, 2, 2, 2, 2, 2])
    want = torch.bmm(torch.from_numpy(w)[owner], x[1:9, :, None])[..., 0] + torch.from_numpy(bias)[owner]
    assert np.allclose(y[1:9], want.detach().numpy(), rtol=1e-12) and np.all(mag[1:9] >= np.abs(y[1:9]) * (1 - 1e-12))
    want.backward(torch.from_numpy(dy[1:9]))
    assert np.allclose(dx[1:9], x.grad.numpy()[1:9], rtol=1e-12, atol=1e-13)
    assert written.tolist() == also.tolist() == [False] + [True] * 8 + [False] and not y[[0, 9]].any()


def test_chain_equals_the_fused_layer():
    spec = W.LAYERS["tiny"]
    layer, k = W.make_layer(spec, seed=5), spec.top_k
    ids, w = O.route(layer["router_logits"], k)
    _, off, order = O.group_by_expert(ids, spec.E)
    rows, at = X.permute(O.bf16_decode(layer["x"]), order, k)
    h = X.linear(rows, X.weights_of(layer["w13_blocks"], layer["w13_scales"]), off, O.bf16_decode(layer["w13_bias"]))[0]
    a = O.swiglu_clamped(h[:, 0::2], h[:, 1::2])
    z = X.linear(a, X.weights_of(layer["w2_blocks"], layer["w2_scales"]), off, O.bf16_decode(layer["w2_bias"]))[0]
    assert np.allclose(X.unpermute(z, at, w)[0], O.moe_forward(layer, k), rtol=1e-10, atol=1e-12)
