"""Shared by the tests of the operators around the expert products."""

import numpy as np
import torch

from oracle import layer_ops as L

U = 2.0 ** -24
TYPES = [torch.bfloat16, torch.float16, torch.float32]


def f64(t):
    return t.detach().double().cpu().numpy()


def normal(seed, *shape, dtype=torch.float32, scale=1.0):
    return (torch.from_numpy(np.random.default_rng(seed).standard_normal(shape)) * scale).to(dtype).cuda()


def half_step(want, dtype):
    """Half a step of dtype around `want` (fp32 is what the kernels compute in: its own half step)."""
    info = torch.finfo(dtype)
    return np.abs(want) * info.eps / 2 + info.tiny * info.eps / 2


def assert_near(got, want, slack, dtype, label=""):
    g = f64(got)
    bound = slack + half_step(np.abs(want) + slack, dtype)
    assert g.shape == want.shape and np.all(np.isfinite(g)), label
    off = np.abs(g - want) - bound
    assert off.size == 0 or off.max() <= 0, f"{label}: {off.max():.3e} over its bound at {np.argwhere(off > 0)[:4].tolist()}"


def bytes_of(codes):
    return codes.view(torch.uint8).cpu().numpy()


def assert_codes_near(codes, scales, want, slack, label=""):
    """Codes and scales of rows whose exact values are `want`, up to slack (relative)."""
    s = f64(scales)
    exact = L.block_scales(want)
    assert np.all(np.abs(s - exact) <= (slack + 2 * U) * exact), f"{label} scales"
    wide = np.repeat(exact, 128, axis=1)[:, : want.shape[1]]
    # half a step of e4m3: 2^-4 of the value, or half of the smallest subnormal 2^-9
    bound = np.maximum(np.abs(want) * 2.0 ** -4, wide * 2.0 ** -10) + 2 * (slack + 8 * U) * np.abs(want)
    off = np.abs(L.values(bytes_of(codes), s) - want) - bound
    assert off.size == 0 or off.max() <= 0, f"{label} codes: {off.max():.3e} at {np.argwhere(off > 0)[:4].tolist()}"
