"""The short host path of the new entry points (csrc/host_calls.cpp) against the step-by-step one:
the same bits for the calls it takes, the same errors for those it leaves."""

import pytest
import torch

pytestmark = pytest.mark.gpu


def _inputs(T=9, H=40, k=3, E=6, N=24, K=64):
    g = torch.Generator("cuda").manual_seed(1)
    d = {"x": torch.randn((T, H), generator=g, device="cuda").bfloat16(),
         "pairs": torch.randperm(T * k, generator=g, device="cuda").to(torch.int32),
         "w": torch.rand((T, k), generator=g, device="cuda"), "dw": torch.randn((T, k), generator=g, device="cuda"),
         "ids": torch.randint(0, E, (T, k), generator=g, device="cuda", dtype=torch.int32),
         "rows": torch.randn((T * k, H), generator=g, device="cuda").bfloat16(),
         "lx": torch.randn((T * k, K), generator=g, device="cuda").bfloat16(),
         "ly": torch.randn((T * k, N), generator=g, device="cuda").bfloat16(),
         "blocks": torch.randint(0, 256, (E, N, K // 2), generator=g, device="cuda", dtype=torch.uint8),
         "s32": torch.randint(120, 130, (E, N, K // 32), generator=g, device="cuda", dtype=torch.uint8),
         "s16": torch.randint(0x30, 0x48, (E, N, K // 16), generator=g, device="cuda", dtype=torch.uint8),
         "scale2": torch.rand(E, generator=g, device="cuda"), "bias": torch.zeros((E, N), device="cuda").bfloat16(),
         "off": torch.arange(E + 1, device="cuda", dtype=torch.int32) * (T * k) // E}
    return d, k, E


def _calls(gpu, d, k, E):
    off = d["off"].to(torch.int32)
    pr = gpu.moe_permute(d["x"], d["pairs"], k)[1]
    return {
        "permute": lambda: gpu.moe_permute(d["x"], d["pairs"], k),
        "permute_backward": lambda: gpu.moe_permute_backward(d["rows"], pr, k),
        "unpermute": lambda: gpu.moe_unpermute(d["rows"], pr, d["w"]),
        "unpermute_backward": lambda: gpu.moe_unpermute_backward(d["x"], d["rows"], d["pairs"], pr, d["w"]),
        "route_backward": lambda: gpu.moe_route_backward(d["ids"], d["w"], d["dw"], E),
        "mxfp4": lambda: gpu.moe_mxfp4_linear(d["lx"], d["blocks"], d["s32"], d["bias"], off),
        "mxfp4_dense": lambda: gpu.moe_mxfp4_linear(d["lx"], d["blocks"][1], d["s32"][1]),
        "mxfp4_backward": lambda: gpu.moe_mxfp4_linear_backward(d["ly"], d["blocks"], d["s32"], off),
        "nvfp4": lambda: gpu.moe_nvfp4_linear(d["lx"], d["blocks"], d["s16"], d["scale2"], None, off),
        "nvfp4_backward": lambda: gpu.moe_nvfp4_linear_backward(d["ly"], d["blocks"], d["s16"], d["scale2"], off),
    }


def _list(v):
    return list(v) if isinstance(v, tuple) else [v]


def test_same_results_as_step_by_step(gpu, monkeypatch):
    calls = _calls(gpu, *_inputs())
    assert gpu._host is not None, "the module of the short host path is not built"
    short = {n: _list(f()) for n, f in calls.items()}
    monkeypatch.setattr(gpu, "_host", None)
    for n, f in calls.items():
        for a, b in zip(short[n], _list(f())):
            assert a.shape == b.shape and a.dtype == b.dtype and torch.equal(a, b), n


def test_plain_calls_are_taken(gpu):
    d, k, E = _inputs()
    h = gpu._host
    rows, pr = h.permute(d["x"], d["pairs"], k)
    assert h.permute_backward(d["rows"], pr, k) is not None and h.unpermute(d["rows"], pr, d["w"]) is not None
    assert h.unpermute_backward(d["x"], d["rows"], d["pairs"], pr, d["w"]) is not None
    assert h.route_backward(d["ids"], d["w"], d["dw"], E) is not None
    assert h.linear(False, 32, d["lx"], d["blocks"][0], d["s32"][0], None, None, None) is not None
    leaf = d["x"].clone().requires_grad_()
    assert not gpu.moe_permute(leaf, d["pairs"], k)[0].requires_grad


@pytest.mark.parametrize("short", [True, False])
def test_refusals(gpu, monkeypatch, short):
    d, k, E = _inputs()
    if not short:
        monkeypatch.setattr(gpu, "_host", None)
    x, pairs, w, rows = d["x"], d["pairs"], d["w"], d["rows"]
    pr = gpu.moe_permute(x, pairs, k)[1]
    with pytest.raises(ValueError, match="contiguous"):
        gpu.moe_permute(x.t(), pairs, k)
    with pytest.raises(ValueError, match="contiguous"):
        gpu.moe_unpermute(rows, pr, d["w"].t().contiguous().t())
    with pytest.raises(TypeError):
        gpu.moe_permute(x.double(), pairs, k)
    with pytest.raises(TypeError):
        gpu.moe_permute(x, pairs.long(), k)
    with pytest.raises((ValueError, TypeError)):
        gpu.moe_permute(x, pairs.cpu(), k)
    with pytest.raises(ValueError):
        gpu.moe_permute(x, pairs, 0)
    with pytest.raises(gpu.MXFP4MoEError):
        gpu.moe_permute(x, pairs, 33)
    with pytest.raises(ValueError):
        gpu.moe_permute_backward(rows, pr, 2 * k + 1)
    with pytest.raises(ValueError):
        gpu.moe_unpermute(rows, pr[:-1], w)
    with pytest.raises(TypeError):
        gpu.moe_unpermute_backward(x.float(), rows, pairs, pr, w)
    with pytest.raises(ValueError):
        gpu.moe_route_backward(d["ids"][:, :2].contiguous(), w, d["dw"], E)
    with pytest.raises(gpu.MXFP4MoEError):
        gpu.moe_route_backward(d["ids"], w, d["dw"], 513)
    with pytest.raises(ValueError):
        gpu.moe_mxfp4_linear(d["lx"][:, :32].contiguous(), d["blocks"][0], d["s32"][0])
    with pytest.raises(ValueError):
        gpu.moe_mxfp4_linear(d["lx"], d["blocks"][0], d["s16"][0])
    with pytest.raises(ValueError):
        gpu.moe_mxfp4_linear(d["lx"], d["blocks"], d["s32"])
    with pytest.raises((ValueError, TypeError)):
        gpu.moe_nvfp4_linear(d["lx"], d["blocks"], d["s16"], None, None, d["off"])
    with pytest.raises(gpu.MXFP4MoEError):  # K = 48: no whole group
        gpu.moe_mxfp4_linear(torch.zeros((2, 48), device="cuda").bfloat16(),
                             torch.zeros((4, 24), dtype=torch.uint8, device="cuda"),
                             torch.zeros((4, 1), dtype=torch.uint8, device="cuda"))
    flat = torch.zeros(2 * 64 + 4, device="cuda").bfloat16()
    with pytest.raises(gpu.MXFP4MoEError):  # x off its 16-byte alignment
        gpu.moe_mxfp4_linear(flat[4:].view(2, 64), d["blocks"][0], d["s32"][0])


def test_another_stream_is_current(gpu):
    d, k, E = _inputs(T=2000, H=512)
    want = _list(gpu.moe_permute(d["x"], d["pairs"], k))
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        got = _list(gpu.moe_permute(d["x"], d["pairs"], k))
    s.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_torch_makes_the_outputs_where_a_mode_looks_at_them(gpu):
    """New tensors filled under deterministic algorithms, and modes that see every call of torch."""
    from torch.utils._python_dispatch import TorchDispatchMode

    rng = torch.Generator("cuda").manual_seed(2)
    blocks = torch.randint(0, 256, (2, 40, 32), generator=rng, device="cuda", dtype=torch.uint8)
    scales = torch.full((2, 40, 2), 127, dtype=torch.uint8, device="cuda")
    x = torch.randn((9, 64), generator=rng, device="cuda").bfloat16()
    offsets = torch.tensor([1, 4, 7], dtype=torch.int32, device="cuda")
    want = gpu.moe_mxfp4_linear(x, blocks, scales, None, offsets)[1:7].clone()
    was = torch.are_deterministic_algorithms_enabled()
    try:
        torch.use_deterministic_algorithms(True)
        y = gpu.moe_mxfp4_linear(x, blocks, scales, None, offsets)
    finally:
        torch.use_deterministic_algorithms(was)
    assert torch.equal(y[1:7], want) and bool(torch.isnan(y[[0, 7, 8]]).all())

    class Seen(TorchDispatchMode):
        names = []

        def __torch_dispatch__(self, func, types, args=(), kwargs=None):
            self.names.append(str(func))
            return func(*args, **(kwargs or {}))

    with Seen():
        y = gpu.moe_mxfp4_linear(x, blocks, scales, None, offsets)
    assert any("empty" in n for n in Seen.names)
    assert torch.equal(y[1:7], want)


def test_outputs_that_share_memory_with_an_input_are_refused(gpu):
    """The kernels read and write in no order of their own: such a call would race with itself."""
    d, k, E = _inputs(T=8, H=64, k=1, N=64, K=64)
    x, pairs, w, off = d["x"], d["pairs"], d["w"], d["off"].to(torch.int32)
    pr = gpu.moe_permute(x, pairs, k)[1]
    both = torch.zeros(2 * x.numel() - 8, dtype=x.dtype, device="cuda")
    first, second = both[:x.numel()].view_as(x), both[x.numel() - 8:].view_as(x)  # overlapping by a piece
    lx, ly = d["lx"], d["ly"]
    calls = [
        lambda: gpu.moe_permute(x, pairs, k, out=x),
        lambda: gpu.moe_permute(first, pairs, k, out=second),
        lambda: gpu.moe_permute(second, pairs, k, out=first),
        lambda: gpu.moe_permute(x, pairs, k, pair_rows=pairs),
        lambda: gpu.moe_permute_backward(x, pr, k, out=x),
        lambda: gpu.moe_unpermute(x, pr, w, out=x),
        lambda: gpu.moe_unpermute_backward(d["rows"], x, pairs, pr, w, d_rows=x),
        lambda: gpu.moe_unpermute_backward(x, d["rows"], pairs, pr, w, d_rows=x),
        lambda: gpu.moe_unpermute_backward(x, d["rows"], pairs, pr, w, d_weights=w),
        lambda: gpu.moe_route_backward(d["ids"], w, d["dw"], 1, out=w),
        lambda: gpu.moe_route_backward(d["ids"], w, d["dw"], 1, out=d["dw"]),
        lambda: gpu.moe_mxfp4_linear(lx, d["blocks"], d["s32"], None, off, out=lx),
        lambda: gpu.moe_nvfp4_linear(lx, d["blocks"], d["s16"], d["scale2"], None, off, out=lx),
        lambda: gpu.moe_mxfp4_linear_backward(ly, d["blocks"], d["s32"], off, out=ly),
        lambda: gpu.moe_nvfp4_linear_backward(ly, d["blocks"], d["s16"], d["scale2"], off, out=ly),
    ]
    before = {n: t.clone() for n, t in d.items()}
    for i, f in enumerate(calls):
        with pytest.raises(ValueError, match="shares memory"):
            f()
            pytest.fail(f"call {i} was taken")
    assert all(torch.equal(d[n], t) for n, t in before.items())
    ends = both[:x.numel() - 8].view(-1, 8)  # side by side is no overlap
    rows, _ = gpu.moe_permute(ends, torch.arange(len(ends), device="cuda", dtype=torch.int32), 1,
                              out=both[x.numel() - 8:][:ends.numel()].view_as(ends))
    assert torch.equal(rows, ends)
