"""The short host path (csrc/host_calls.cpp) of the norm, the activation, the 8-bit products and the
balance loss against the step-by-step one: the same bits for the calls it takes, the same errors for
those it leaves, the current stream, two threads, and a backward pass recorded into a graph."""

import threading

import pytest
import torch

from tests.op_helpers import normal

pytestmark = pytest.mark.gpu

E4M3 = torch.float8_e4m3fn


def _inputs(T=9, H=144, k=2, E=4, N=40):
    d = {"x": normal(1, T, H, dtype=torch.bfloat16), "res": normal(2, T, H, dtype=torch.bfloat16),
         "w": normal(3, H), "dy": normal(4, T, H, dtype=torch.bfloat16), "h": normal(5, T, 2 * H, dtype=torch.float16),
         "da": normal(6, T, H, dtype=torch.float16), "lg": normal(7, T, E), "add": normal(8, T, E),
         "wq": (100 * normal(9, E, N, H)).to(E4M3), "ws": normal(10, E, 1, 2).abs(), "bias": normal(11, E, N, dtype=torch.bfloat16),
         "dn": normal(12, T, N, dtype=torch.bfloat16), "one": torch.ones((), device="cuda")}
    d["ids"] = torch.argsort(d["lg"], dim=1, descending=True)[:, :k].to(torch.int32).contiguous()
    d["mask"] = torch.arange(T, device="cuda") % 3 != 0
    d["off"] = torch.tensor([0, 2, 2, 7, T], dtype=torch.int32, device="cuda")
    return d


def _calls(gpu, d):
    c, sc = gpu.moe_fp8_quantize(d["x"])
    _, s, r = gpu.moe_rms_norm(d["x"], d["w"], d["res"])
    density = gpu.moe_balance_loss(d["lg"], d["ids"], d["mask"])[2]
    return {
        "norm": lambda: gpu.moe_rms_norm(d["x"], d["w"], d["res"]),
        "norm_alone": lambda: gpu.moe_rms_norm(d["x"], d["w"], eps=0.5),
        "norm_fp8": lambda: gpu.moe_rms_norm_fp8(d["x"], d["w"], d["res"]),
        "norm_fp8_alone": lambda: gpu.moe_rms_norm_fp8(d["x"], d["w"]),
        "norm_backward": lambda: gpu.moe_rms_norm_backward(d["dy"], s, d["w"], r, d["res"]),
        "norm_backward_alone": lambda: gpu.moe_rms_norm_backward(d["dy"], s, d["w"], r),
        "quantize": lambda: gpu.moe_fp8_quantize(d["h"]),
        "linear": lambda: gpu.moe_fp8_linear(c, sc, d["wq"], d["ws"], d["bias"], d["off"]),
        "linear_dense": lambda: gpu.moe_fp8_linear(c, sc, d["wq"][1], d["ws"][1]),
        "linear_backward": lambda: gpu.moe_fp8_linear_backward(d["dn"], d["wq"], d["ws"], d["off"]),
        "linear_backward_dense": lambda: gpu.moe_fp8_linear_backward(d["dn"], d["wq"][0], d["ws"][0]),
        "swiglu": lambda: gpu.moe_swiglu(d["h"]),
        "swiglu_split": lambda: gpu.moe_swiglu(d["h"], True, 1.0, float("inf"), 0.0),
        "swiglu_fp8": lambda: gpu.moe_swiglu_fp8(d["h"], True),
        "swiglu_backward": lambda: gpu.moe_swiglu_backward(d["da"], d["h"], alpha=1, limit=2, offset=0),
        "balance": lambda: gpu.moe_balance_loss(d["lg"], d["ids"], d["mask"]),
        "balance_all": lambda: gpu.moe_balance_loss(d["lg"], d["ids"]),
        "balance_backward": lambda: gpu.moe_balance_loss_backward(d["lg"], density, d["one"], d["mask"], d["add"]),
        "balance_backward_all": lambda: gpu.moe_balance_loss_backward(d["lg"], density, d["one"]),
    }


def _bytes(v):
    """Outputs for a comparison of bits, as whole numbers of their width: a weight that has no 8-bit
    code is NaN, and so are its outputs."""
    whole = {1: torch.uint8, 2: torch.int16, 4: torch.int32}
    return [t.view(whole[t.element_size()]) for t in (v if isinstance(v, tuple) else (v,))]


def test_same_results_as_step_by_step(gpu, monkeypatch):
    calls = _calls(gpu, _inputs())
    assert gpu._host is not None, "the module of the short host path is not built"
    taken = []

    class Spy:
        def __getattr__(self, name, host=gpu._host):
            def call(*a):
                got = getattr(host, name)(*a)
                taken.append(got is not None)
                return got
            return call

    monkeypatch.setattr(gpu, "_host", Spy())
    short = {n: f() for n, f in calls.items()}
    assert len(taken) == len(calls) and all(taken)
    monkeypatch.setattr(gpu, "_host", None)
    for n, f in calls.items():
        a, b = short[n], f()
        assert isinstance(a, tuple) == isinstance(b, tuple), n
        a, b = (v if isinstance(v, tuple) else (v,) for v in (a, b))
        assert len(a) == len(b), n
        for s, t in zip(a, b):
            assert s.shape == t.shape and s.dtype == t.dtype and s.device == t.device, n
            assert not s.requires_grad and not t.requires_grad
            assert torch.equal(*_bytes(s), *_bytes(t)), n


@pytest.mark.parametrize("short", [True, False])
def test_refusals(gpu, monkeypatch, short):
    if not short:
        monkeypatch.setattr(gpu, "_host", None)
    d = _inputs()
    x, w = d["x"], d["w"]
    c, sc = gpu.moe_fp8_quantize(x)
    for call in (lambda: gpu.moe_rms_norm(x.t(), w[:9].contiguous()), lambda: gpu.moe_rms_norm(x, w[1:]),
                 lambda: gpu.moe_rms_norm(x, w, d["res"][:3]), lambda: gpu.moe_rms_norm(x.double(), w),
                 lambda: gpu.moe_rms_norm_fp8(x, w.half()), lambda: gpu.moe_rms_norm(x.cpu(), w),
                 lambda: gpu.moe_rms_norm_backward(d["dy"], x, w, w), lambda: gpu.moe_fp8_quantize(x[:, ::2]),
                 lambda: gpu.moe_fp8_quantize(x.long()), lambda: gpu.moe_fp8_linear(c, sc, d["wq"], d["ws"]),
                 lambda: gpu.moe_fp8_linear(x, sc, d["wq"], d["ws"], None, d["off"]),
                 lambda: gpu.moe_fp8_linear(c, sc[:, :1], d["wq"][0], d["ws"][0]),
                 lambda: gpu.moe_fp8_linear(c, sc, d["wq"], d["ws"], None, d["off"].long()),
                 lambda: gpu.moe_fp8_linear(c, sc, d["wq"], d["ws"], d["bias"].float(), d["off"]),
                 lambda: gpu.moe_fp8_linear_backward(d["dn"].float(), d["wq"], d["ws"], d["off"]),
                 lambda: gpu.moe_swiglu(d["h"][:, 1:]), lambda: gpu.moe_swiglu(d["h"][:, 1:].contiguous()),
                 lambda: gpu.moe_swiglu_backward(d["da"].float(), d["h"]),
                 lambda: gpu.moe_balance_loss(d["lg"], d["ids"].long()),
                 lambda: gpu.moe_balance_loss(d["lg"], d["ids"], d["mask"][:5]),
                 lambda: gpu.moe_balance_loss_backward(d["lg"], w, d["one"])):
        with pytest.raises((ValueError, TypeError)):
            call()


def test_another_stream_is_current(gpu):
    d = _inputs(T=700)
    d["off"][-1] = 700
    want = [t for f in _calls(gpu, d).values() for t in _bytes(f())]
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        got = [t for f in _calls(gpu, d).values() for t in _bytes(f())]
    s.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_two_threads(gpu):
    """Each on a stream of its own, with the same inputs."""
    d = _inputs(T=300)
    d["off"][-1] = 300
    want = [t for f in _calls(gpu, d).values() for t in _bytes(f())]
    torch.cuda.synchronize()
    failed = []

    def work():
        s = torch.cuda.Stream()
        with torch.cuda.stream(s):
            for _ in range(10):
                got = [t for f in _calls(gpu, d).values() for t in _bytes(f())]
            s.synchronize()
        if not all(torch.equal(a, b) for a, b in zip(got, want)):
            failed.append(1)

    threads = [threading.Thread(target=work) for _ in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not failed


def test_every_call_in_a_graph(gpu):
    """Recorded together, replayed with eager calls of the same operators between the replays."""
    d = _inputs(T=600, E=40, k=4)
    d["off"] = torch.arange(41, device="cuda", dtype=torch.int32) * 15
    calls = _calls(gpu, d)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = [t for f in calls.values() for t in _bytes(f())]
    for i in range(4):
        d["lg"].add_(0.25)
        d["x"].neg_()
        d["h"].neg_()
        g.replay()
        eager = [t for f in calls.values() for t in _bytes(f())]
        torch.cuda.synchronize()
        for a, b in zip(out, eager):
            assert torch.equal(a, b)
