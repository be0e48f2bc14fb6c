"""Two threads at once through the norm, the activation, the 8-bit products and the balance loss, each
with inputs, sizes and results of its own, so that a workspace or an output that calls shared would show."""

import threading

import pytest
import torch

from tests.test_gpu_layer_host_calls import _bytes, _calls, _inputs

pytestmark = pytest.mark.gpu


def _of_a_thread(i):
    """More tokens of four experts than one block of the balance loss takes, and others in each thread."""
    T = (1500, 2300)[i]
    d = _inputs(T=T)
    d["off"][-1] = T
    if i:
        for name in ("x", "res", "dy", "h", "da", "dn", "add"):
            d[name] = d[name].flip(0).contiguous()
        d["lg"] = d["lg"].roll(1, 1).contiguous()
        d["mask"] = ~d["mask"]
    return d


@pytest.mark.parametrize("short", [True, False])
def test_two_threads_with_inputs_of_their_own(gpu, monkeypatch, short):
    if not short:
        monkeypatch.setattr(gpu, "_host", None)
    inputs = [_of_a_thread(i) for i in range(2)]
    want = [[t.clone() for f in _calls(gpu, d).values() for t in _bytes(f())] for d in inputs]
    for a, b in zip(*want):  # every output tells the threads apart
        assert a.shape != b.shape or not torch.equal(a, b)
    torch.cuda.synchronize()
    failed, start = [], threading.Barrier(2)

    def work(i):
        s = torch.cuda.Stream()
        start.wait()
        with torch.cuda.stream(s):
            all_got = [[t for f in _calls(gpu, inputs[i]).values() for t in _bytes(f())] for _ in range(10)]
            s.synchronize()
            for n, got in enumerate(all_got):
                if not all(torch.equal(a, b) for a, b in zip(got, want[i])):
                    failed.append((i, n))

    threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not failed
