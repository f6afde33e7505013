"""Two host threads that call the gradients on one stream (the default one, which
all threads share unless told otherwise): the bits of the same calls made one
after the other."""
import threading

import pytest
import torch

from precision_linear_amd import binding
from test_gpu_layer_norm import make as make_norm
from test_gpu_linear_backward import make as make_linear

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
REPEATS = 40


def norm_call(rows, cols, seed):
    x, w, _ = (t.to(DEV) for t in make_norm(rows, cols, torch.bfloat16, seed))
    dy = make_norm(rows, cols, torch.bfloat16, seed + 1)[0].to(DEV)
    st = binding.fp8_layer_norm(x, stats=True)
    return lambda **kw: binding.fp8_layer_norm_backward(dy, x, st.mean, st.rstd, w, **kw)


def linear_call(M, N, K, seed, act):
    args = [t.to(DEV) for t in make_linear(M, N, K, seed)]
    return lambda **kw: binding.fp8_linear_backward(*args, activation=act, **kw)


@pytest.mark.parametrize("path", ["short", "whole"])
def test_gradients_from_two_threads(monkeypatch, path):
    binding.lib()
    if path == "whole":
        monkeypatch.setattr(binding, "_calls", None)     # the calls through ctypes
    calls = [[norm_call(2000, 1000, 1), linear_call(500, 1024, 768, 2, "gelu"), linear_call(130, 8336, 32, 3, "silu")],
             [norm_call(3000, 520, 4), linear_call(300, 2048, 512, 5, "relu"), linear_call(150, 8448, 48, 6, "gelu")]]
    want = [[f() for f in part] for part in calls]
    torch.cuda.synchronize()
    got, failed = [[], []], []
    ready = threading.Barrier(2)

    def run(i):
        try:
            ready.wait()
            for _ in range(REPEATS):
                got[i].append([f() for f in calls[i]])
        except Exception as e:      # (shown below; a thread's own is only printed)
            failed.append(e)

    threads = [threading.Thread(target=run, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not failed, failed
    for i in range(2):
        assert len(got[i]) == REPEATS
        for rep, outs in enumerate(got[i]):
            for k, (have, right) in enumerate(zip(outs, want[i])):
                assert all(torch.equal(a, b) for a, b in zip(have, right)), (i, rep, k)
