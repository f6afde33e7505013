"""The linear layer's gradient takes its scratch memory for the call alone, and
finds it with any contents."""
import pytest
import torch

from precision_linear_amd import binding
from test_gpu_linear_backward import DEV, make

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("path", ["short", "whole"])
def test_memory_is_torchs_again_after_the_call(monkeypatch, path):
    binding.lib()
    if path == "whole":
        monkeypatch.setattr(binding, "_calls", None)
    args = [t.to(DEV) for t in make(4000, 4096, 1024, 1)]
    need = int(binding.lib().fp8_linear_backward_workspace_size(4000, 4096, 1024, 1, 1))
    assert need > 32 << 20
    stream = torch.cuda.Stream()        # (none of its workspaces exist)
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        before = torch.cuda.memory_allocated()
        outs = binding.fp8_linear_backward(*args, activation="relu")
        torch.cuda.synchronize()
        kept = torch.cuda.memory_allocated() - before
    # the outputs (each rounded up to 512 bytes, or to 2 MiB where it is large) and, at most, a split K's workspace
    assert kept <= sum(t.numel() * t.element_size() for t in outs) + (8 << 20), kept
    assert kept < need


# one launch for both products (split over K or not), two, the products alone, no product
@pytest.mark.parametrize("M,N,K", [(500, 2048, 2048), (64, 4096, 1024), (17, 64, 4096), (130, 8336, 32), (1, 16, 16),
                                   (16, 28672, 512), (5000, 1024, 128)])
def test_a_workspace_of_any_contents(M, N, K):
    dy, x, wt, sw, z = (t.to(DEV) for t in make(M, N, K, 3))
    f = binding.fp8_linear_backward
    need = int(binding.lib().fp8_linear_backward_workspace_size(M, N, K, 1, 1))
    for w in (wt, wt.float().to(torch.float8_e5m2)):
        for kw in (dict(), dict(dx=False), dict(dw=False), dict(dx=False, dw=False)):
            want = f(dy, x, w, sw, z, activation="silu", workspace=torch.zeros(need, dtype=torch.uint8, device=DEV), **kw)
            for byte in (0xFF, 1, 0x55):
                print(f"[linear_backward] {M} x {N} x {K} {w.dtype} {kw} workspace of {byte}", flush=True)
                ws = torch.full((need,), byte, dtype=torch.uint8, device=DEV)
                got = f(dy, x, w, sw, z, activation="silu", workspace=ws, **kw)
                assert all(a is b is None or torch.equal(a, b) for a, b in zip(got, want)), (kw, byte)
