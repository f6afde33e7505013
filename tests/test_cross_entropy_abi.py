"""Host-side checks of the cross entropy's C ABI and binding: exports, workspace
sizes and every refusal before anything touches a device."""
import os
import re

import pytest
import torch

from precision_linear_amd import binding

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
P = 0x10000          # a 64 KiB-aligned fake device address, never dereferenced
BIG = 1 << 50


@pytest.fixture(scope="module")
def L():
    if not os.path.exists(binding.library_path):
        from precision_linear_amd import build
        build.build()
    return binding.lib()


def test_exports_every_declared_function(L):
    text = open(os.path.join(ROOT, "include", "fp8_cross_entropy.h")).read()
    text = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
    names = set(re.findall(r"\b(fp8_\w+)\s*\(", text))
    assert names == set(binding.CROSS_ENTROPY_EXPORTS)
    for n in names:
        assert hasattr(L, n), n


def fwd(L, A=P, fa=0, B=P, fb=0, sa=P, sb=P, t=P, ignore=-100, loss=P, lse=P, M=64, V=1000, K=64, mode=1, ws=P,
        nbytes=BIG):
    return L.fp8_linear_cross_entropy(A, fa, B, fb, sa, sb, t, ignore, loss, lse, M, V, K, mode, None, ws, nbytes)


def bwd(L, dl=P, stride=1, A=P, fa=0, B=P, fb=0, sa=P, sb=P, t=P, ignore=-100, loss=P, lse=P, x=P, wt=P, fw=0, sw=P,
        dx=P, dw=P, M=64, V=1000, K=64, mode=1, ws=P, nbytes=BIG):
    return L.fp8_linear_cross_entropy_backward(dl, stride, A, fa, B, fb, sa, sb, t, ignore, loss, lse, x, wt, fw, sw,
                                               dx, dw, M, V, K, mode, None, ws, nbytes)


SHARED = [
    (dict(A=None), binding.ERR_NULL), (dict(B=None), binding.ERR_NULL), (dict(sa=None), binding.ERR_NULL),
    (dict(sb=None), binding.ERR_NULL), (dict(t=None), binding.ERR_NULL), (dict(loss=None), binding.ERR_NULL),
    (dict(lse=None), binding.ERR_NULL), (dict(fa=2), binding.ERR_FORMAT), (dict(fb=-1), binding.ERR_FORMAT),
    (dict(mode=2), binding.ERR_MODE), (dict(M=-1), binding.ERR_SHAPE), (dict(M=2 ** 23 + 1), binding.ERR_SHAPE),
    (dict(V=0), binding.ERR_SHAPE), (dict(V=2 ** 23 + 1), binding.ERR_SHAPE), (dict(K=0), binding.ERR_SHAPE),
    (dict(K=40), binding.ERR_SHAPE), (dict(K=2 ** 23 + 16), binding.ERR_SHAPE),
    (dict(A=P + 8), binding.ERR_ALIGN), (dict(B=P + 8), binding.ERR_ALIGN), (dict(sa=P + 2), binding.ERR_ALIGN),
    (dict(sb=P + 2), binding.ERR_ALIGN), (dict(t=P + 4), binding.ERR_ALIGN), (dict(loss=P + 2), binding.ERR_ALIGN),
    (dict(lse=P + 2), binding.ERR_ALIGN), (dict(ws=P + 64), binding.ERR_ALIGN),
    (dict(ws=None), binding.ERR_WORKSPACE), (dict(nbytes=1 << 10), binding.ERR_WORKSPACE)]


@pytest.mark.parametrize("kw,code", SHARED)
def test_refusals(L, kw, code):
    assert fwd(L, **kw) == code


@pytest.mark.parametrize("kw,code", SHARED + [
    (dict(dl=None), binding.ERR_NULL), (dict(stride=2), binding.ERR_SHAPE), (dict(x=None), binding.ERR_NULL),
    (dict(wt=None), binding.ERR_NULL), (dict(sw=None), binding.ERR_NULL), (dict(fw=2), binding.ERR_FORMAT),
    (dict(dx=None, dw=None), binding.ERR_NULL), (dict(dl=P + 2), binding.ERR_ALIGN), (dict(x=P + 1), binding.ERR_ALIGN),
    (dict(wt=P + 8), binding.ERR_ALIGN), (dict(sw=P + 2), binding.ERR_ALIGN), (dict(dx=P + 1), binding.ERR_ALIGN),
    (dict(dw=P + 1), binding.ERR_ALIGN)])
def test_backward_refusals(L, kw, code):
    assert bwd(L, **kw) == code


def test_what_passes_the_checks_gets_as_far_as_the_missing_device(L):
    if torch.cuda.is_available():
        pytest.skip("a GPU is present: these cases would launch on fake pointers")
    assert fwd(L) == binding.ERR_DEVICE or fwd(L) == binding.ERR_LAUNCH
    for kw in (dict(), dict(dx=None, wt=None, sw=None), dict(dw=None, x=None), dict(stride=0),
               dict(M=0, A=None, B=None, t=None, dl=None, ws=None)):
        assert bwd(L, **kw) in (binding.ERR_DEVICE, binding.ERR_LAUNCH), kw
    assert fwd(L, M=0, A=None, B=None, sa=None, sb=None, t=None, loss=None, lse=None, ws=None) == binding.OK


def test_workspace_sizes(L):
    size, back = L.fp8_linear_cross_entropy_workspace_size, L.fp8_linear_cross_entropy_backward_workspace_size
    for bad in ((-1, 10, 64), (10, 0, 64), (10, 10, 8), (2 ** 23 + 1, 10, 64)):
        assert size(*bad) == -1 and back(*bad, 1, 1) == -1
    for M, V, K in ((0, 1, 16), (1, 1, 16), (1000, 50255, 2048), (8192, 131072, 4096), (16384, 262144, 64),
                    (2 ** 23, 300, 16), (3, 2 ** 23, 16)):
        n = size(M, V, K)
        assert n >= 8 * M * (V // 128)
        if M:
            assert fwd(L, M=M, V=V, K=K, nbytes=n - 1) == binding.ERR_WORKSPACE
        both, dx, dw = (back(M, V, K, a, b) for a, b in ((1, 1), (1, 0), (0, 1)))
        assert 0 <= dx <= both and 0 <= dw <= both
        if M:
            for kw, n in ((dict(), both), (dict(dw=None), dx), (dict(dx=None), dw)):
                assert bwd(L, M=M, V=V, K=K, nbytes=n - 1, **kw) == binding.ERR_WORKSPACE
            # codes of a piece, K columns of x, dx's sums: not M V values
            assert both < (1 << 30) + 2 * K * (M + 128) + 8 * (M + 256) * (K + 256) + 64 * M + 2048 * M


def test_binding_refuses_before_the_library():
    a, b = torch.zeros(4, 32, dtype=torch.uint8), torch.zeros(100, 32, dtype=torch.uint8)
    sa, sb, t = torch.ones(4), torch.ones(100), torch.zeros(4, dtype=torch.int64)
    for args, kw in (((a, b, sa, sb, t), dict()), ((a, b, sa, sb, t), dict(mode="columnwise")),
                     ((a, b[:, :16], sa, sb, t), dict()), ((a.float(), b, sa, sb, t), dict()),
                     ((a, b, sa, sb, t), dict(a_format="e3m4")), ((a, b[:0], sa, sb, t), dict())):
        with pytest.raises(ValueError):
            binding.fp8_linear_cross_entropy(*args, **kw)
    x, wt, f = torch.zeros(4, 32, dtype=torch.bfloat16), torch.zeros(32, 112, dtype=torch.uint8), torch.ones(4)
    for args, kw in (((f, a, b, sa, sb, t, f, f, x, wt, f), dict()), ((f, a, b, sa, sb, t, f, f, None, wt, f), dict()),
                     ((f, a, b, sa, sb, t, f, f, x, None, f), dict()), ((f, a, b, sa, sb, t, f, f, x, wt, None), dict()),
                     ((f, a, b, sa, sb, t, f, f, x, wt, f), dict(dx=False, dw=False)),
                     ((f, a, b, sa, sb, t, f, f, x, wt, f), dict(dx=3))):
        with pytest.raises(ValueError):
            binding.fp8_linear_cross_entropy_backward(*args, **kw)
