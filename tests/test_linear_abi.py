"""Host-side checks of the linear layer's C ABI and binding: exports and every
refusal before anything touches a device."""
import os
import re

import pytest
import torch

from precision_linear_amd import binding

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
P = 0x10000          # a 64 KiB-aligned fake device address, never dereferenced


@pytest.fixture(scope="module")
def L():
    if not os.path.exists(binding.library_path):
        from precision_linear_amd import build
        build.build()
    return binding.lib()


def test_exports_every_declared_function(L):
    text = open(os.path.join(ROOT, "include", "fp8_linear.h")).read()
    text = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
    names = set(re.findall(r"\b(fp8_\w+)\s*\(", text))
    assert names == set(binding.LINEAR_EXPORTS)
    for n in names:
        assert hasattr(L, n), n


def test_status_text(L):
    assert binding.status_string(binding.ERR_ACTIVATION) == "unknown activation"


def call(L, A=P, fa=0, B=P, fb=0, sa=P, sb=P, bias=P, res=P, act=2, pre=P, out=P, M=64, N=64, K=64, mode=1,
         cfg=-1, splits=0, ws=None, nbytes=0):
    return L.fp8_linear(A, fa, B, fb, sa, sb, bias, res, act, pre, out, M, N, K, mode, None, cfg, splits, ws, nbytes)


@pytest.mark.parametrize("kw,code", [
    (dict(A=None), binding.ERR_NULL), (dict(B=None), binding.ERR_NULL), (dict(sa=None), binding.ERR_NULL),
    (dict(sb=None), binding.ERR_NULL), (dict(out=None), binding.ERR_NULL),
    (dict(act=-1), binding.ERR_ACTIVATION), (dict(act=5), binding.ERR_ACTIVATION),
    (dict(mode=2), binding.ERR_MODE), (dict(fa=2), binding.ERR_FORMAT), (dict(fb=-1), binding.ERR_FORMAT),
    (dict(M=-1), binding.ERR_SHAPE), (dict(N=2 ** 31), binding.ERR_SHAPE), (dict(K=8), binding.ERR_SHAPE),
    (dict(K=40), binding.ERR_SHAPE), (dict(A=P + 8), binding.ERR_ALIGN), (dict(out=P + 1), binding.ERR_ALIGN),
    (dict(res=P + 1), binding.ERR_ALIGN), (dict(pre=P + 1), binding.ERR_ALIGN),
    (dict(bias=P + 1), binding.ERR_ALIGN), (dict(cfg=99), binding.ERR_CONFIG),
    (dict(splits=65), binding.ERR_CONFIG), (dict(splits=-1, ws=P, nbytes=1 << 40), binding.ERR_CONFIG),
    (dict(K=4096, splits=2, cfg=8), binding.ERR_WORKSPACE),
])
def test_refusals(L, kw, code):
    assert call(L, **kw) == code


def test_empty_output_is_a_noop(L):
    assert call(L, M=0) == binding.OK and call(L, N=0) == binding.OK
    assert call(L, A=None, B=None, sa=None, sb=None, bias=None, res=None, pre=None, out=None, N=0) == binding.OK


def test_no_device_reported(L):
    if torch.cuda.is_available():
        pytest.skip("a GPU is present: this case would launch on fake pointers")
    assert call(L) == binding.ERR_DEVICE


def test_binding_refuses_before_the_library():
    a = torch.zeros(4, 32, dtype=torch.uint8)
    s = torch.ones(4)
    for kw in (dict(), dict(activation="tanh"), dict(mode="columnwise")):
        with pytest.raises(ValueError):
            binding.fp8_linear(a, a, s, s, **kw)


BIG = 1 << 45


def bwd(L, dy=P, x=P, wt=P, fw=0, sw=P, z=P, act=2, dx=P, dw=P, db=P, M=64, N=64, K=64, ws=P, nbytes=BIG):
    return L.fp8_linear_backward(dy, x, wt, fw, sw, z, act, dx, dw, db, M, N, K, None, ws, nbytes)


@pytest.mark.parametrize("kw,code", [
    (dict(act=-1), binding.ERR_ACTIVATION), (dict(act=5), binding.ERR_ACTIVATION),
    (dict(fw=2), binding.ERR_FORMAT), (dict(dy=None), binding.ERR_NULL), (dict(z=None), binding.ERR_NULL),
    (dict(x=None), binding.ERR_NULL), (dict(wt=None), binding.ERR_NULL), (dict(sw=None), binding.ERR_NULL),
    (dict(dx=None, dw=None, db=None), binding.ERR_NULL),
    (dict(M=-1), binding.ERR_SHAPE), (dict(M=2 ** 23 + 1), binding.ERR_SHAPE),
    (dict(N=0), binding.ERR_SHAPE), (dict(N=24), binding.ERR_SHAPE), (dict(K=8), binding.ERR_SHAPE),
    (dict(K=2 ** 23 + 16), binding.ERR_SHAPE), (dict(M=2 ** 23, N=2 ** 23), binding.ERR_SHAPE),
    (dict(dy=P + 1), binding.ERR_ALIGN), (dict(z=P + 1), binding.ERR_ALIGN), (dict(x=P + 1), binding.ERR_ALIGN),
    (dict(wt=P + 8), binding.ERR_ALIGN), (dict(sw=P + 2), binding.ERR_ALIGN), (dict(dx=P + 1), binding.ERR_ALIGN),
    (dict(dw=P + 1), binding.ERR_ALIGN), (dict(db=P + 2), binding.ERR_ALIGN), (dict(ws=P + 64), binding.ERR_ALIGN),
    (dict(ws=None), binding.ERR_WORKSPACE), (dict(nbytes=1 << 18), binding.ERR_WORKSPACE),
])
def test_backward_refusals(L, kw, code):
    assert bwd(L, **kw) == code


def test_backward_needs_only_what_its_outputs_need(L):
    if torch.cuda.is_available():
        pytest.skip("a GPU is present: these cases would launch on fake pointers")
    # what passes the checks gets as far as the missing device
    for kw in (dict(act=0, z=None), dict(dx=None, wt=None, sw=None), dict(dw=None, x=None),
               dict(dx=None, dw=None, wt=None, sw=None, x=None), dict(db=None), dict(M=0, dy=None, x=None, ws=None)):
        assert bwd(L, **kw) == binding.ERR_DEVICE, kw


def test_backward_workspace_sizes(L):
    size = L.fp8_linear_backward_workspace_size
    assert size(-1, 64, 64, 1, 1) == -1 and size(64, 24, 64, 1, 1) == -1 and size(64, 64, 0, 1, 1) == -1
    for M, N, K in ((0, 16, 16), (1, 16, 16), (500, 2048, 2048), (8191, 1008, 4160), (4096, 28672, 8192)):
        both, dx, dw, none = (size(M, N, K, a, b) for a, b in ((1, 1), (1, 0), (0, 1), (0, 0)))
        mp = (M + 15) // 16 * 16
        assert both >= (256 << 10) + M * N + N * mp + K * mp     # counters, then the codes
        assert none <= dx <= both and none <= dw <= both
        for kw, n in ((dict(), both), (dict(dw=None), dx), (dict(dx=None), dw), (dict(dx=None, dw=None), none)):
            if M:
                assert bwd(L, M=M, N=N, K=K, nbytes=n - 1, **kw) == binding.ERR_WORKSPACE


def test_backward_binding_refuses_before_the_library():
    dy = torch.zeros(4, 32, dtype=torch.bfloat16)
    w = torch.zeros(16, 32, dtype=torch.uint8)
    s = torch.ones(16)
    for kw in (dict(), dict(activation="tanh"), dict(dx=False, dw=False, dbias=False), dict(dx=3), dict(dbias=s)):
        with pytest.raises(ValueError):
            binding.fp8_linear_backward(dy, dy, w, s, **kw)
