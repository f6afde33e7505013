"""Host-side checks of the weight quantisation's C ABI and binding: exports, workspace
sizes and every refusal before anything touches a device."""
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
    text = open(os.path.join(ROOT, "include", "fp8_quantize_weight.h")).read()
    text = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
    names = set(re.findall(r"\b(fp8_\w+)\s*\(", text))
    assert names == set(binding.QUANTIZE_WEIGHT_EXPORTS)
    for n in names:
        assert hasattr(L, n), n


def call(L, w=P, dt=0, fmt=0, q=P, s=P, qt=P, st=P, N=64, K=64, ws=P, nbytes=1 << 45):
    return L.fp8_quantize_weight(w, dt, fmt, q, s, qt, st, N, K, None, ws, nbytes)


@pytest.mark.parametrize("kw,code", [
    (dict(dt=2), binding.ERR_FORMAT), (dict(dt=-1), binding.ERR_FORMAT), (dict(fmt=2), binding.ERR_FORMAT),
    (dict(N=-1), binding.ERR_SHAPE), (dict(N=2 ** 31 - 15), binding.ERR_SHAPE), (dict(K=0), binding.ERR_SHAPE),
    (dict(K=24), binding.ERR_SHAPE), (dict(K=2 ** 23 + 16), binding.ERR_SHAPE),
    (dict(N=2 ** 30, K=2 ** 23), binding.ERR_SHAPE),
    (dict(w=None), binding.ERR_NULL), (dict(q=None), binding.ERR_NULL), (dict(s=None), binding.ERR_NULL),
    (dict(qt=None), binding.ERR_NULL), (dict(st=None), binding.ERR_NULL), (dict(N=0, st=None), binding.ERR_NULL),
    (dict(w=P + 1), binding.ERR_ALIGN), (dict(w=P + 2, dt=1), binding.ERR_ALIGN), (dict(q=P + 8), binding.ERR_ALIGN),
    (dict(qt=P + 8), binding.ERR_ALIGN), (dict(s=P + 2), binding.ERR_ALIGN), (dict(st=P + 1), binding.ERR_ALIGN),
    (dict(ws=P + 64), binding.ERR_ALIGN), (dict(ws=None), binding.ERR_WORKSPACE), (dict(nbytes=64), binding.ERR_WORKSPACE),
])
def test_refusals(L, kw, code):
    assert call(L, **kw) == code


def test_no_device_reported(L):
    if torch.cuda.is_available():
        pytest.skip("a GPU is present: this case would launch on fake pointers")
    assert call(L) in (binding.ERR_DEVICE, binding.ERR_LAUNCH)
    assert call(L, N=0, w=None, q=None, s=None, qt=None, ws=None) in (binding.ERR_DEVICE, binding.ERR_LAUNCH)


def test_workspace_sizes(L):
    size = L.fp8_quantize_weight_workspace_size
    assert size(-1, 64) == -1 and size(64, 24) == -1 and size(0, 64) == 0
    for N, K in ((1, 16), (1000, 4160), (28672, 8192), (10 ** 6, 64), (1, 2 ** 23)):
        n = size(N, K)
        assert 4 * (N + K) <= n <= 4 * ((K + 127) // 128 * N + (N // 64 + 1) * K)
        assert call(L, N=N, K=K, nbytes=n - 1) == binding.ERR_WORKSPACE


def test_the_largest_sizes_are_those_that_can_be_launched(L):
    """A launch has fewer than 2^32 threads: 1024 for each 64 rows, 256 for each 128 x 128."""
    size = L.fp8_quantize_weight_workspace_size
    for N, K in ((2 ** 27, 16), (2 ** 27, 1920), (2 ** 24, 16256), (1, 2 ** 23)):
        assert size(N, K) > 0
        assert call(L, N=N, K=K, nbytes=64) == binding.ERR_WORKSPACE
    for N, K in ((2 ** 27 + 1, 16), (2 ** 27, 2048), (2 ** 24, 16384), (2 ** 28, 16)):
        assert size(N, K) == -1 and call(L, N=N, K=K) == binding.ERR_SHAPE


def test_binding_refuses_before_the_library():
    w = torch.zeros(4, 32)
    for args, kw in (((w,), dict()), ((w, "int8"), dict()), ((w.half(),), dict()), ((w[0],), dict())):
        with pytest.raises(ValueError):
            binding.fp8_quantize_weight(*args, **kw)
