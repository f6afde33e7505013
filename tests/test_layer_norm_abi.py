"""Host-side checks of the layer norm's C ABI and binding: exports, status
strings, workspace sizes, and every refusal before anything touches a device."""
import os
import re

import pytest
import torch

from precision_linear_amd import binding

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
P = 0x10000          # a 64 KiB-aligned fake device address, never dereferenced
BIG = 1 << 40


@pytest.fixture(scope="module")
def L():
    if not os.path.exists(binding.library_path):
        from precision_linear_amd import build
        build.build()
    return binding.lib()


def test_exports_every_declared_function(L):
    text = open(os.path.join(ROOT, "include", "fp8_layer_norm.h")).read()
    text = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
    names = set(re.findall(r"\b(fp8_\w+)\s*\(", text))
    assert names == set(binding.LAYER_NORM_EXPORTS)
    for n in names:
        assert hasattr(L, n), n


def test_status_strings(L):
    texts = [L.fp8_layer_norm_status_string(s) for s in range(9)]
    assert len(set(texts)) == 9 and b"unknown status" not in texts
    assert L.fp8_layer_norm_status_string(99) == b"unknown status"


def fwd(L, x=P, dtype=0, w=P, b=P, pdt=1, eps=1e-5, y=P, q=P, fmt=0, scale=P, mean=P, rstd=P, rows=4, cols=64):
    return L.fp8_layer_norm(x, dtype, w, b, pdt, eps, y, q, fmt, scale, mean, rstd, rows, cols, None)


def bwd(L, dy=P, x=P, dtype=0, mean=P, rstd=P, w=P, pdt=1, res=P, dx=P, dw=P, db=P, rows=4, cols=64, ws=P,
        nbytes=BIG):
    return L.fp8_layer_norm_backward(dy, x, dtype, mean, rstd, w, pdt, res, dx, dw, db, rows, cols, ws, nbytes, None)


@pytest.mark.parametrize("kw,code", [
    (dict(x=None), binding.LN_ERR_NULL), (dict(y=None, q=None, scale=None), binding.LN_ERR_NULL),
    (dict(scale=None), binding.LN_ERR_NULL), (dict(q=None), binding.LN_ERR_NULL),
    (dict(mean=None), binding.LN_ERR_NULL), (dict(rstd=None), binding.LN_ERR_NULL),
    (dict(rows=-1), binding.LN_ERR_SHAPE), (dict(rows=2 ** 31), binding.LN_ERR_SHAPE),
    (dict(cols=0), binding.LN_ERR_SHAPE), (dict(cols=2 ** 24 + 16), binding.LN_ERR_SHAPE),
    (dict(cols=24), binding.LN_ERR_SHAPE), (dict(dtype=2), binding.LN_ERR_DTYPE),
    (dict(pdt=-1), binding.LN_ERR_DTYPE), (dict(fmt=2), binding.LN_ERR_DTYPE),
    (dict(eps=-1.0), binding.LN_ERR_VALUE), (dict(eps=float("nan")), binding.LN_ERR_VALUE),
    (dict(eps=float("inf")), binding.LN_ERR_VALUE),
    (dict(x=P + 1), binding.LN_ERR_ALIGN), (dict(y=P + 1), binding.LN_ERR_ALIGN),
    (dict(x=P + 2, dtype=1), binding.LN_ERR_ALIGN), (dict(w=P + 2), binding.LN_ERR_ALIGN),
    (dict(b=P + 2), binding.LN_ERR_ALIGN), (dict(b=P + 1, pdt=0), binding.LN_ERR_ALIGN),
    (dict(q=P + 8), binding.LN_ERR_ALIGN), (dict(scale=P + 2), binding.LN_ERR_ALIGN),
    (dict(mean=P + 2), binding.LN_ERR_ALIGN), (dict(rstd=P + 2), binding.LN_ERR_ALIGN),
])
def test_forward_refusals(L, kw, code):
    assert fwd(L, **kw) == code


@pytest.mark.parametrize("kw,code", [
    (dict(dy=None), binding.LN_ERR_NULL), (dict(x=None), binding.LN_ERR_NULL),
    (dict(mean=None), binding.LN_ERR_NULL), (dict(rstd=None), binding.LN_ERR_NULL),
    (dict(dx=None), binding.LN_ERR_NULL), (dict(dw=None), binding.LN_ERR_NULL),
    (dict(db=None), binding.LN_ERR_NULL), (dict(rows=0, dw=None), binding.LN_ERR_NULL),
    (dict(rows=-1), binding.LN_ERR_SHAPE), (dict(cols=0), binding.LN_ERR_SHAPE),
    (dict(dtype=3), binding.LN_ERR_DTYPE), (dict(pdt=2), binding.LN_ERR_DTYPE),
    (dict(dy=P + 1), binding.LN_ERR_ALIGN), (dict(x=P + 1), binding.LN_ERR_ALIGN),
    (dict(res=P + 1), binding.LN_ERR_ALIGN), (dict(dx=P + 1), binding.LN_ERR_ALIGN),
    (dict(w=P + 2), binding.LN_ERR_ALIGN), (dict(mean=P + 1), binding.LN_ERR_ALIGN),
    (dict(dw=P + 2), binding.LN_ERR_ALIGN), (dict(ws=P + 128), binding.LN_ERR_ALIGN),
    (dict(ws=None), binding.LN_ERR_WORKSPACE), (dict(nbytes=16), binding.LN_ERR_WORKSPACE),
])
def test_backward_refusals(L, kw, code):
    assert bwd(L, **kw) == code


def test_empty_forward_is_a_noop(L):
    assert fwd(L, rows=0) == binding.LN_OK
    assert fwd(L, rows=0, x=None, y=None, q=None, scale=None, mean=None, rstd=None) == binding.LN_OK


def test_no_device_reported(L):
    if torch.cuda.is_available():
        pytest.skip("a GPU is present: this case would launch on fake pointers")
    assert fwd(L) == binding.LN_ERR_DEVICE
    assert bwd(L) == binding.LN_ERR_DEVICE


def test_workspace_sizes(L):
    size = L.fp8_layer_norm_backward_workspace_size
    assert size(0, 64) == 0 and size(-1, 64) == 0 and size(4, 0) == 0
    for rows in (1, 3, 255, 256, 257, 4096, 2 ** 31 - 1):
        for cols in (1, 63, 64, 65, 1024, 1025, 8192, 16391, 16392, 2 ** 24):
            n = size(rows, cols)
            # two sums of whole 64-column blocks for at least one and at most 256 workgroups
            pitch = (cols + 63) // 64 * 64
            assert n % (8 * pitch) == 0 and 1 <= n // (8 * pitch) <= min(rows, 256)
            assert bwd(L, rows=rows, cols=cols, nbytes=n - 1) == binding.LN_ERR_WORKSPACE


def test_binding_refuses_before_the_library():
    x = torch.zeros(4, 64, dtype=torch.bfloat16)
    s = torch.zeros(4)
    for call in (lambda: binding.fp8_layer_norm(x),                              # not on the GPU
                 lambda: binding.fp8_layer_norm(x.half()),
                 lambda: binding.fp8_layer_norm(x[0]),
                 lambda: binding.fp8_layer_norm(x.t()),
                 lambda: binding.fp8_layer_norm_backward(x, x, s, s)):
        with pytest.raises(ValueError):
            call()
