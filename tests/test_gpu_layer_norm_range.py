"""Rows of the layer norm whose sums leave the fp32 range, of finite values: they
show it as rows with an infinity do, and leave the others."""
import pytest
import torch

from precision_linear_amd import binding
from test_gpu_layer_norm import BF16, DEV, FP32, make

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("cols", [64, 1008, 1024, 4096, 8192, 16384, 20000])
@pytest.mark.parametrize("value,spread", [(1e20, True), (3e38, True), (3e38, False)])
def test_a_row_beyond_the_range_shows_it(cols, dtype, value, spread):
    x, w, b = make(5, cols, dtype, 12)
    args = (w.to(DEV), b.to(DEV))
    clean = binding.fp8_layer_norm(x.to(DEV), *args, fmt="e4m3fn", stats=True)
    x[2] = value
    if spread:                      # the sum stays small, the squares do not
        x[2, 1::2] = -value
    r = binding.fp8_layer_norm(x.to(DEV), *args, fmt="e4m3fn", stats=True)
    assert r.y[2].isnan().all() and r.scale[2].isnan() and r.rstd[2].isnan()
    assert (r.q[2] & 0x7F == 0x7F).all()
    keep = [0, 1, 3, 4]
    for got, want in zip(r, clean):
        assert torch.equal(got[keep], want[keep])
    dx, _, _ = binding.fp8_layer_norm_backward(x.to(DEV), x.to(DEV), r.mean, r.rstd, args[0], residual_grad=x.to(DEV))
    assert dx[2].isnan().all() and dx[keep].isfinite().all()


@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("cols", [64, 8192, 20000])
def test_large_rows_within_the_range_are_ordinary(cols, dtype):
    # squares of 2^57 in size over up to 2^15 columns: sums under 2^130, so with 2^55 under 2^126
    x, w, b = make(4, cols, dtype, 13)
    x = (x.float() * 2.0 ** 53).to(dtype)
    assert (x.double() ** 2).sum(1).max() < 2.0 ** 127
    got = binding.fp8_layer_norm(x.to(DEV), w.to(DEV), b.to(DEV), stats=True)
    d = x.double() - x.double().mean(1, keepdim=True)
    rstd = d.square().mean(1).rsqrt()
    # the sums' relative error: test_gpu_layer_norm's 2 (32 + cols / 1024) roundings of values up to 8 times the spread
    tol = 16 * (32 + cols / 1024) * 2.0 ** -24
    assert ((got.rstd.double().cpu() / rstd - 1).abs() <= tol).all()
    want = d * rstd[:, None] * w.double() + b.double()
    half = torch.finfo(dtype).eps / 2
    assert ((got.y.double().cpu() - want).abs() <= half * want.abs() + tol * (want.abs() + 8 * w.abs() + 1)).all()
