"""Rows of zeros without eps: 0 times an infinite rstd, so y, its scale and its
codes are NaN."""
import pytest
import torch

from precision_linear_amd import binding
from test_gpu_layer_norm import BF16, DEV, FP32, make

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("cols", [64, 1008, 8192, 20000])
@pytest.mark.parametrize("fmt,largest", [("e4m3fn", 0x7E), ("e5m2", 0x7C)])
def test_rows_of_zeros_without_eps(cols, dtype, fmt, largest):
    x, w, b = make(4, cols, dtype, 3)
    x[1] = 0
    r = binding.fp8_layer_norm(x.to(DEV), w.to(DEV), b.to(DEV), 0.0, fmt=fmt, stats=True)
    assert r.rstd[1] == float("inf") and r.mean[1] == 0
    assert r.y[1].isnan().all() and r.scale[1].isnan() and ((r.q[1] & 0x7F) > largest).all()
    keep = [0, 2, 3]
    assert r.y[keep].isfinite().all() and r.scale[keep].isfinite().all()
