"""The float8 codes of dz in the linear layer's gradient, one by one: W (x) is the
unit matrix, so that each output is a code times its scale, without the products'
sums between.

A code may be the neighbouring one where the slope's error (test_gpu_linear_backward's,
absolute) takes the quotient over a tie, and the scale moves with the largest value
of its row or column by 2e-5 at most; the output's half step comes on top.
"""
import pytest
import torch

from precision_linear_amd import binding
from test_gpu_linear_backward import ACTS, BF16, DEV, E5M2, HALF, make, quantised, slope64, within

pytestmark = pytest.mark.gpu


# 64-row tiles; 128-row ones with the slope table; too many column blocks to join
@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("M,N", [(500, 1024), (1100, 7552), (512, 16512)])
def test_codes_of_dz(M, N, act):
    K = -(-M // 16) * 16
    dy, _, _, _, z = make(M, N, 16, M + N)
    x = torch.eye(M, K, device=DEV).to(BF16)
    wt = torch.eye(K, N, device=DEV).to(torch.float8_e4m3fn)
    print(f"[linear_backward] codes {M} x {N} {act}", flush=True)
    dx, dw, _ = binding.fp8_linear_backward(dy.to(DEV), x, wt, torch.ones(K, device=DEV), z.to(DEV), activation=act)
    dz = dy.double() * slope64(z.double(), act)
    err = None
    if act not in ("none", "relu"):
        err = dy.double().abs() * (4e-7 * z.double().abs().clamp(min=1) + 2.0 ** -23) + 2.0 ** -23 * dz.abs()
    for name, got, axis in (("dx", dx, 1), ("dw", dw.t(), 0)):
        want, dev = quantised(dz, axis, E5M2, err)
        tol = dev + 2e-5 * want.abs()
        if axis == 1:
            want, tol = want[:, :K], tol[:, :K]
        got = got[:, :want.shape[1]] if axis == 1 else got[:M]
        within(name, got, want, tol + HALF * (want.abs() + tol))
