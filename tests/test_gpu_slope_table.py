"""The gelus' slopes from a table (the linear layer's gradient, dz of at least 512
tiles of 128 x 128).

Tolerances: the slope's own (the fit of the normal distribution function 1.5e-7, z^2
rounded in an exponent, a few fp32 roundings: 4e-7 max(1, |z|)) and two more roundings
of values up to 1.13, of the table's value and of its sum with 1/2 (2^-24 each).
"""
import pytest
import torch

from precision_linear_amd import binding
from test_gpu_linear_backward import BF16, DEV, act64, check, make, slope64, within

pytestmark = pytest.mark.gpu
GELUS = ("gelu", "gelu_tanh")


def tabled(M, N):
    return -(-M // 128) * -(-N // 128) >= 512


def slopes(z, act):
    """act'(z) of a row of values, by way of dbias: one row of ones among zeros."""
    M = 300
    assert tabled(M, z.numel())
    dy = torch.zeros(M, z.numel(), dtype=BF16, device=DEV)
    dy[137] = 1
    return binding.fp8_linear_backward(dy, None, None, None, z.to(DEV).expand(M, -1).contiguous(), activation=act,
                                       dx=False, dw=False)[2]


@pytest.mark.parametrize("act", GELUS)
def test_slope_of_every_finite_bf16_value(act):
    v = torch.arange(65536, dtype=torch.int32).to(torch.int16).view(BF16)
    v = v[torch.isfinite(v.float())]
    n = v.numel() // 16 * 16
    for z in (v[:n], v[-n:]):
        z64 = z.double()
        want = torch.where(z64.abs() > 100, (z64 > 0).double(), slope64(z64, act))
        tol = 4e-7 * z64.abs().clamp(1, 16) + 2.0 ** -23
        got = slopes(z, act)
        within("slope", got, want, tol)
        near = z64.abs() < 20
        h = 1e-5
        diff = (act64(z64 + h, act) - act64(z64 - h, act)) / (2 * h)
        within("differences", got[near.to(DEV)], diff[near], tol[near] + 1e-8)


@pytest.mark.parametrize("act", GELUS)
def test_values_that_are_not_finite(act):
    z = torch.randn(128 * 256, generator=torch.Generator().manual_seed(0)).to(BF16)
    z[5], z[100], z[1000], z[4001] = float("inf"), float("-inf"), float("nan"), -float("nan")
    got = slopes(z, act).cpu()
    assert got[5] == 1 and got[100] == 0 and got[[1000, 4001]].isnan().all()
    assert got.isnan().sum() == 2


@pytest.mark.parametrize("act", GELUS)
@pytest.mark.parametrize("M,N,K", [(1100, 7296, 48), (8200, 1008, 80), (130, 33008, 32)])
def test_gradient_against_64_bits(M, N, K, act):
    assert tabled(M, N)
    check(make(M, N, K, M + N), act)
