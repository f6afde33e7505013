"""The gelus' slopes where z is far below 0: a relative bound, with and without the
table (dz of at least 512 tiles of 128 x 128 takes it).

With t = -z >= 2 the slope is the difference of Q(t) and t times the density (gelu),
or of p and p t (1 - p) u' (gelu_tanh), whose sum is at most 1.6 times as large.
Each term is off by the fit of Q (1.5e-7) and at most 12 roundings of 2^-24 (a
hardware exp2 or reciprocal counts as 2), and, common to both, by the exponent's
own roundings times ln 2: of -z^2 log2(e) / 2 two (z^2 is exact), of 2 u log2(e)
at most 4 (two constants, the sum, the product).
"""
import pytest
import torch

from precision_linear_amd import binding
from test_gpu_linear_backward import BF16, DEV, E4M3, E5M2, HALF, quantised, slope64, within

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
GELUS = ("gelu", "gelu_tanh")


def relative(z, act):
    z = z.double()
    if act == "gelu":
        exponent = z * z / 2
        roundings = 2
    else:
        exponent = (2 * (2 / torch.pi) ** 0.5 * (z + 0.044715 * z ** 3)).abs()
        roundings = 4
    return 1.6 * (1.5e-7 + 12 * U) + roundings * U * exponent


def tail(act):
    """The bf16 values from -2 down to where the slope is about 2^-110."""
    v = torch.arange(65536, dtype=torch.int32).to(torch.int16).view(BF16)
    v = v[(v.float() <= -2) & (v.float() >= -12)]
    return v[slope64(v.double(), act).abs() > 2.0 ** -110]


@pytest.mark.parametrize("act", GELUS)
@pytest.mark.parametrize("M,N", [(1, 1024), (300, 22016)])
def test_slope_far_below_zero(M, N, act):
    v = tail(act)
    assert v.numel() > 200
    z = v.repeat(-(-N // v.numel()))[:N]
    dy = torch.zeros(M, N, dtype=BF16, device=DEV)
    dy[M // 2] = 1
    got = binding.fp8_linear_backward(dy, None, None, None, z.to(DEV).expand(M, -1).contiguous(), activation=act,
                                      dx=False, dw=False)[2]
    want = slope64(z.double(), act)
    within("slope", got, want, relative(z, act) * want.abs())


@pytest.mark.parametrize("act", GELUS)
@pytest.mark.parametrize("M,N,K", [(300, 2048, 48), (300, 22016, 48)])
def test_gradient_of_units_that_are_far_below_zero(M, N, K, act):
    g = torch.Generator().manual_seed(M + N)
    dy = torch.randn(M, N, generator=g).to(BF16)
    z = (-6 + 0.5 * torch.randn(M, N, generator=g)).clamp(-8, -4).to(BF16)
    x = torch.randn(M, K, generator=g).to(BF16)
    wt = (2 * torch.randn(K, N, generator=g)).to(torch.float8_e4m3fn)
    sw = torch.rand(K, generator=g) + 0.5
    got = binding.fp8_linear_backward(*(t.to(DEV) for t in (dy, x, wt, sw, z)), activation=act)
    dz = dy.double() * slope64(z.double(), act)
    err = (relative(z, act) + U) * dz.abs()
    w = wt.double() * sw.double()[:, None]
    rows, rdev = quantised(dz, 1, E5M2, err)
    cols, cdev = quantised(dz, 0, E5M2, err)
    xq, _ = quantised(x.double(), 0, E4M3)
    mm = 1e-3 + 2e-5                          # the products' parity bound, the scales
    dx, dw, db = rows @ w.t(), cols.t() @ xq, dz.sum(0)
    dxe = rdev @ w.abs().t() + mm * (rows.abs() @ w.abs().t())
    dwe = cdev.t() @ xq.abs() + mm * (cols.abs().t() @ xq.abs())
    within("dx", got[0], dx, dxe + HALF * (dx.abs() + dxe))
    within("dw", got[1], dw, dwe + HALF * (dw.abs() + dwe))
    within("dbias", got[2], db, err.sum(0) + (M / 256 + 32) * U * dz.abs().sum(0))
