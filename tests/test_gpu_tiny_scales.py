"""The linear layer's gradient where scales are tiny (from 2^-126 on): the codes
are those of the correctly rounded quotients, as at ordinary scales.

Every mantissa of a bf16 maximum meets every mantissa of a value over the format's
exponents, so that the quotients which lie on a tie between two codes are among
them.  One factor of each product picks single values of the other: with a row
(column) of one nonzero value, whose code is the largest and whose scale times that
is the value, an output is a code times its scale times 2^100, within 2^-7 (two
scales' roundings and the output's half step); neighbouring codes are 2^-4 apart
or more.
"""
import pytest
import torch

from precision_linear_amd import binding
from test_gpu_linear_backward import BF16, DEV, E4M3, E5M2, quantised

pytestmark = pytest.mark.gpu
UP = 2.0 ** 100
MANTISSAS = 1 + torch.arange(128, dtype=torch.float64) / 128


def pairs(exponents, span, copies=1):
    """One row for each maximum: its mantissa times 2^exponent, then values of `span` binades below."""
    top = (2.0 ** torch.tensor(exponents, dtype=torch.float64)[:, None] * MANTISSAS).reshape(-1, 1)
    below = (MANTISSAS * 2.0 ** -torch.arange(span, dtype=torch.float64)[:, None]).reshape(1, -1)
    v = 2.0 ** torch.tensor(exponents, dtype=torch.float64).repeat_interleave(128)[:, None] * below
    v = torch.minimum(v, top)
    v[:, 0] = top[:, 0]
    v[:, 1::2] *= -1
    return v.repeat(1, copies).to(BF16)


def wanted(v, axis, fmt):
    s = (v.double().abs().amax(axis, keepdim=True) / fmt[2]).float()
    return torch.where(s >= 2.0 ** -126, quantised(v.double(), axis, fmt)[0], 0.0)


def check(got, want):
    got, want = got.double().cpu(), want * UP
    bad = ~((got - want).abs() <= 2.0 ** -7 * want.abs())
    assert not bad.any(), (int(bad.sum()), bad.numel(), bad.nonzero()[0].tolist(), got[bad][0], want[bad][0])


def pick(n):
    return (torch.eye(n, device=DEV) * UP).to(BF16)


DZ = [-111, -110, -109, -105, -101, -90, -76, -40]
X = [-118, -117, -116, -113, -112, -109, -60, -40]


@pytest.mark.parametrize("act", ["none", "relu"])
@pytest.mark.parametrize("copies", [1, 2])       # 2: too many columns for the third pass to join
def test_codes_of_dz_by_rows(copies, act):
    dy = pairs(DZ, 34, copies)
    M, N = dy.shape
    wt = torch.eye(N, device=DEV).to(torch.float8_e4m3fn)
    dx, _, _ = binding.fp8_linear_backward(dy.to(DEV), None, wt, torch.full((N,), UP, device=DEV),
                                           torch.ones(M, N, dtype=BF16, device=DEV), activation=act, dw=False)
    check(dx, wanted(dy, 1, E5M2))


@pytest.mark.parametrize("act", ["none", "relu"])
def test_codes_of_dz_by_columns(act):
    dy = pairs(DZ, 34).t().contiguous()
    M, N = dy.shape
    _, dw, _ = binding.fp8_linear_backward(dy.to(DEV), pick(M), None, None,
                                           torch.ones(M, N, dtype=BF16, device=DEV), activation=act, dx=False)
    check(dw, wanted(dy, 0, E5M2).t())


@pytest.mark.parametrize("copies", [1, 4])
def test_codes_of_x(copies):
    x = pairs(X, 19, copies).t().contiguous()
    dw = binding.fp8_linear_backward(pick(x.shape[0]), x.to(DEV), None, None, activation="none", dx=False)[1]
    check(dw, wanted(x, 0, E4M3))


def test_codes_of_x_beside_a_smooth_activation():
    x = pairs(X, 19).t().contiguous()
    M = x.shape[0]
    z = torch.full((M, M), 200.0, dtype=BF16, device=DEV)        # slope 1
    dw = binding.fp8_linear_backward(pick(M), x.to(DEV), None, None, z, activation="silu", dx=False)[1]
    check(dw, wanted(x, 0, E4M3))
