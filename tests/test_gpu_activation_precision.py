"""The linear layer's activations in fp32: a residual of minus the rounded result
leaves only its last bits, which an output's rounding no longer hides.

The products are 0, so that z is the bias.  Bounds (U = 2^-24, a hardware exp2 or
reciprocal counts as 2 roundings): gelu is z (1 - q) or z q with q off by the fit of
the normal distribution function (1.5e-7), 12 roundings and 2 of an exponent of
z^2 / 2; gelu_tanh and silu are z p with p off by 5 roundings and 4 (1) of an
exponent of |2 u| (|z|); then the product, the addition, and the output's own
rounding of half a step.
"""
import pytest
import torch

from precision_linear_amd import binding
from test_gpu_linear import BF16, CONFIGS, DEV, F8, HALF, act64, within

pytestmark = pytest.mark.gpu
U = 2.0 ** -24


def bound(z, act):
    y = act64(z, act).abs()
    if act == "gelu":
        q = 0.5 * torch.special.erfc(z.abs() / 2 ** 0.5)
        return z.abs() * (q * (1.5e-7 + 12 * U + 2 * U * z * z / 2) + U) * (1 + U) + U * y
    if act == "gelu_tanh":
        exponent = (2 * (2 / torch.pi) ** 0.5 * (z + 0.044715 * z ** 3)).abs()
        return y * (6 * U + 4 * U * exponent)
    return y * (6 * U + 2 * U * z.abs())


@pytest.mark.parametrize("act", ["gelu", "gelu_tanh", "silu"])
@pytest.mark.parametrize("config", [-1, *CONFIGS])
def test_what_a_residual_leaves(config, act):
    v = torch.arange(65536, dtype=torch.int32).to(torch.int16).view(BF16)
    v = v[(v.float().abs() >= 2.0 ** -6) & (v.float().abs() <= 8)]
    N, M = v.numel() // 16 * 16, 3
    v = v[:N].contiguous()
    z = v.double()
    y = act64(z, act)
    res = (-y).to(BF16)
    print(f"[linear] {act} config={config}", flush=True)
    out = binding.fp8_linear(torch.zeros(M, 512).to(F8["e4m3fn"]).to(DEV), torch.zeros(N, 512).to(F8["e4m3fn"]).to(DEV),
                             torch.ones(M, device=DEV), torch.ones(N, device=DEV), v.to(DEV),
                             res.to(DEV).expand(M, -1).contiguous(), activation=act, config=config)
    want = y + res.double()
    err = bound(z, act) + U * want.abs()
    for row in out:
        within(act, row, want, err + HALF * (want.abs() + err))
