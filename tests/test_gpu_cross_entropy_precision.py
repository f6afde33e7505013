"""How exact the cross entropy of an FP8 linear layer is on operands of a model: quantised
normal values, rows that have learnt their target more or less, half of the targets ignored.

test_gpu_cross_entropy allows each of a logit's K products the largest loss there can be, all
of one sign.  Here 2-norms over the rows are held to what products lose that are rounded
independently of each other, u = 2^-24 below:

 - The matrix instruction takes in at most 128 products and keeps each to 2^-13 of the largest, so
   a product loses at most 2^-13 max|a| max|b| over its 128, and the K of them, independent of
   each other, the root of the sum of these squares; K / 64 additions between instructions
   round by at most u of the sum of magnitudes S each.  That times the scale is d[m, j].
 - The target's logit is summed in fp32: at most K / 256 + 8 additions one after another, each off by
   at most u S at most: d[m, t] of a row that is not ignored.
 - lse moves by the sum of p[j] times a logit's error, the root of the sum of (p d)^2 for errors
   independent of each other; the sum of exponentials is off by `rel` of itself and the last
   steps round by 4 u (|lse| + 1), as there.
 - loss = log(1 + sum of the others over the target's) moves by p[j] times a logit's error for the
   others, by 1 - p[t] times the target's; all of the rest (rel, and the roundings of the
   exponent's two terms, 4 u of each) comes times 1 - p[t] too, and the logarithm rounds by 4 u of
   the loss.
"""
import math

import pytest
import torch

from precision_linear_amd import binding

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
U = 2.0 ** -24


def operands(M, V, K, mode, seed=0):
    g = torch.Generator(device=DEV).manual_seed(seed)
    w = 0.02 * torch.randn(V, K, generator=g, device=DEV)
    t = torch.randint(0, V, (M,), generator=g, device=DEV)
    rise = 18 * torch.rand(M, 1, generator=g, device=DEV)       # of the target's logit
    x = torch.randn(M, K, generator=g, device=DEV) + w[t] * (rise / (0.0004 * K))
    a, sa = binding.fp8_quantize(x.bfloat16(), mode)
    b, sb = binding.fp8_quantize(w.bfloat16(), mode)
    return (a, b, sa.reshape(-1), sb.reshape(-1)), torch.where(torch.arange(M, device=DEV) % 2 == 0, -100, t), t


@pytest.mark.parametrize("mode", ["rowwise", "per_tensor"])
@pytest.mark.parametrize("M,V,K", [(2000, 5000, 2048), (300, 1200, 4096), (1000, 20000, 512), (1500, 3001, 128),
                                   (400, 40000, 64), (16, 9000, 1024)])
def test_loss_and_lse_on_a_models_operands(M, V, K, mode):
    print(f"[cross entropy precision] {M} x {V} x {K} {mode}", flush=True)
    t, target, entry = operands(M, V, K, mode)
    loss, lse = binding.fp8_linear_cross_entropy(*t, target, mode=mode)
    a, b = (x.view(torch.float8_e4m3fn).double() for x in t[:2])
    s = t[2].double()[:, None] * t[3].double()[None, :] if mode == "rowwise" else t[2].double() * t[3].double()
    z = torch.mm(a, b.t()) * s
    want = torch.logsumexp(z, 1)
    p = torch.exp(z - want[:, None])
    most = z.amax(1).abs()

    per = min(128, K)
    largest = [x.abs().view(x.shape[0], K // per, per).amax(2) for x in (a, b)]
    sums = torch.mm(a.abs(), b.abs().t()) * s
    d = 2.0 ** -13 * (per * torch.mm(largest[0].square(), largest[1].square().t())).sqrt() * s + U * K / 64 * sums
    kept = target != -100
    rows = torch.arange(M, device=DEV)
    at = entry[:, None]
    d_target = (K / 256 + 8) * U * sums.gather(1, at)[:, 0] + 3 * U * z.gather(1, at)[:, 0].abs()
    d[rows[kept], entry[kept]] = d_target[kept]
    pd = (p * d).square()
    rel = U * (3 * (p * (z.abs() + most[:, None])).sum(1) + 74 + 8 * (math.ceil(V / 16 / 1024) + 18))
    tol_lse = pd.sum(1).sqrt() + rel + 4 * U * (want.abs() + 1)

    zt, pt = (x.gather(1, at)[:, 0] for x in (z, p))
    exact = torch.where(kept, want - zt, 0.0)
    left = torch.where(kept, 1 - pt, 0.0)
    others = (pd.sum(1) - pd.gather(1, at)[:, 0]).clamp(min=0).sqrt()
    tol_loss = torch.where(kept, others, 0.0) + left * (d_target + rel + 4 * U * (most + zt.abs())) + 4 * U * exact

    norm = lambda x: float(x.square().mean().sqrt())            # noqa: E731
    off = lse.double() - want
    figures = []
    for rows_of in (kept, ~kept):
        got, most_ = norm(off[rows_of]), norm(tol_lse[rows_of])
        figures.append(f"lse {got:.1e} of {most_:.1e}")
        assert got <= most_
    got, most_ = norm(loss.double() - exact), norm(tol_loss)
    print(*figures, f"loss {got:.1e} of {most_:.1e}, relative {got / norm(exact):.1e}", flush=True)
    assert got <= most_
    assert (loss[~kept] == 0).all()
    # What this tells apart: a sum that is off by a thousandth in every row.
    assert norm(tol_lse[kept]) < 1e-3 and norm(tol_loss) < 1e-3
