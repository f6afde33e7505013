"""The softmax cross entropy of an FP8 linear layer on the GPU against 64 bits.

Tolerances.  A logit is a sum of K products and two multiplications by its scale.  The
matrix instruction keeps a product to 2^-13 of the largest one that it takes in (seen
with two products, the smaller one halved until it is lost: 2^8 + 2^-5 is kept, 2^8 +
2^-6 gives 2^8), so each of K products loses at most 2^-13 of max|a| max|b|, and the
fp32 additions between instructions round by at most u = 2^-24 of the sum of magnitudes
S: a logit is off by at most dz = (2^-13 K max|a| max|b| + u K S) s + 4 u |z| (it is kept
times log2(e): three multiplications, and the constant's own u / 4).  Where a and b are
halves up to 2 (whole=True), products are multiples of 1/4 up to 4, every sum is exact,
and dz = 4 u |z|.  lse moves by at most the largest dz of its row; the sum of
exponentials adds, relative to itself, the rounding of each exponent (at most 3 u (|z| +
|largest|)), of each exponential (the hardware's 2^x is off by at most 2 u) and of the
additions: 64 within a lane, 8 between lanes and, for each join of two partial sums, up
to 8192 in a row in the slices and 10 after, twice the two exponentials' 2 u and two
roundings.  The last steps, the logarithm, its addition and the multiplication by
ln(2), round by 4 u (|lse| + 1).
"""
import math

import pytest
import torch

from precision_linear_amd import binding

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
U = 2.0 ** -24
FP8 = {"e4m3fn": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2}


def make(M, V, K, mode="rowwise", fa="e4m3fn", fb="e4m3fn", seed=0, ignore=None, size=1.0, whole=False):
    g = torch.Generator(device=DEV).manual_seed(seed + 7 * M + V)
    a = (size * torch.randn(M, K, generator=g, device=DEV)).clamp(-400, 400).to(FP8[fa])
    b = torch.randn(V, K, generator=g, device=DEV).to(FP8[fb])
    if whole:
        a, b = ((torch.randint(-4, 5, t.shape, generator=g, device=DEV) / 2).to(t.dtype) for t in (a, b))
    scale = lambda n: 2.0 ** (torch.rand(n, generator=g, device=DEV) - 0.5)      # noqa: E731
    one = mode == "per_tensor"
    sa, sb = scale(1 if one else M), scale(1 if one else V) / math.sqrt(K)
    t = torch.randint(0, V, (M,), generator=g, device=DEV)
    if ignore is not None:
        t[torch.rand(M, generator=g, device=DEV) < 0.3] = ignore
    return a, b, sa, sb, t


def logits64(a, b, sa, sb):
    """(logits, bound of their fp32 form's error)"""
    s = sa.double()[:, None] * sb.double()[None, :] if sa.numel() == a.shape[0] and sb.numel() == b.shape[0] else \
        sa.double() * sb.double()
    x, y = a.double(), b.double()
    z = torch.mm(x, y.t()) * s
    if all(t.numel() == 0 or (t * 2 == (t * 2).round()).all() and t.abs().max() <= 2 for t in (x, y)):
        return z, 4 * U * z.abs()
    largest = x.abs().amax(1)[:, None] * y.abs().amax(1)[None, :]
    return z, a.shape[1] * (2.0 ** -13 * largest + U * torch.mm(x.abs(), y.abs().t())) * s.abs() + 4 * U * z.abs()


def check(loss, lse, a, b, sa, sb, t, ignore=-100):
    z, dz = logits64(a, b, sa, sb)
    M, V = z.shape
    most = z.amax(1)
    want = torch.logsumexp(z, 1)
    p = torch.exp(z - want[:, None])
    rel = U * (3 * (p * (z.abs() + most.abs()[:, None])).sum(1) + 2 + 72 + 8 * (math.ceil(V / 16 / 1024) + 18))
    tol = dz.amax(1) + rel + 4 * U * (want.abs() + 1)
    assert lse.dtype == loss.dtype == torch.float32 and lse.shape == loss.shape == (M,)
    assert ((lse.double() - want).abs() <= tol).all(), ((lse.double() - want).abs() / tol).max()
    kept = t != ignore
    zt = z.gather(1, torch.where(kept, t, 0)[:, None])[:, 0]
    want = torch.where(kept, want - zt, 0.0)
    tol = tol + dz.amax(1) + 4 * U * (most.abs() + zt.abs())
    assert ((loss.double() - want).abs() <= torch.where(kept, tol, 0.0)).all()


SHAPES = [(1, 1, 16), (1, 2, 32), (1, 17, 16), (1, 32000, 2048), (2, 100, 48), (3, 1000, 1024), (15, 255, 16),
          (16, 257, 512), (17, 113, 64), (33, 5000, 4096), (64, 4096, 128), (65, 33, 8192), (100, 513, 160),
          (129, 10007, 1024), (256, 256, 128), (257, 1008, 256), (511, 50255, 272), (1000, 6001, 2048),
          (2048, 8200, 384), (4099, 12289, 144), (70000, 300, 32)]


@pytest.mark.parametrize("M,V,K", SHAPES)
def test_loss(M, V, K):
    for mode, ignore, whole in (("rowwise", None, False), ("per_tensor", -100, False), ("rowwise", -100, True),
                                ("per_tensor", None, True)):
        print(f"[cross entropy] {M} x {V} x {K} {mode} {whole}", flush=True)
        t = make(M, V, K, mode, ignore=ignore, whole=whole)
        loss, lse = binding.fp8_linear_cross_entropy(*t, mode=mode)
        check(loss, lse, *t)


@pytest.mark.parametrize("fa", ["e4m3fn", "e5m2"])
@pytest.mark.parametrize("fb", ["e4m3fn", "e5m2"])
@pytest.mark.parametrize("M,V,K", [(1, 3000, 512), (70, 1001, 256), (1300, 9000, 256)])
def test_formats(fa, fb, M, V, K):
    t = make(M, V, K, fa=fa, fb=fb, seed=3, whole=True)
    print(f"[cross entropy] {M} x {V} x {K} {fa} {fb}", flush=True)
    loss, lse = binding.fp8_linear_cross_entropy(*t)
    check(loss, lse, *t)
    bytes_ = binding.fp8_linear_cross_entropy(t[0].view(torch.uint8), t[1].view(torch.uint8), *t[2:], a_format=fa,
                                              b_format=fb)
    assert torch.equal(bytes_[0], loss) and torch.equal(bytes_[1], lse)


@pytest.mark.parametrize("size", [0.01, 300.0])
def test_logits_of_any_size(size):
    """Exponentials of logits around +-10000 are taken against the largest; equal logits give log V."""
    t = make(300, 2100, 1024, size=size, seed=5)
    if size > 1:
        t = (*t[:2], t[2] * 8, *t[3:])
        assert logits64(*t[:4])[0].abs().max() > 5000
    loss, lse = binding.fp8_linear_cross_entropy(*t)
    check(loss, lse, *t)


def test_no_logits():
    for M, V in ((5, 1000), (700, 2 ** 14)):
        t = make(M, V, 64)
        t[0].view(torch.uint8).zero_()
        loss, lse = binding.fp8_linear_cross_entropy(*t)
        assert torch.allclose(loss, torch.full_like(loss, math.log(V)), rtol=4 * U * 8, atol=0)
        assert torch.equal(loss, lse)


def test_a_sure_row_keeps_its_small_loss():
    """log(1 + V exp(-40)) is far below the last bit of its two logits."""
    a, b, sa, sb, t = make(20, 1000, 64)
    b.view(torch.uint8).zero_()
    t = torch.arange(20, device=DEV) * 49
    one = torch.ones(64, device=DEV).to(torch.float8_e4m3fn)
    b[t] = one
    a[:] = one
    sa, sb = torch.full_like(sa, 40 / 64), torch.ones_like(sb)
    loss, lse = binding.fp8_linear_cross_entropy(a[:1], b, sa[:1], sb, t[:1])
    want = math.log(20 + 980 * math.exp(-40.0))
    assert abs(float(loss) - want) < 4e-6 * want
    b[t[1:]] = 0
    loss, lse = binding.fp8_linear_cross_entropy(a[:1], b, sa[:1], sb, t[:1])
    want = math.log1p(999 * math.exp(-40.0))
    # the exponent, 40 log2(e) after three roundings and a difference, is off by 5 u of itself
    assert abs(float(loss) - want) <= 2 * 5 * U * 40 * want
    # 40 log2(e) after three multiplications, back by a fourth, each rounding by u, and the
    # two constants' own u / 4 and u / 20
    assert abs(float(lse) - 40) <= 5 * U * 40


@pytest.mark.parametrize("M,V", [(6, 100), (600, 9000)])
def test_rows_that_do_not_count(M, V):
    t = make(M, V, 64, ignore=-100, seed=9)
    a, b, sa, sb, target = t
    target[0], target[1], target[2], target[3] = -100, V, -1, 2 ** 40
    loss, lse = binding.fp8_linear_cross_entropy(*t)
    assert float(loss[0]) == 0 and loss[1:4].isnan().all() and lse.isfinite().all()
    check(torch.where(loss.isnan(), 0.0, loss), lse, a, b, sa, sb, torch.where(loss.isnan(), -100, target))
    for ignore in (0, V - 1, -1, 2 ** 40):
        got, _ = binding.fp8_linear_cross_entropy(*t, ignore_index=ignore)
        assert ((got == 0) == (target == ignore)).all()
    everything = torch.full_like(target, -100)
    assert (binding.fp8_linear_cross_entropy(a, b, sa, sb, everything)[0] == 0).all()


@pytest.mark.parametrize("M,V", [(1, 20), (6, 100), (600, 9000)])
def test_an_ignored_entry_of_the_vocabulary_is_in_the_sum(M, V):
    t = make(M, V, 64, seed=21, whole=True)
    for ignore in {int(t[4][0]), V - 1}:
        t[4][M // 2:] = ignore
        loss, lse = binding.fp8_linear_cross_entropy(*t, ignore_index=ignore)
        check(loss, lse, *t, ignore=ignore)


@pytest.mark.parametrize("M,V", [(6, 100), (600, 9000)])
def test_nan_rows_show(M, V):
    a, b, sa, sb, t = make(M, V, 64, seed=11)
    a.view(torch.uint8)[3, 5] = 0x7f
    loss, lse = binding.fp8_linear_cross_entropy(a, b, sa, sb, t)
    rest = torch.arange(M, device=DEV) != 3
    assert loss[3].isnan() and lse[3].isnan() and loss[rest].isfinite().all()
    t[3] = -100
    loss, lse = binding.fp8_linear_cross_entropy(a, b, sa, sb, t)
    assert float(loss[3]) == 0
    b.view(torch.uint8)[V - 1, 0] = 0x7f      # an entry of the vocabulary: every row
    loss, lse = binding.fp8_linear_cross_entropy(a, b, sa, sb, t)
    assert lse.isnan().all()


def test_infinite_logits():
    """-inf is no more than an exponential of 0, unless the target's; +inf shows."""
    M, V, K = 70, 1000, 64
    a, b, sa, sb, t = make(M, V, K, fb="e5m2", seed=12, whole=True)
    a.view(torch.uint8)[:, 0] = 0x38                     # 1
    clean = b.clone()
    clean[5] = 0
    b.view(torch.uint8)[5, 0] = 0xfc                     # -inf
    t[:] = torch.where(t == 5, 6, t)
    t[1] = 5
    loss, lse = binding.fp8_linear_cross_entropy(a, b, sa, sb, t)
    z = logits64(a, clean, sa, sb)[0]
    z[:, 5] = -math.inf
    want = torch.logsumexp(z, 1)
    assert ((lse.double() - want).abs() < 1e-5 * (1 + want.abs())).all()
    assert loss[1] == math.inf and loss[torch.arange(M, device=DEV) != 1].isfinite().all()
    b.view(torch.uint8)[5, 0] = 0x7c                     # +inf
    loss, lse = binding.fp8_linear_cross_entropy(a, b, sa, sb, t)
    assert loss.isnan().all() and lse.isnan().all()


def test_a_target_of_minus_infinity_hides_no_nan():
    a, b, sa, sb, t = make(70, 1000, 64, fb="e5m2", seed=22, whole=True)
    a.view(torch.uint8)[:, 0] = 0x38                     # 1
    b.view(torch.uint8)[5, 0] = 0xfc                     # -inf
    t[:] = 5
    loss, lse = binding.fp8_linear_cross_entropy(a, b, sa, sb, t)
    assert (loss == math.inf).all() and lse.isfinite().all()
    b.view(torch.uint8)[900, 0] = 0x7f
    loss, lse = binding.fp8_linear_cross_entropy(a, b, sa, sb, t)
    assert loss.isnan().all() and lse.isnan().all()
    # nothing but -inf: lse is that, and its difference to the target's no number
    loss, lse = binding.fp8_linear_cross_entropy(a, b[5:6], sa, sb[5:6], torch.zeros_like(t))
    assert loss.isnan().all() and (lse == -math.inf).all()


@pytest.mark.parametrize("M,V", [(2 ** 23 - 5, 40), (3, 2 ** 23 - 5)])
def test_the_largest_sizes(M, V):
    t = make(M, V, 16, seed=23, whole=True)
    loss, lse = binding.fp8_linear_cross_entropy(*t)
    check(loss, lse, *t)


def test_no_rows():
    t = make(0, 100, 64)
    loss, lse = binding.fp8_linear_cross_entropy(*t)
    assert loss.shape == lse.shape == (0,)


def test_equal_calls_equal_bits_whatever_the_workspace_holds():
    t = make(200, 3000, 4096, seed=13)
    need = binding.lib().fp8_linear_cross_entropy_workspace_size(200, 3000, 4096)
    got = []
    for fill in (0, 0xff, 0x7f):
        ws = torch.full((need,), fill, dtype=torch.uint8, device=DEV)
        got.append(binding.fp8_linear_cross_entropy(*t, workspace=ws))
    for loss, lse in got[1:]:
        assert torch.equal(loss, got[0][0]) and torch.equal(lse, got[0][1])
    check(*got[0], *t)
    with pytest.raises(ValueError):
        binding.fp8_linear_cross_entropy(*t, workspace=torch.empty(need - 1, dtype=torch.uint8, device=DEV))


def test_captured_and_replayed():
    calls = [make(M, V, K, seed=17) for M, V, K in ((1, 2000, 4096), (700, 9000, 256), (64, 1024, 8192))]
    want = [binding.fp8_linear_cross_entropy(*t) for t in calls]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=torch.cuda.Stream()):
        outs = [binding.fp8_linear_cross_entropy(*t) for t in calls]
    for rep in range(3):
        for o in outs:
            for x in o:
                x.fill_(-1)
        binding.fp8_linear_cross_entropy(*calls[rep])
        graph.replay()
        torch.cuda.synchronize()
        for o, w in zip(outs, want):
            assert all(torch.equal(x, y) for x, y in zip(o, w)), rep
