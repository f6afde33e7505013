"""The linear layer's epilogue (fp8_linear) on the GPU against 64 bits.

Tolerances.  The sum over K is the scaled multiply's, held to that multiply's
parity bound, 1e-3 of the sum of magnitudes (the additions inside a matrix
instruction are not single fp32 roundings); where the operands are whole numbers
whose sums fp32 holds exactly, z is exact up to the roundings of its scale and
bias and the epilogue is seen alone.  The activations' slopes are at most 1.13 in size, their
own error is at most 4e-5 relative (the fit of the normal distribution function)
plus a few fp32 roundings of z, and each output is rounded once, by at most
torch.finfo(bf16).eps / 2 of the value.
"""
import numpy as np
import pytest
import torch

from precision_linear_amd import binding

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF16 = torch.bfloat16
HALF = torch.finfo(BF16).eps / 2
ACTS = ("none", "relu", "gelu", "gelu_tanh", "silu")
F8 = {"e4m3fn": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2}


def act64(z, act):
    if act == "relu":
        return z.clamp(min=0)
    if act == "gelu":
        return z * 0.5 * torch.special.erfc(-z / 2 ** 0.5)
    if act == "gelu_tanh":
        return z * torch.sigmoid(2 * (2 / torch.pi) ** 0.5 * (z + 0.044715 * z ** 3))
    if act == "silu":
        return z * torch.sigmoid(z)
    return z


def make(M, N, K, mode, seed, fa="e4m3fn", fb="e4m3fn", bias=True, residual=True):
    g = torch.Generator().manual_seed(seed)
    a = (2 * torch.randn(M, K, generator=g)).to(F8[fa])
    b = (2 * torch.randn(N, K, generator=g)).to(F8[fb])
    row = mode == "rowwise"
    sa = torch.rand(M if row else 1, generator=g) + 0.5
    sb = (torch.rand(N if row else 1, generator=g) + 0.5) / (4 * K ** 0.5)
    bi = torch.randn(N, generator=g).to(BF16) if bias else None
    re = torch.randn(M, N, generator=g).to(BF16) if residual else None
    return dict(a=a, b=b, scale_a=sa, scale_b=sb, bias=bi, residual=re)


def make_whole(M, N, K, mode, seed, **kw):
    """The same with whole numbers of at most 4 in size as operands: sums below 2^24 are exact."""
    t = make(M, N, K, mode, seed, **kw)
    assert 16 * K < 2 ** 24
    for k in ("a", "b"):
        t[k] = t[k].float().round().clamp(-4, 4).to(t[k].dtype)
    return {**t, "whole": True}


def reference(t, act):
    """(z, bound of its fp32 error, out, bound) in 64 bits."""
    a, b = t["a"].double(), t["b"].double()
    s = t["scale_a"].double().reshape(-1, 1) * t["scale_b"].double().reshape(1, -1)
    bias = 0 if t["bias"] is None else t["bias"].double()
    z = s * (a @ b.t()) + bias
    if t.get("whole"):      # the scales' product, and the scaling and the bias in one fma
        zerr = 2.0 ** -24 * (s * (a @ b.t())).abs() + 2.0 ** -24 * z.abs()
    else:
        zerr = 1e-3 * s * (a.abs() @ b.abs().t()) + 2.0 ** -23 * z.abs()
    y = act64(z, act)
    res = 0 if t["residual"] is None else t["residual"].double()
    out = y + res
    err = 1.13 * zerr + (4e-5 * y.abs() + 2.0 ** -22 * z.abs() if act not in ("none", "relu") else 0)
    return z, zerr, out, err + 2.0 ** -24 * out.abs()


def within(name, got, want, tol):
    got = got.double().cpu()
    bad = ~((got - want).abs() <= tol)
    assert not bad.any(), (f"{name}: {int(bad.sum())} of {bad.numel()} outside, first at "
                           f"{tuple(bad.nonzero()[0].tolist())}: {got[bad][0]} against {want[bad][0]}")


def to_dev(t):
    return {k: None if v is None else v.to(DEV) for k, v in t.items() if k != "whole"}


def check(t, act="none", preact=True, **kw):
    M, N = t["a"].shape[0], t["b"].shape[0]
    print(f"[linear] {M} x {N} x {t['a'].shape[1]} act={act} preact={preact} {kw}", flush=True)
    pre = torch.full((M, N), float("nan"), dtype=BF16, device=DEV) if preact else None
    out = binding.fp8_linear(**to_dev(t), activation=act, preact=pre, **kw)
    torch.cuda.synchronize()
    z, zerr, want, err = reference(t, act)
    if preact:
        within("preact", pre, z, zerr + HALF * (z.abs() + zerr))
    within("out", out, want, err + HALF * (want.abs() + err))
    return out, pre


CONFIGS = range(12)
PLANS = [(c, s) for c in CONFIGS for s in (1, 3)]


@pytest.mark.parametrize("config,splits", PLANS)
@pytest.mark.parametrize("M,N", [(300, 264), (129, 203), (17, 100)])
def test_every_configuration(M, N, config, splits):
    K = 1040
    check(make(M, N, K, "rowwise", config + M), "gelu", mode="rowwise", config=config, splits=splits)
    t = make_whole(M, N, K, "rowwise", config + M)
    check(t, "gelu", mode="rowwise", config=config, splits=splits)
    check({**t, "residual": None}, "silu", preact=False, mode="rowwise", config=config, splits=splits)


@pytest.mark.parametrize("mode", ["rowwise", "per_tensor"])
@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("bias", [True, False])
@pytest.mark.parametrize("residual", [True, False])
@pytest.mark.parametrize("preact", [True, False])
def test_every_epilogue(mode, act, bias, residual, preact):
    for M, N, K in ((512, 512, 256), (40, 1000, 2048)):
        check(make(M, N, K, mode, M, bias=bias, residual=residual), act, preact, mode=mode)
        check(make_whole(M, N, K, mode, M, bias=bias, residual=residual), act, preact, mode=mode)


@pytest.mark.parametrize("fa", F8)
@pytest.mark.parametrize("fb", F8)
def test_operand_formats(fa, fb):
    for config in (2, 8, 11):
        check(make(256, 512, 400, "rowwise", 3, fa, fb), "gelu_tanh", config=config)


@pytest.mark.parametrize("M,N,K", [(1, 1, 16), (1, 28672, 8192), (3, 5, 32), (64, 8192, 4096), (1152, 4096, 2048),
                                   (2049, 1000, 96), (4095, 4097, 96), (256, 257, 48), (700, 3, 512)])
def test_automatic_plans(M, N, K):
    check(make(M, N, K, "rowwise", M + N), "gelu", mode="rowwise")
    check(make_whole(M, N, K, "rowwise", M + N), "gelu", mode="rowwise")
    check(make(M, N, K, "per_tensor", M + N, bias=False), "relu", preact=False, mode="per_tensor")


@pytest.mark.parametrize("act", ACTS)
def test_activation_of_every_finite_bf16_value(act):
    # codes 0: z is the bias itself
    bits = torch.arange(65536, dtype=torch.int32).to(torch.int16)
    v = bits.view(BF16)
    v = v[torch.isfinite(v.float())]
    n = v.numel() // 16 * 16
    for part in (v[:n], v[-n:]):
        t = dict(a=torch.zeros(2, 16).to(F8["e4m3fn"]), b=torch.zeros(n, 16).to(F8["e4m3fn"]),
                 scale_a=torch.ones(2), scale_b=torch.ones(n), bias=part.contiguous(), residual=None)
        pre = torch.empty(2, n, dtype=BF16, device=DEV)
        out = binding.fp8_linear(**to_dev(t), activation=act, preact=pre).double().cpu()
        assert torch.equal(pre[0].cpu().float(), part.float())
        z = part.double()
        want = act64(z, act)
        big = z.abs() > 1e12                      # (the cube of gelu_tanh leaves fp32 first)
        want = torch.where(big & (torch.tensor(act != "none")), z.clamp(min=0), want)
        # z^2 in the exponent is off by 2^-24 z^2 (a relative error of the tail), and results below
        # 2^-120 may be flushed to 0
        tol = want.abs() * (HALF + 4e-5 + 2.0 ** -23 * torch.minimum(z.square(), torch.tensor(200.0)).double()) + 2.0 ** -118
        within(act, out[0], want, tol)
        assert torch.equal(out[0], out[1])


def test_epilogue_without_anything_is_the_multiply():
    t = to_dev(make(700, 520, 640, "rowwise", 5, residual=False))
    want = binding.fp8_scaled_mm(t["a"], t["b"], t["scale_a"], t["scale_b"], t["bias"], mode="rowwise")
    pre = torch.empty_like(want)
    zero = torch.zeros_like(want)
    assert torch.equal(binding.fp8_linear(**t), want)
    for config in CONFIGS:
        out = binding.fp8_linear(**t, preact=pre, config=config, splits=1)
        ref = binding.fp8_scaled_mm(t["a"], t["b"], t["scale_a"], t["scale_b"], t["bias"], mode="rowwise",
                                    config=config, splits=1)
        assert torch.equal(out, ref) and torch.equal(pre, ref), config
        assert torch.equal(binding.fp8_linear(**{**t, "residual": zero}, config=config, splits=1), ref), config


@pytest.mark.parametrize("M,N", [(300, 264), (70, 203)])
@pytest.mark.parametrize("config", [1, 8, 9, 11])
def test_residual_in_place_and_tensors_off_the_vector_boundary(M, N, config):
    t = make(M, N, 272, "rowwise", 9)
    want, pre0 = check(t, "silu", config=config)
    d = to_dev(t)
    buf = d["residual"].clone()
    assert binding.fp8_linear(**{**d, "residual": buf}, activation="silu", out=buf, config=config) is buf
    assert torch.equal(buf, want)

    def shifted(x, by):
        store = torch.full((x.numel() + 64,), 5.0, dtype=BF16, device=DEV)
        view = store[by:by + x.numel()].view(x.shape)
        view.copy_(x)
        return view, store

    for by in (1, 2, 4, 8):
        (res, _), (pre, ps), (out, os_) = shifted(t["residual"], by), shifted(want, 9 - by), shifted(want, by + 1)
        bias, _ = shifted(t["bias"], by)
        binding.fp8_linear(**{**d, "residual": res, "bias": bias}, activation="silu", preact=pre, out=out,
                           config=config)
        assert torch.equal(out, want) and torch.equal(pre, pre0)
        for store, at in ((ps, 9 - by), (os_, by + 1)):
            assert (store[:at] == 5).all() and (store[at + M * N:] == 5).all()


def test_not_finite_values_stay_where_they_are():
    t = make(40, 64, 64, "rowwise", 2)
    clean = binding.fp8_linear(**to_dev(t), activation="gelu")
    t["residual"][3, 5] = float("inf")
    t["bias"][7] = float("nan")
    for act in ACTS:
        out = binding.fp8_linear(**to_dev(t), activation=act)
        assert out[:, 7].isnan().all() and out[3, 5] == float("inf")
        if act == "gelu":
            keep = torch.ones_like(out, dtype=torch.bool)
            keep[:, 7] = keep[3, 5] = False
            assert torch.equal(out[keep], clean[keep])


def test_empty_outputs():
    t = to_dev(make(4, 32, 64, "rowwise", 1))
    assert binding.fp8_linear(**{**t, "a": t["a"][:0], "scale_a": t["scale_a"][:0], "residual": t["residual"][:0]},
                              activation="gelu").shape == (0, 32)


def test_graph_replays_match_eager():
    plain = to_dev(make(512, 768, 1024, "per_tensor", 1))
    split = to_dev(make(128, 1024, 8192, "rowwise", 2))
    assert binding.select_splits(128, 1024, 8192, "rowwise", True) > 1
    outs = [torch.empty(512, 768, dtype=BF16, device=DEV), torch.empty(128, 1024, dtype=BF16, device=DEV)]
    pres = [torch.empty_like(o) for o in outs]

    def calls():
        binding.fp8_linear(**plain, activation="gelu", preact=pres[0], out=outs[0], mode="per_tensor")
        binding.fp8_linear(**split, activation="silu", preact=pres[1], out=outs[1])

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        calls()
    torch.cuda.synchronize()
    want = [t.clone() for t in outs + pres]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        calls()
    for rep in range(4):
        for t in outs + pres:
            t.zero_()
        junk = torch.randn(256, 256, device=DEV) @ torch.randn(256, 256, device=DEV)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for a, c in zip(outs + pres, want):
            assert torch.equal(a, c), f"replay {rep} differs"
        del junk


def test_refusals_with_gpu_tensors():
    t = to_dev(make(16, 32, 64, "rowwise", 1))
    good = torch.empty(16, 32, dtype=BF16, device=DEV)
    f = binding.fp8_linear
    for kw in (dict(activation="swish"), dict(activation=2), dict(residual=good.float()), dict(residual=good[:8]),
               dict(residual=good.cpu()), dict(residual=good.t().contiguous().t()), dict(preact=good.float()),
               dict(preact=good[:, :16]), dict(preact=good.cpu()), dict(out=good[:8]), dict(mode="blockwise"),
               dict(scale_a=t["scale_a"][:3]), dict(bias=t["bias"].float()), dict(config=99),
               dict(preact=good, splits=binding.SPLITS_STREAM_K)):
        with pytest.raises(ValueError):
            f(**{**t, **kw})
