"""A weight's codes in both layouts on the GPU: the bits of the plain definition (scales
the fp32 maxima over qmax, quotients correctly rounded, torch's CPU float8 casts)."""
import math

import pytest
import torch

from precision_linear_amd import binding

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
QMAX = {"e4m3fn": 448.0, "e5m2": 57344.0}
FP8 = {"e4m3fn": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2}


def plain(w, fmt):
    """(q, scale) of w's rows, on the CPU."""
    w = w.float()
    amax = torch.where(w.isnan(), 0.0, w.abs()).amax(1) if w.shape[1] else torch.zeros(w.shape[0])
    scale = amax / torch.full_like(amax, QMAX[fmt])
    v = torch.where(scale[:, None] > 0, w / scale[:, None], w * 0)
    return v.clamp(-QMAX[fmt], QMAX[fmt]).to(FP8[fmt]).view(torch.uint8), scale


def same_codes(got, want, fmt):
    """Equal bits; NaNs of either sign."""
    nan = want.view(FP8[fmt]).float().isnan()
    assert torch.equal(got.view(FP8[fmt]).float().isnan(), nan)
    assert torch.equal(torch.where(nan, 0, got), torch.where(nan, 0, want))


def check(w, got, fmt):
    w = w.cpu()
    N, K = w.shape
    q, scale = plain(w, fmt)
    qt, scale_t = plain(w.t(), fmt)
    assert got.q.shape == (N, K) and got.qt.shape == (K, (N + 15) // 16 * 16)
    assert torch.equal(got.scale.cpu(), scale) and torch.equal(got.scale_t.cpu(), scale_t)
    same_codes(got.q.cpu().view(torch.uint8), q, fmt)
    same_codes(got.qt.cpu().view(torch.uint8)[:, :N].contiguous(), qt, fmt)
    assert (got.qt.view(torch.uint8)[:, N:] == 0).all()


def make(N, K, dtype, seed=0):
    g = torch.Generator(device=DEV).manual_seed(seed + N)
    w = torch.randn(N, K, generator=g, device=DEV) * torch.exp(torch.randn(N, 1, generator=g, device=DEV))
    return (w * torch.exp(torch.randn(1, K, generator=g, device=DEV))).to(dtype)


SHAPES = [(1, 16), (1, 4096), (2, 48), (15, 32), (16, 16), (17, 144), (63, 128), (64, 1008), (65, 112), (127, 272),
          (1000, 4160), (2049, 1024), (100, 9008), (9001, 96), (70001, 32), (300, 28672)]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("N,K", SHAPES)
def test_codes(N, K, dtype):
    w = make(N, K, dtype)
    for fmt in ("e4m3fn", "e5m2"):
        print(f"[quantize_weight] {N} x {K} {dtype} {fmt}", flush=True)
        check(w, binding.fp8_quantize_weight(w, fmt), fmt)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("N,K", [(255, 2048), (256, 4096), (256, 4112), (257, 2064), (128, 8192), (128, 8208), (1023, 1024),
                                 (1024, 1024), (1025, 1008), (1009, 32), (1, 8192), (1, 8208)])
def test_around_the_variants(N, K, dtype):
    w = make(N, K, dtype, seed=4)
    w[N // 2] = 0
    w[:, K - 1] = 0
    check(w, binding.fp8_quantize_weight(w), "e4m3fn")
    w[N // 3] *= 2.0 ** -70                    # (scales whose quotients are divisions)
    w[:, 5] *= 2.0 ** -75
    check(w, binding.fp8_quantize_weight(w, "e5m2"), "e5m2")


@pytest.mark.parametrize("N,K", [(2000, 4096), (64, 144)])
def test_the_quantisers_own_bits(N, K):
    w = make(N, K, torch.bfloat16)
    got = binding.fp8_quantize_weight(w)
    q, scale = binding.fp8_quantize(w, "rowwise")
    assert torch.equal(got.q, q) and torch.equal(got.scale, scale)
    q, scale = binding.fp8_quantize(w.t().contiguous(), "rowwise")
    assert torch.equal(got.qt, q) and torch.equal(got.scale_t, scale)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_beyond_the_memory_side_cache(dtype):
    """Rows and columns do not depend on the matrix's other ones' codes: a large one has the
    bits of its parts."""
    N, K = 20001, 8192
    assert N * K * 2 > 256 << 20
    w = make(N, K, dtype)
    got = binding.fp8_quantize_weight(w)
    for r0, r1 in ((0, 300), (9000, 9300), (N - 65, N)):
        part = binding.fp8_quantize_weight(w[r0:r1])
        assert torch.equal(got.q[r0:r1], part.q) and torch.equal(got.scale[r0:r1], part.scale)
    for c in (0, 4096, K - 128):
        part = binding.fp8_quantize_weight(w[:, c:c + 128].contiguous())
        assert torch.equal(got.qt[c:c + 128], part.qt) and torch.equal(got.scale_t[c:c + 128], part.scale_t)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("N,K", [(20, 32), (1000, 1040)])
def test_zeros_tiny_values_and_no_numbers(N, K, dtype):
    w = make(N, K, dtype)
    w[3] = 0
    w[:, 5] = 0
    w[4] *= 1e-36             # scales below 2^-60, where the fast quotient does not hold
    w[:, 6] = 2.0 ** -130
    w[7, 8] = 3e38
    for fmt in ("e4m3fn", "e5m2"):
        check(w, binding.fp8_quantize_weight(w, fmt), fmt)
    w[9, 10] = math.nan
    w[11] = math.nan
    w[12, 13] = -math.inf
    for fmt in ("e4m3fn", "e5m2"):
        check(w, binding.fp8_quantize_weight(w, fmt), fmt)


def test_odd_addresses():
    for dtype in (torch.bfloat16, torch.float32):
        flat = make(1, 100 * 64 + 16, dtype).flatten()
        for off in (1, 3):
            w = flat[off:off + 6400].view(100, 64)
            check(w, binding.fp8_quantize_weight(w), "e4m3fn")


def test_no_rows():
    got = binding.fp8_quantize_weight(torch.empty(0, 64, device=DEV))
    assert got.q.shape == (0, 64) and got.qt.shape == (64, 0) and got.scale.shape == (0,)
    assert (got.scale_t == 0).all() and got.scale_t.shape == (64,)


def test_given_buffers_and_any_workspace():
    N, K = 333, 208
    w = make(N, K, torch.float32)
    want = binding.fp8_quantize_weight(w)
    need = binding.lib().fp8_quantize_weight_workspace_size(N, K)
    for fill in (0, 0xff):
        ws = torch.full((need,), fill, dtype=torch.uint8, device=DEV)
        out = dict(q=torch.full((N, K), 1, dtype=torch.uint8, device=DEV).view(torch.float8_e4m3fn),
                   scale=torch.full((N,), -1.0, device=DEV), qt=torch.full((K, 336), 1, dtype=torch.uint8, device=DEV),
                   scale_t=torch.full((K,), -1.0, device=DEV))
        got = binding.fp8_quantize_weight(w, **out, workspace=ws)
        for a, b, c in zip(got, want, out.values()):
            assert a is c and torch.equal(a.view(b.dtype), b)
    with pytest.raises(ValueError):
        binding.fp8_quantize_weight(w, workspace=ws[:-1])


def test_given_buffers_count_as_written():
    """A graph that saved the old codes refuses to run backward on the new ones."""
    w = make(64, 32, torch.float32)
    out = binding.fp8_quantize_weight(w)
    x = torch.ones(64, device=DEV, requires_grad=True)
    y = (x * out.scale).sum()
    before = [t._version for t in out]
    binding.fp8_quantize_weight(w, **out._asdict())
    assert all(t._version > v for t, v in zip(out, before))
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        y.backward()


def test_the_most_rows():
    N, K = 2 ** 27 - 13, 16                     # elements past 2^31
    w = torch.empty(N, K, dtype=torch.bfloat16, device=DEV)
    w.uniform_(-1, 1, generator=torch.Generator(device=DEV).manual_seed(3))
    w[N - 5] *= 3
    w[:, 3] /= 4
    got = binding.fp8_quantize_weight(w)
    most = w.abs().amax(1).cpu().float()
    assert torch.equal(got.scale.cpu(), most / torch.full_like(most, 448))
    most = w.abs().amax(0).cpu().float()
    assert torch.equal(got.scale_t.cpu(), most / torch.full_like(most, 448))
    assert (got.qt[:, N:] == 0).all()
    for r in (0, 2 ** 26 - 40, 2 ** 27 - 100):
        part = w[r:r + 87].cpu().float()
        for codes, scale in ((got.q[r:r + 87], got.scale[r:r + 87, None]), (got.qt[:, r:r + 87].t(), got.scale_t)):
            assert torch.equal(codes.cpu(), (part / scale.cpu()).to(FP8["e4m3fn"]).view(torch.uint8)), r


def test_captured_and_replayed():
    ws = [make(N, K, dt) for N, K, dt in ((50, 64, torch.bfloat16), (3000, 4096, torch.float32), (100, 9008, torch.bfloat16))]
    want = [binding.fp8_quantize_weight(w) for w in ws]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=torch.cuda.Stream()):
        outs = [binding.fp8_quantize_weight(w) for w in ws]
    for rep in range(3):
        for o in outs:
            for x in o:
                x.zero_()
        binding.fp8_quantize_weight(ws[rep])
        graph.replay()
        torch.cuda.synchronize()
        for o, w in zip(outs, want):
            assert all(torch.equal(x, y) for x, y in zip(o, w)), rep
