"""Layer norm, its quantisation and its gradient on the GPU against the
formulas in 64 bits.

Tolerances.  u = 2^-24 is the relative error of one fp32 operation.  A sum over
a row goes through at most 16 + 1 additions per lane and 4 + 2 + 4 levels of
joining (longer rows: cols / 8192 * 8 per lane), so a row's sum is off by at
most C u times the sum of magnitudes with C = 32 + cols / 1024, its square root
and quotient add a few u more; 2 C u covers each of mean, rstd and the sums of
the gradient.  A column sum takes rows / 256 + 64 additions.  Each output's own
rounding is half a step: torch.finfo(t).eps / 2 relative to the value.
"""
import numpy as np
import pytest
import torch

from precision_linear_amd import binding

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
U = 2.0 ** -24
EPS = 1e-5
QMAX = {"e4m3fn": 448.0, "e5m2": 57344.0}
F8 = {"e4m3fn": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2}
HALF_STEP = {"e4m3fn": (2.0 ** -4, 2.0 ** -10), "e5m2": (2.0 ** -3, 2.0 ** -17)}   # relative, subnormal
BF16, FP32 = torch.bfloat16, torch.float32


def steps(cols):
    return 2 * (32 + cols / 1024)


def make(rows, cols, dtype, seed, params=FP32):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(rows, cols, generator=g) * torch.exp(torch.randn(rows, 1, generator=g))
    x += 3 * torch.randn(rows, 1, generator=g)
    w = 1 + 0.3 * torch.randn(cols, generator=g)
    b = 0.3 * torch.randn(cols, generator=g)
    return x.to(dtype), w.to(params), b.to(params)


def reference(x, w, b, eps=EPS):
    """(y, mean, rstd, bound on the fp32 y's error) in 64 bits."""
    x = x.double()
    n = x.shape[1]
    w = torch.ones(n, dtype=torch.float64) if w is None else w.double()
    b = torch.zeros(n, dtype=torch.float64) if b is None else b.double()
    mean = x.mean(1, keepdim=True)
    d = x - mean
    rstd = ((d * d).mean(1, keepdim=True) + eps) ** -0.5
    y = d * rstd * w + b
    c = steps(n) * U
    mag = x.abs().mean(1, keepdim=True)
    # an error of the mean moves the variance by its square only
    moved = (c * mag * rstd).square()
    err = w.abs() * rstd * (c * mag + d.abs() * (c + 4 * U + moved)) + 2 * U * (y.abs() + b.abs())
    return y, mean[:, 0], rstd[:, 0], err


def within(name, got, want, tol):
    got, want = got.double().cpu(), want.double()
    bad = ~((got - want).abs() <= tol)
    assert not bad.any(), (f"{name}: {int(bad.sum())} of {bad.numel()} outside, first at "
                           f"{tuple(bad.nonzero()[0].tolist())}: {got[bad][0]} against {want[bad][0]}")


def check_forward(x, w, b, y=True, fmt=None, eps=EPS):
    rows, cols = x.shape
    print(f"[layer_norm] {rows} x {cols} {x.dtype} fmt={fmt}", flush=True)
    dev = [None if t is None else t.to(DEV) for t in (x, w, b)]
    r = binding.fp8_layer_norm(*dev, eps, y=y, fmt=fmt, stats=True)
    torch.cuda.synchronize()
    ry, rm, rr, err = reference(x, w, b, eps)
    c = steps(cols) * U
    mag = x.double().abs().mean(1)
    within("mean", r.mean, rm, c * mag)
    within("rstd", r.rstd, rr, rr * (c + 4 * U + (c * mag * rr).square()))
    half = torch.finfo(x.dtype).eps / 2
    if y:
        assert r.y.dtype == x.dtype
        within("y", r.y, ry, err + half * (ry.abs() + err))
    else:
        assert r.y is None
    if fmt is None:
        assert r.q is None and r.scale is None
        return r
    amax = ry.abs().amax(1)
    serr = err.amax(1) / QMAX[fmt] + 2 * U * amax / QMAX[fmt]
    within("scale", r.scale, amax / QMAX[fmt], serr)
    rel, least = HALF_STEP[fmt]
    s = r.scale.double().cpu()[:, None]
    value = r.q.view(F8[fmt]).double().cpu() * s
    within("q", value, ry, torch.maximum(rel * ry.abs(), least * s) + 2 * err)
    return r


SHAPES = [(1, 1), (3, 7), (5, 8), (2, 15), (7, 64), (600, 96), (4, 1000), (33, 1024), (4, 1031), (17, 1025),
          (1, 8192), (3, 8200), (6, 4097), (300, 2047), (2, 16384), (2, 16391), (3, 16392), (2, 20000), (1, 40003),
          (5000, 72)]


@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("rows,cols", SHAPES)
def test_forward(rows, cols, dtype):
    check_forward(*make(rows, cols, dtype, rows * 7 + cols))


@pytest.mark.parametrize("fmt", ["e4m3fn", "e5m2"])
@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("y", [True, False])
@pytest.mark.parametrize("rows,cols", [(1, 16), (9, 48), (600, 1024), (5, 1040), (300, 8192), (2, 16384), (3, 16400),
                                       (1, 65536)])
def test_forward_with_codes(rows, cols, y, dtype, fmt):
    check_forward(*make(rows, cols, dtype, rows + cols), y=y, fmt=fmt)


@pytest.mark.parametrize("fmt", ["e4m3fn", "e5m2"])
@pytest.mark.parametrize("rows,cols", [(40, 512), (30, 4096), (4, 16400)])
def test_codes_are_the_quantised_fp32_result_bit_for_bit(rows, cols, fmt):
    # with fp32 x, y is the very value the codes are made from
    x, w, b = make(rows, cols, FP32, 5)
    r = binding.fp8_layer_norm(x.to(DEV), w.to(DEV), b.to(DEV), EPS, fmt=fmt)
    y = r.y.cpu()
    scale = y.abs().amax(1) / torch.tensor(QMAX[fmt])
    assert torch.equal(r.scale.cpu(), scale)
    q = (y / scale[:, None]).clamp(-QMAX[fmt], QMAX[fmt]).to(F8[fmt]).view(torch.uint8)
    assert torch.equal(r.q.cpu(), q)


@pytest.mark.parametrize("params", [BF16, None])
def test_parameters_in_bf16_or_absent(params):
    for rows, cols in ((5, 1000), (4, 4096), (2, 20000)):
        x, w, b = make(rows, cols, BF16, 3, params or FP32)
        if params is None:
            check_forward(x, None, None)
            check_forward(x, w, None)
            check_forward(x, None, b)
            check_backward(x, None, seed=2)
        else:
            check_forward(x, w, b)
            check_backward(x, w, seed=2)


@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("cols", [8, 1000, 8192, 20000])
def test_rows_with_a_far_mean_and_equal_elements(cols, dtype):
    x, w, b = make(6, cols, FP32, 1)
    x[0] = x[0] * 0.25 + 1000
    x[1] = 3.3
    x[2] = 0
    x[3] = x[3] * 1e-20
    x[4] = x[4] * 1e12
    x[5] = 0
    x[5, -1] = 50
    check_forward(x.to(dtype), w, b)
    check_forward(x.to(dtype), w, torch.zeros(cols))     # rows 1 and 2: y near or at 0
    if cols % 16 == 0:
        check_forward(x.to(dtype), w, b, fmt="e4m3fn")
        check_forward(x.to(dtype), w, torch.zeros(cols), fmt="e4m3fn")


def test_zero_rows_and_eps():
    x = torch.zeros(3, 64, dtype=BF16, device=DEV)
    r = binding.fp8_layer_norm(x, eps=0.0, fmt="e4m3fn", stats=True)    # 0 / 0: no variance and no eps
    assert r.y.isnan().all() or (r.y == 0).all()
    r = binding.fp8_layer_norm(x, eps=1e-5, fmt="e4m3fn", stats=True)
    assert (r.y == 0).all() and (r.scale == 0).all() and (r.q == 0).all() and (r.mean == 0).all()
    e = binding.fp8_layer_norm(x[:0], fmt="e4m3fn", stats=True)
    assert e.y.shape == (0, 64) and e.q.shape == (0, 64) and e.scale.numel() == 0 and e.mean.numel() == 0


@pytest.mark.parametrize("value", [float("nan"), float("inf"), float("-inf")])
@pytest.mark.parametrize("cols", [64, 1008, 8192, 20000])
def test_a_row_that_is_not_finite_shows_it_and_leaves_the_others(cols, value):
    x, w, b = make(5, cols, BF16, 11)
    clean = binding.fp8_layer_norm(x.to(DEV), w.to(DEV), b.to(DEV), fmt="e4m3fn", stats=True)
    x[2, cols // 2] = value
    r = binding.fp8_layer_norm(x.to(DEV), w.to(DEV), b.to(DEV), fmt="e4m3fn", stats=True)
    assert r.y[2].isnan().all() and r.scale[2].isnan() and r.rstd[2].isnan()
    assert (r.q[2] & 0x7F == 0x7F).all()
    keep = [0, 1, 3, 4]
    for got, want in zip(r, clean):
        assert torch.equal(got[keep], want[keep])


def backward_reference(dy, x, mean, rstd, w, res):
    dy, x = dy.double(), x.double()
    mean, rstd = mean.double()[:, None], rstd.double()[:, None]
    w = torch.ones(x.shape[1], dtype=torch.float64) if w is None else w.double()
    xh = (x - mean) * rstd
    g = dy * w
    c1, c2 = g.mean(1, keepdim=True), (g * xh).mean(1, keepdim=True)
    dx = rstd * (g - c1 - xh * c2) + (0 if res is None else res.double())
    c = steps(x.shape[1]) * U
    err = c * rstd * (g.abs() + g.abs().mean(1, keepdim=True) + 2 * xh.abs() * (g * xh).abs().mean(1, keepdim=True))
    err = err + 2 * U * dx.abs() + (0 if res is None else U * res.double().abs())
    k = (x.shape[0] / 64 + 72) * U     # (64 workgroups share the rows of long ones)
    return (dx, (dy * xh).sum(0), dy.sum(0)), (err, k * (dy * xh).abs().sum(0), k * dy.abs().sum(0))


def check_backward(x, w, seed, residual=False, workspace=None):
    rows, cols = x.shape
    print(f"[layer_norm_backward] {rows} x {cols} {x.dtype} residual={residual}", flush=True)
    g = torch.Generator().manual_seed(seed)
    dy = (0.1 * torch.randn(rows, cols, generator=g)).to(x.dtype)
    res = torch.randn(rows, cols, generator=g).to(x.dtype) if residual else None
    _, mean, rstd, _ = reference(x, w, None)
    mean, rstd = mean.float(), rstd.float()
    dev = [None if t is None else t.to(DEV) for t in (dy, x, mean, rstd, w)]
    got = binding.fp8_layer_norm_backward(*dev, residual_grad=None if res is None else res.to(DEV),
                                          workspace=workspace)
    torch.cuda.synchronize()
    want, err = backward_reference(dy, x, mean, rstd, w, res)
    half = torch.finfo(x.dtype).eps / 2
    within("dx", got[0], want[0], err[0] + half * (want[0].abs() + err[0]))
    within("dw", got[1], want[1], err[1])
    within("db", got[2], want[2], err[2])
    return got


@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("residual", [False, True])
@pytest.mark.parametrize("rows,cols", SHAPES + [(257, 1000), (1025, 520), (4100, 1), (700, 3000), (513, 8192)])
def test_backward(rows, cols, residual, dtype):
    x, w, _ = make(rows, cols, dtype, rows + 3 * cols)
    check_backward(x, w, 5, residual)


def test_backward_without_rows_gives_zero_parameter_gradients():
    for cols in (5, 1000, 20000):
        x = torch.zeros(0, cols, dtype=BF16, device=DEV)
        s = torch.zeros(0, device=DEV)
        dx, dw, db = binding.fp8_layer_norm_backward(x, x, s, s, torch.ones(cols, device=DEV))
        assert dx.shape == (0, cols) and dw.shape == db.shape == (cols,)
        assert (dw == 0).all() and (db == 0).all()


def test_gradient_against_differences():
    # d/dt of sum(dy * y(x + t vx, w + t vw, b + t vb)) at t = 0, by central differences in 64 bits
    x, w, b = make(9, 130, FP32, 4)
    g = torch.Generator().manual_seed(9)
    dy = torch.randn(9, 130, generator=g)
    vx, vw, vb = (torch.randn(s, generator=g, dtype=torch.float64) for s in ((9, 130), (130,), (130,)))
    _, mean, rstd, _ = reference(x, w, b)
    dx, dw, db = binding.fp8_layer_norm_backward(*(t.to(DEV) for t in (dy, x, mean.float(), rstd.float(), w)))
    h = 1e-5

    def loss(t):
        return (dy.double() * reference(x.double() + t * vx, w.double() + t * vw, b.double() + t * vb)[0]).sum()

    want = (loss(h) - loss(-h)) / (2 * h)
    parts = [dx.double().cpu() * vx, dw.double().cpu() * vw, db.double().cpu() * vb]
    got = sum(p.sum() for p in parts)
    size = sum(p.abs().sum() for p in parts)
    # fp32 errors (2 * 33 u of each term, and of terms that cancel inside dx), and h^2 of the differences
    assert (got - want).abs() <= size * 1e-4, (got, want, size)


@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("cols", [72, 1000, 8192, 20000])
def test_tensors_that_start_off_the_vector_boundary(cols, dtype):
    rows = 7
    x, w, b = make(rows, cols, dtype, 21)

    def shifted(t, by=1):
        store = torch.empty(t.numel() + 16, dtype=t.dtype, device=DEV)
        view = store[by:by + t.numel()].view(t.shape)
        view.copy_(t)
        return view

    ref = binding.fp8_layer_norm(x.to(DEV), w.to(DEV), b.to(DEV), stats=True)
    xs, ws, bs = shifted(x), shifted(w), shifted(b, 3)
    out = shifted(torch.zeros(rows, cols, dtype=dtype), 5)
    got = binding.fp8_layer_norm(xs, ws, bs, y=out, stats=True)
    assert got.y is out
    for a, c in zip(got, ref):
        assert a is c or torch.equal(a, c)
    want = binding.fp8_layer_norm_backward(x.to(DEV), x.to(DEV), ref.mean, ref.rstd, w.to(DEV),
                                           residual_grad=x.to(DEV))
    have = binding.fp8_layer_norm_backward(xs, shifted(x, 3), ref.mean, ref.rstd, ws, residual_grad=shifted(x, 7),
                                           dx=shifted(torch.zeros(rows, cols, dtype=dtype), 1))
    for a, c in zip(have, want):
        assert torch.equal(a, c)


@pytest.mark.parametrize("cols", [72, 1000, 8192, 20000])
def test_nothing_is_written_outside_the_outputs(cols):
    rows = 5
    x, w, b = make(rows, cols, BF16, 8)
    guard = torch.full((rows * cols + 128,), 7.0, dtype=BF16, device=DEV)
    y = guard[64:64 + rows * cols].view(rows, cols)
    binding.fp8_layer_norm(x.to(DEV), w.to(DEV), b.to(DEV), y=y)
    assert (guard[:64] == 7).all() and (guard[64 + rows * cols:] == 7).all()
    need = int(binding.lib().fp8_layer_norm_backward_workspace_size(rows, cols))
    ws = torch.full((need + 512,), 3, dtype=torch.uint8, device=DEV)
    _, mean, rstd, _ = reference(x, w, b)
    guard.fill_(7.0)
    args = [t.to(DEV) for t in (x, x, mean.float(), rstd.float(), w)]
    got = binding.fp8_layer_norm_backward(*args, dx=y, workspace=ws[:need])
    assert (ws[need:] == 3).all()
    assert (guard[:64] == 7).all() and (guard[64 + rows * cols:] == 7).all()
    for a, c in zip(got, binding.fp8_layer_norm_backward(*args)):     # another workspace, with other contents
        assert torch.equal(a, c)
    with pytest.raises(ValueError):
        binding.fp8_layer_norm_backward(*args, workspace=ws[:need - 256])


def test_equal_calls_give_equal_bits():
    x, w, _ = make(2000, 3000, BF16, 2)
    _, mean, rstd, _ = reference(x, w, None)
    args = [t.to(DEV) for t in (x, x, mean.float(), rstd.float(), w)]
    first = binding.fp8_layer_norm_backward(*args)
    for _ in range(4):
        for a, c in zip(first, binding.fp8_layer_norm_backward(*args)):
            assert torch.equal(a, c)


def test_on_another_stream_and_in_a_graph():
    x, w, b = (t.to(DEV) for t in make(300, 2000, BF16, 2))
    y = torch.empty_like(x)
    q = torch.empty(300, 2000, dtype=torch.uint8, device=DEV)
    s = torch.empty(300, device=DEV)
    dx = torch.empty_like(x)
    outs = {}

    def calls():
        r = binding.fp8_layer_norm(x, w, b, y=y, fmt="e4m3fn", q=q, scale=s, stats=True)
        outs["g"] = binding.fp8_layer_norm_backward(y, x, r.mean, r.rstd, w, residual_grad=y, dx=dx)

    calls()
    torch.cuda.synchronize()
    want = [t.clone() for t in (y, q, s, *outs["g"])]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        calls()
    torch.cuda.synchronize()
    for a, c in zip((y, q, s, *outs["g"]), want):
        assert torch.equal(a, c)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        calls()
    held = (y, q, s, *outs["g"])
    for rep in range(4):
        for t in held:
            t.zero_()
        junk = torch.randn(256, 256, device=DEV) @ torch.randn(256, 256, device=DEV)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for a, c in zip(held, want):
            assert torch.equal(a, c), f"replay {rep} differs"
        del junk


def test_refusals_with_gpu_tensors():
    x = torch.zeros(4, 64, dtype=BF16, device=DEV)
    w = torch.ones(64, device=DEV)
    s = torch.zeros(4, device=DEV)
    f = binding.fp8_layer_norm
    g = binding.fp8_layer_norm_backward
    for call in (lambda: f(x, w[:32]), lambda: f(x, w.double()), lambda: f(x, w, w.bfloat16()),
                 lambda: f(x, w.cpu()), lambda: f(x, eps=-1.0), lambda: f(x, eps=float("nan")),
                 lambda: f(x, fmt="e3m4"), lambda: f(x, y=False), lambda: f(x, q=x),
                 lambda: f(x, fmt="e4m3fn", q=x), lambda: f(x, fmt="e4m3fn", scale=s[:2]),
                 lambda: f(x[:, :40].contiguous(), fmt="e4m3fn"), lambda: f(x[:, ::2]),
                 lambda: f(x, y=x.float()), lambda: f(x[:, :0]),
                 lambda: g(x.float(), x, s, s), lambda: g(x, x, s[:2], s), lambda: g(x, x, s, s.double()),
                 lambda: g(x, x, s, s, w[:8]), lambda: g(x, x, s, s, residual_grad=x[:2]),
                 lambda: g(x, x, s, s, dx=x.float()), lambda: g(x, x, s.cpu(), s)):
        with pytest.raises(ValueError):
            call()


@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("cols", [8, 72, 1000, 4104, 8208])
@pytest.mark.parametrize("rows", [63, 65, 97, 255, 260, 300, 769])
def test_backward_on_both_sides_of_the_row_counts_where_its_launches_change(rows, cols, dtype):
    x, w, _ = make(rows, cols, dtype, rows + cols)
    check_backward(x, w, 6, residual=True)
