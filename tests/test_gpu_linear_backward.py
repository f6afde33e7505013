"""The linear layer's gradient (fp8_linear_backward) on the GPU against 64 bits.

Tolerances.  The reference quantises dz and x, computed in 64 bits, by the same
definition.  The library's slope is off by at most 4e-7 max(1, |z|) (the fit of
the normal distribution function 1.5e-7, z^2 rounded in an exponent, a few fp32
roundings; the slope has roots, so this is no relative error), so a code may be
the neighbouring one where the quotient is that close to a tie: the codes of dz - d
and dz + d bound it.  The products are the scaled multiply's, held to its parity bound of 1e-3 of
the sum of magnitudes, except with whole numbers whose codes, scales and sums
are exact.  Outputs are rounded once (torch.finfo(bf16).eps / 2).  dbias adds at
most M / 256 + 32 fp32 numbers in a row per partial sum.
"""
import pytest
import torch

from precision_linear_amd import binding

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF16 = torch.bfloat16
HALF = torch.finfo(BF16).eps / 2
ACTS = ("none", "relu", "gelu", "gelu_tanh", "silu")
E5M2 = (2, -14, 57344.0)
E4M3 = (3, -6, 448.0)


def slope64(z, act):
    if act == "relu":
        return (z > 0).double()
    if act == "gelu":
        return 0.5 * torch.special.erfc(-z / 2 ** 0.5) + z * torch.exp(-z * z / 2) / (2 * torch.pi) ** 0.5
    if act == "gelu_tanh":
        a = (2 / torch.pi) ** 0.5
        p = torch.sigmoid(2 * a * (z + 0.044715 * z ** 3))
        return p + z * p * (1 - p) * 2 * a * (1 + 3 * 0.044715 * z * z)
    if act == "silu":
        p = torch.sigmoid(z)
        return p + z * p * (1 - p)
    return torch.ones_like(z)


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


def quantised(v, axis, fmt, err=None):
    """(values the codes stand for, how far a code of a value within `err` of v may be from them)."""
    mant, least, qmax = fmt
    s = (v.abs().amax(axis, keepdim=True) / qmax).float().double()

    def code(t):
        t = t.clamp(-qmax, qmax)
        _, e = torch.frexp(t)
        step = torch.ldexp(torch.ones_like(t), (e - 1).clamp(min=least) - mant)
        return torch.round(t / step) * step

    q = torch.where(s > 0, v / s, torch.zeros_like(v)).float().double()
    mid = code(q)
    if err is None:
        return mid * s, torch.zeros_like(v)
    # the scale moves with the largest value, by its relative error
    d = torch.where(s > 0, err / s, torch.zeros_like(v))
    d = d + q.abs() * (d.amax(axis, keepdim=True) / qmax + 2.0 ** -22)
    lo, hi = code(q - d), code(q + d)
    return mid * s, torch.maximum((lo - mid).abs(), (hi - mid).abs()) * s


def make(M, N, K, seed, scale=1e-3):
    g = torch.Generator().manual_seed(seed)
    dy = (scale * torch.exp(0.5 * torch.randn(M, 1, generator=g)) * torch.randn(M, N, generator=g)).to(BF16)
    z = (1.5 * torch.randn(M, N, generator=g)).to(BF16)
    x = torch.randn(M, K, generator=g).to(BF16)
    wt = (2 * torch.randn(K, N, generator=g)).to(torch.float8_e4m3fn)
    sw = (torch.rand(K, generator=g) + 0.5) * 0.02
    return dy, x, wt, sw, z


def make_whole(M, N, K, seed):
    """Whole numbers of at most 7 in size, 7 in every row and column: every scale is a power of 2."""
    g = torch.Generator().manual_seed(seed)
    assert 49 * max(M, N) < 2 ** 24
    dy = torch.randint(-7, 8, (M, N), generator=g).to(BF16)
    x = torch.randint(-7, 8, (M, K), generator=g).to(BF16)
    i = torch.arange(max(M, N, K))
    dy[i[:max(M, N)] % M, i[:max(M, N)] % N] = 7
    x[i[:max(M, K)] % M, i[:max(M, K)] % K] = 7
    wt = torch.randint(-7, 8, (K, N), generator=g).float().to(torch.float8_e4m3fn)
    return dy, x, wt, torch.full((K,), 0.5), torch.randn(M, N, generator=g).to(BF16)


def reference(dy, x, wt, sw, z, act, whole):
    dz = dy.double() * slope64(z.double(), act)
    z64 = z.double()
    each = dy.double().abs() * (4e-7 * z64.abs().clamp(min=1) + 2.0 ** -23) + 2.0 ** -23 * dz.abs()
    err = None if act in ("none", "relu") else each
    w = wt.double() * sw.double()[:, None]
    rows, rdev = quantised(dz, 1, E5M2, err)
    cols, cdev = quantised(dz, 0, E5M2, err)
    xq, _ = quantised(x.double(), 0, E4M3)
    mm = 0.0 if whole else 1e-3
    rel = 0.0 if whole else 2e-5                       # the scales (of largest values, whose slopes are not near a root)
    dx, dw = rows @ w.t(), cols.t() @ xq
    dxe = rdev @ w.abs().t() + (mm + rel) * (rows.abs() @ w.abs().t())
    dwe = cdev.t() @ xq.abs() + (mm + rel) * (cols.abs().t() @ xq.abs())
    M = dy.shape[0]
    dbe = each.sum(0) + (M / 256 + 32) * 2.0 ** -24 * dz.abs().sum(0)
    return (dx, dxe), (dw, dwe), (dz.sum(0), dbe)


def within(name, got, want, tol):
    got = got.double().cpu()
    bad = ~((got - want).abs() <= tol)
    assert not bad.any(), (f"{name}: {int(bad.sum())} of {bad.numel()} outside, first at "
                           f"{tuple(bad.nonzero()[0].tolist())}: {got[bad][0]} against {want[bad][0]}")


def check(args, act, whole=False, **kw):
    dy, x, wt, sw, z = args
    print(f"[linear_backward] {dy.shape[0]} x {dy.shape[1]} x {x.shape[1]} act={act} {list(kw)}", flush=True)
    got = binding.fp8_linear_backward(*(t.to(DEV) for t in args), activation=act, **kw)
    torch.cuda.synchronize()
    ref = reference(dy, x, wt, sw, z, act, whole)
    for name, g, (want, err), half in zip(("dx", "dw", "dbias"), got, ref, (HALF, HALF, 0.0)):
        within(name, g, want, err + half * (want.abs() + err))
    return got


SHAPES = [(1, 16, 16), (1, 2048, 512), (3, 48, 32), (15, 128, 144), (16, 160, 16), (129, 272, 400), (500, 2048, 2048),
          (257, 1040, 128), (1000, 128, 1296), (4097, 64, 80), (64, 4096, 1024)]


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("M,N,K", SHAPES)
def test_against_64_bits(M, N, K, act):
    check(make(M, N, K, M + N + K), act)


@pytest.mark.parametrize("act", ["none", "relu"])
@pytest.mark.parametrize("M,N,K", SHAPES)
def test_whole_numbers_are_exact(M, N, K, act):
    args = make_whole(M, N, K, M * 3 + N + K)
    if act == "relu":        # keep the sevens
        dy, x, wt, sw, z = args
        args = (dy, x, wt, sw, torch.where(dy == 7, z.abs() + 1, z))
    check(args, act, whole=True)


def test_every_part_alone_gives_the_same():
    args = [t.to(DEV) for t in make(300, 272, 144, 4)]
    dy, x, wt, sw, z = args
    f = binding.fp8_linear_backward
    dx, dw, db = f(*args, activation="gelu")
    for want_dx, want_dw, want_db in ((1, 0, 0), (0, 1, 0), (0, 0, 1), (1, 1, 0), (1, 0, 1), (0, 1, 1)):
        got = f(dy, x if want_dw else None, wt if want_dx else None, sw if want_dx else None, z, activation="gelu",
                dx=bool(want_dx), dw=bool(want_dw), dbias=bool(want_db))
        for have, want, asked in zip(got, (dx, dw, db), (want_dx, want_dw, want_db)):
            assert (have is None) if not asked else torch.equal(have, want)
    bx, bw = torch.empty_like(dx), torch.empty_like(dw)
    got = f(*args, activation="gelu", dx=bx, dw=bw)
    assert got[0] is bx and got[1] is bw and torch.equal(bx, dx) and torch.equal(bw, dw)
    # 'none' does without z
    a, b = f(dy, x, wt, sw, z, activation="none"), f(dy, x, wt, sw, activation="none")
    assert all(torch.equal(p, q) for p, q in zip(a, b))


def test_weights_in_e5m2_and_as_bytes():
    dy, x, wt, sw, z = make(70, 160, 48, 8)
    w5 = wt.float().to(torch.float8_e5m2)
    check((dy, x, w5, sw, z), "silu")
    args = [t.to(DEV) for t in (dy, x, w5, sw, z)]
    a = binding.fp8_linear_backward(*args, activation="silu")
    args[2] = args[2].view(torch.uint8)
    b = binding.fp8_linear_backward(*args, activation="silu", wt_format="e5m2")
    assert all(torch.equal(p, q) for p, q in zip(a, b))


@pytest.mark.parametrize("act", ACTS)
def test_slope_of_every_finite_bf16_value(act):
    # one row of ones: dbias is act'(z) itself; against the formula, and against differences of act
    v = torch.arange(65536, dtype=torch.int32).to(torch.int16).view(BF16)
    v = v[torch.isfinite(v.float())]
    n = v.numel() // 16 * 16
    for part in (v[:n], v[-n:]):
        z = part.reshape(1, -1)
        _, _, db = binding.fp8_linear_backward(torch.ones_like(z).to(DEV), None, None, None, z.to(DEV), activation=act,
                                               dx=False, dw=False)
        z64 = z[0].double()
        want = slope64(z64, act)
        want = torch.where(z64.abs() > 100, (z64 > 0).double() if act != "none" else torch.ones_like(z64), want)
        within("slope", db, want, 4e-7 * z64.abs().clamp(1, 16) + 2.0 ** -22)
        near = (z64.abs() < 20) & ((z64.abs() > 1e-3) | torch.tensor(act not in ("relu",)))
        h = 1e-5
        diff = (act64(z64 + h, act) - act64(z64 - h, act)) / (2 * h)
        # (h^2 of the differences, and 2^-53 |z| / h of their cancellation)
        within("differences", db[near.to(DEV)], diff[near], 4e-7 * z64[near].abs().clamp(1, 16) + 1e-8)


def test_values_that_are_not_finite_come_out():
    for act in ACTS:
        for bad in (float("nan"), float("inf")):
            dy, x, wt, sw, z = make(40, 64, 48, 2)
            clean = binding.fp8_linear_backward(*(t.to(DEV) for t in (dy, x, wt, sw, z)), activation=act)
            dy[3, 5], z[3, 5] = bad, 1.0
            dx, dw, db = binding.fp8_linear_backward(*(t.to(DEV) for t in (dy, x, wt, sw, z)), activation=act)
            assert not dx[3].isfinite().any() and not dw[5].isfinite().any() and not db[5].isfinite()
            keep_m, keep_n = torch.arange(40) != 3, torch.arange(64) != 5
            assert torch.equal(dx[keep_m.to(DEV)], clean[0][keep_m.to(DEV)])
            assert torch.equal(dw[keep_n.to(DEV)], clean[1][keep_n.to(DEV)])
            assert torch.equal(db[keep_n.to(DEV)], clean[2][keep_n.to(DEV)])
            x[7, 9] = bad
            _, dw, _ = binding.fp8_linear_backward(*(t.to(DEV) for t in (dy, x, wt, sw, z)), activation=act)
            assert not dw[:, 9].isfinite().any()


def test_rows_and_columns_of_zeros_and_of_tiny_values():
    dy, x, wt, sw, z = make(50, 64, 48, 6)
    dy[4] = 0
    dy[:, 9] = 0
    x[:, 11] = 0
    dx, dw, db = check((dy, x, wt, sw, z), "gelu")
    assert (dx[4] == 0).all() and (dw[9] == 0).all() and (dw[:, 11] == 0).all() and db[9] == 0
    for scale in (1e-30, 1e25):
        check(make(50, 64, 48, 6, scale), "relu")
    dy, x, wt, sw, z = make(50, 64, 48, 6, 1e-37)       # below qmax * 2^-126: codes 0, not infinities
    dx, dw, db = binding.fp8_linear_backward(*(t.to(DEV) for t in (dy, x, wt, sw, z)), activation="silu")
    assert (dx == 0).all() and (dw == 0).all() and db.isfinite().all()


def test_without_rows():
    dy = torch.zeros(0, 64, dtype=BF16, device=DEV)
    x = torch.zeros(0, 48, dtype=BF16, device=DEV)
    _, _, wt, sw, _ = make(1, 64, 48, 6)
    dx, dw, db = binding.fp8_linear_backward(dy, x, wt.to(DEV), sw.to(DEV), dy, activation="gelu")
    assert dx.shape == (0, 48) and dw.shape == (64, 48) and (dw == 0).all() and (db == 0).all()


def test_one_workspace_for_calls_of_any_shape():
    calls = [([t.to(DEV) for t in make(m, n, k, m)], act) for m, n, k, act in
             ((500, 2048, 2048, "gelu"), (17, 64, 4096, "relu"), (1000, 128, 1296, "none"), (64, 4096, 1024, "silu"))]
    need = max(int(binding.lib().fp8_linear_backward_workspace_size(a[0].shape[0], a[0].shape[1], a[1].shape[1], 1, 1))
               for a, _ in calls)
    ws = torch.zeros(need + 512, dtype=torch.uint8, device=DEV)
    ws[need:] = 9
    want = [binding.fp8_linear_backward(*a, activation=act) for a, act in calls]
    for rep in range(3):
        for (a, act), w in zip(calls, want):
            got = binding.fp8_linear_backward(*a, activation=act, workspace=ws[:need])
            assert all(torch.equal(p, q) for p, q in zip(got, w))
    assert (ws[need:] == 9).all() and (ws[:256 << 10] == 0).all()
    a, act = calls[0]
    with pytest.raises(ValueError):
        binding.fp8_linear_backward(*a, activation=act, workspace=ws[:1 << 20])


def test_tensors_off_the_vector_boundary_and_guards():
    args = make(130, 160, 144, 3)
    dy, x, wt, sw, z = [t.to(DEV) for t in args]
    want = binding.fp8_linear_backward(dy, x, wt, sw, z, activation="gelu_tanh")

    def shifted(t, by):
        store = torch.full((t.numel() + 64,), 5.0, dtype=t.dtype, device=DEV)
        view = store[by:by + t.numel()].view(t.shape)
        view.copy_(t)
        return view, store

    (a, _), (b, _), (c, _) = shifted(dy, 1), shifted(x, 3), shifted(z, 5)
    (dx, xs), (dw, ws) = shifted(want[0] * 0, 7), shifted(want[1] * 0, 2)
    got = binding.fp8_linear_backward(a, b, wt, sw, c, activation="gelu_tanh", dx=dx, dw=dw)
    assert all(torch.equal(p, q) for p, q in zip(got, want))
    for store, by, t in ((xs, 7, dx), (ws, 2, dw)):
        assert (store[:by] == 5).all() and (store[by + t.numel():] == 5).all()


def test_on_another_stream_and_in_a_graph():
    args = [t.to(DEV) for t in make(500, 1024, 768, 5)]
    dx = torch.empty(500, 768, dtype=BF16, device=DEV)
    dw = torch.empty(1024, 768, dtype=BF16, device=DEV)
    out = {}

    def calls():
        out["db"] = binding.fp8_linear_backward(*args, activation="gelu", dx=dx, dw=dw)[2]

    calls()
    torch.cuda.synchronize()
    want = [t.clone() for t in (dx, dw, out["db"])]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        calls()
    torch.cuda.synchronize()
    assert all(torch.equal(p, q) for p, q in zip((dx, dw, out["db"]), want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        calls()
    held = (dx, dw, out["db"])
    for rep in range(4):
        for t in held:
            t.zero_()
        junk = torch.randn(256, 256, device=DEV) @ torch.randn(256, 256, device=DEV)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(held, want)), f"replay {rep} differs"
        del junk


def test_refusals_with_gpu_tensors():
    dy, x, wt, sw, z = [t.to(DEV) for t in make(32, 64, 48, 1)]
    f = binding.fp8_linear_backward
    for args, kw in (((dy, x, wt, sw, z), dict(activation="swish")), ((dy.float(), x, wt, sw, z), {}),
                     ((dy, x[:8], wt, sw, z), {}), ((dy, x, wt[:16], sw, z), {}), ((dy, x, wt, sw[:16], z), {}),
                     ((dy, x, wt, sw, z[:8]), dict(activation="relu")), ((dy, x, wt, sw, None), dict(activation="relu")),
                     ((dy, None, wt, sw, z), {}), ((dy, x, None, sw, z), {}), ((dy, x, wt, None, z), {}),
                     ((dy, x, wt.t().contiguous(), sw, z), {}), ((dy, x.cpu(), wt, sw, z), {}),
                     ((dy, x, wt, sw.double(), z), {}), ((dy, x, wt, sw, z), dict(dx=dy)),
                     ((dy, x, wt, sw, z), dict(dw=dy)), ((dy, x, wt, sw, z), dict(dx=False, dw=False, dbias=False)),
                     ((dy, x, wt.view(torch.uint8), sw, z), dict(wt_format="fp4")),
                     ((dy[:, :40].contiguous(), x, wt[:, :40].contiguous(), sw, z[:, :40].contiguous()), {})):
        with pytest.raises(ValueError):
            f(*args, **kw)
