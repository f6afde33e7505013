"""The gradient of the FP8 linear layer's softmax cross entropy on the GPU.

Tolerances.  The reference quantises the logits' gradient and x by the same
definition in 64 bits.  The exponent of a code's value, z log2(e) + f with f = log2(57344 /
h) - lse log2(e), is off by at most the logit's dz (test_gpu_cross_entropy) times
log2(e), and by 4 u (u = 2^-24) of the magnitudes of its terms; 2^x by 2 u of itself; h
= -expm1(-loss) and its logarithm by 8 u.  So a code may be the neighbouring one where the
value is that close to a tie: the codes of the value's two bounds are the two ends.  x r
is rounded once, and r itself three times, so is x's code.  The products are the scaled
multiply's, held to its parity bound of 1e-3 of the sum of magnitudes; outputs are
rounded once (torch.finfo(bf16).eps / 2).
"""
import math
import threading

import pytest
import torch

from precision_linear_amd import binding
from test_gpu_cross_entropy import DEV, FP8, U, check, logits64
from test_gpu_cross_entropy import make as make_any

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16
HALF = torch.finfo(BF16).eps / 2
E5M2 = (2, -14, 57344.0)
E4M3 = (3, -6, 448.0)
LOG2E = math.log2(math.e)


def make(*args, **kw):
    """Operands whose logits the products give exactly (test_gpu_cross_entropy)."""
    return make_any(*args, whole=True, **kw)


def code(t, fmt):
    mant, least, qmax = fmt
    t = t.clamp(-qmax, qmax)
    _, e = torch.frexp(t)
    # (powers of two from a table: torch's ldexp on the GPU is off in the last bits)
    powers = torch.tensor([2.0 ** i for i in range(-32, 32)], dtype=torch.float64, device=t.device)
    step = powers[((e - 1).clamp(min=least) - mant + 32).long()]
    return torch.round(t / step) * step


def gradient64(dloss, a, b, sa, sb, t, loss, lse, x, wt, swt, ignore=-100):
    """((dx, bound), (dw, bound))"""
    z, dz = logits64(a, b, sa, sb)
    M, V = z.shape
    kept = t != ignore
    l, e = loss.double(), lse.double()[:, None]
    h = torch.where(kept & (l > 0), -torch.expm1(-l), 0.0)
    f = torch.where(h > 0, torch.log2(57344 / h), -math.inf)[:, None]
    err = LOG2E * dz + 4 * U * (z.abs() * LOG2E + e.abs() * LOG2E + torch.where(h > 0, f[:, 0].abs(), 0.0)[:, None]) + 12 * U
    y = (z - e) * LOG2E + f
    q = code(torch.exp2(y), E5M2)
    dq = torch.maximum(q - code(torch.exp2(y - err), E5M2), code(torch.exp2(y + err), E5M2) - q)
    rows = torch.arange(M, device=DEV)[kept]
    q[rows, t[kept]] = -57344.0 * (h[kept] > 0).double()
    dq[rows, t[kept]] = 0
    r = dloss.double().expand(M) * h
    got = []
    wide = wt[:, :V].double()
    s = (r / 57344)[:, None].abs() * swt.double()[None, :]
    dx = torch.mm(q, wide.t()) * (r / 57344)[:, None] * swt.double()[None, :]
    tol = (torch.mm(dq, wide.abs().t()) + 1e-3 * torch.mm(q.abs(), wide.abs().t())) * s + 8 * U * dx.abs()
    got.append((dx, tol + HALF * (dx.abs() + tol)))
    xr = torch.where(r[:, None] == 0, 0.0, x.double() * r[:, None])
    sx = (xr.abs().amax(0) / 448)
    v = torch.where(sx > 0, xr / sx, 0.0)
    c = code(v, E4M3)
    d = 16 * U * v.abs()
    dc = torch.maximum((c - code(v - d, E4M3)).abs(), (code(v + d, E4M3) - c).abs())
    dw = torch.mm(q.t(), c) * (sx / 57344)
    mag = q.abs().t()
    tol = (torch.mm(dq.t(), c.abs() + dc) + torch.mm(mag, dc) + 1e-3 * torch.mm(mag, c.abs())) * (sx / 57344) + 16 * U * dw.abs()
    got.append((dw, tol + HALF * (dw.abs() + tol)))
    return got


def more(t, seed=1, fw="e4m3fn", dloss=None):
    """x, wt with its scales and dloss for a forward problem's tensors."""
    a, b, sa, sb, target = t
    M, K, V = a.shape[0], a.shape[1], b.shape[0]
    g = torch.Generator(device=DEV).manual_seed(seed)
    x = (a.float() * (sa[:, None] if sa.numel() == M else sa)).to(BF16)
    wt = torch.zeros(K, (V + 15) // 16 * 16, device=DEV)
    wt[:, :V] = torch.randn(K, V, generator=g, device=DEV)
    swt = 2.0 ** (torch.rand(K, generator=g, device=DEV) - 6)
    if dloss is None:
        dloss = torch.randn(M, generator=g, device=DEV) / max(M, 1)
    return x, wt.to(FP8[fw]), swt, dloss


def run(t, extra, mode="rowwise", **kw):
    x, wt, swt, dloss = extra
    loss, lse = binding.fp8_linear_cross_entropy(*t, mode=mode)
    got = binding.fp8_linear_cross_entropy_backward(dloss, *t, loss, lse, x, wt, swt, mode=mode, **kw)
    return (dloss, *t, loss, lse, x, wt, swt), got


def close(got, want, what=""):
    for name, g, (w, tol) in zip(("dx", "dw"), got, want):
        if g is None:
            continue
        assert g.dtype == BF16 and g.shape == w.shape
        off = (g.double() - w).abs()
        assert (off <= tol + 1e-37).all(), (what, name, float((off / (tol + 1e-37)).max()))


SHAPES = [(1, 1, 16), (1, 2, 32), (1, 17, 16), (1, 4000, 2048), (2, 100, 48), (15, 255, 16), (16, 257, 512),
          (17, 113, 64), (33, 5000, 4096), (64, 4096, 128), (65, 33, 8192), (100, 513, 160), (129, 10007, 1024),
          (256, 256, 128), (257, 1008, 256), (511, 20255, 272), (1000, 6001, 2048), (2048, 8200, 384),
          (4099, 12289, 144), (40000, 300, 32)]


@pytest.mark.parametrize("M,V,K", SHAPES)
def test_gradient(M, V, K):
    for mode, ignore in (("rowwise", None), ("per_tensor", -100)):
        print(f"[cross entropy gradient] {M} x {V} x {K} {mode}", flush=True)
        t = make(M, V, K, mode, ignore=ignore, seed=1)
        args, got = run(t, more(t), mode)
        close(got, gradient64(*args), mode)


@pytest.mark.parametrize("M,V,K,fa", [(8192, 70000, 80, "e4m3fn"), (70000, 9001, 48, "e5m2"), (8000, 33601, 272, "e4m3fn")])
def test_pieces_of_the_vocabulary(M, V, K, fa):
    """The codes of these take more than the workspace's share."""
    print(f"[cross entropy gradient] {M} x {V} x {K} in pieces", flush=True)
    assert 2 * M * V > 512 << 20
    t = make(M, V, K, fa=fa, ignore=-100, seed=2)
    args, got = run(t, more(t, fw="e5m2" if fa == "e5m2" else "e4m3fn"))
    want = gradient64(*args)
    close(got, want)
    del want
    dx, none = binding.fp8_linear_cross_entropy_backward(*args, dw=False)
    assert none is None and torch.equal(dx, got[0])
    none, dw = binding.fp8_linear_cross_entropy_backward(*args, dx=False)
    assert none is None and torch.equal(dw, got[1])


@pytest.mark.parametrize("fa", ["e4m3fn", "e5m2"])
@pytest.mark.parametrize("fb", ["e4m3fn", "e5m2"])
@pytest.mark.parametrize("fw", ["e4m3fn", "e5m2"])
@pytest.mark.parametrize("M,V,K", [(70, 1001, 256), (1300, 9000, 256)])
def test_formats(fa, fb, fw, M, V, K):
    print(f"[cross entropy gradient] {M} x {V} x {K} {fa} {fb} {fw}", flush=True)
    t = make(M, V, K, fa=fa, fb=fb, seed=3)
    args, got = run(t, more(t, fw=fw))
    close(got, gradient64(*args))


@pytest.mark.parametrize("M", [255, 256, 257, 512, 513, 1023, 1024, 1025])
def test_rows_around_the_variants_of_their_codes(M):
    """Also with x's column scales below 2^-60, where quotients are divisions."""
    t = make(M, 300, 80, seed=27, ignore=-100)
    x, wt, swt, dloss = more(t)
    x[:, 5] = 0
    for size in (1.0, 2.0 ** -80):
        args, got = run(t, (x, wt, swt, dloss * size))
        close(got, gradient64(*args), size)
        assert (got[1][:, 5] == 0).all()


@pytest.mark.parametrize("M,V,K", [(60, 700, 64), (512, 4096, 512), (300, 10000, 512)])
def test_every_code(M, V, K):
    """With x the identity, column m of dw holds row m's codes times r[m] / 57344; the
    same comes back through dx where wt picks K entries of the vocabulary."""
    t = make(M, V, K, seed=4, ignore=-100)
    a, b, sa, sb, target = t
    _, wt, swt, dloss = more(t)
    dloss = dloss.abs() + 1e-4
    x = torch.zeros(M, K, dtype=BF16, device=DEV)
    x[torch.arange(M), torch.arange(M) % K] = 1
    live = torch.arange(M, device=DEV) < K
    target = torch.where(live, target, -100)
    picks = torch.randperm(V, device=DEV)[:K]
    wt = torch.zeros_like(wt.float())
    wt[torch.arange(K, device=DEV), picks] = 1
    swt = torch.ones_like(swt)
    args, (dx, dw) = run((a, b, sa, sb, target), (x, wt.to(torch.float8_e4m3fn), swt, dloss))
    loss, lse = args[6], args[7]
    z, dz = logits64(a, b, sa, sb)
    h = torch.where((target != -100), -torch.expm1(-loss.double()), 0.0)
    y = torch.exp(z - lse.double()[:, None]) / h[:, None] * 57344
    err = 1 + dz + 40 * U * (z.abs() + lse.double().abs()[:, None] + 20)
    lo, hi = code(y / err, E5M2), code(y * err, E5M2)
    r = dloss.double() * h
    hit = torch.zeros_like(y, dtype=torch.bool)
    rows = torch.arange(M, device=DEV)[target != -100]
    hit[rows, target[rows]] = True
    lo, hi = torch.where(hit, -57344.0, lo), torch.where(hit, -57344.0, hi)
    n = min(M, K)
    kept = (target[:n] != -100)
    # (back to a code: bf16 holds it within 2^-8, a code's neighbours are 2^-3 away)
    back = code(dw[:, :n].double().t()[kept] / (r[:n][kept] / 57344)[:, None], E5M2)
    ok = (back >= lo[:n][kept]) & (back <= hi[:n][kept])
    assert ok.all(), (back[~ok][:5], lo[:n][kept][~ok][:5], hi[:n][kept][~ok][:5])
    assert (dw[:, :n].t()[~kept] == 0).all()
    back = code(dx.double()[rows] / (r[rows] / 57344)[:, None], E5M2)
    assert ((back >= lo[rows][:, picks]) & (back <= hi[rows][:, picks])).all()
    assert (dx[target == -100] == 0).all()


@pytest.mark.parametrize("M,V,K", [(30, 3000, 512), (1000, 9000, 256)])
def test_gradient_of_any_operands(M, V, K):
    t = make_any(M, V, K, seed=1)
    args, got = run(t, more(t))
    close(got, gradient64(*args))


def test_against_differences():
    """dloss . loss is moved by a step of one logit's weight as the gradient says, within what
    the codes lose: 2^-3 of an element and the rounding of x."""
    M, V, K = 40, 300, 64
    a, b, sa, sb, t = make(M, V, K, seed=6)
    b2 = b.float() * sb[:, None]
    x = (a.float() * sa[:, None])
    wt = torch.zeros(K, 304, device=DEV)
    wt[:, :V] = b2.t()
    swt = wt.abs().amax(1) / 448
    wtq = (wt / swt[:, None]).to(torch.float8_e4m3fn)
    dloss = torch.rand(M, device=DEV) + 0.5
    args, (dx, dw) = run((a, b, sa, sb, t), (x.to(BF16), wtq, swt, dloss))

    def value(x, w):
        return (dloss.double() * torch.nn.functional.cross_entropy(x @ w.t(), t, reduction="none")).sum()

    xd, wd = x.double(), b2.double()
    g = torch.Generator(device=DEV).manual_seed(0)
    for _ in range(5):
        ux, uw = torch.randn(M, K, generator=g, device=DEV).double(), torch.randn(V, K, generator=g, device=DEV).double()
        eps = 1e-5
        by_x = (value(xd + eps * ux, wd) - value(xd - eps * ux, wd)) / (2 * eps)
        by_w = (value(xd, wd + eps * uw) - value(xd, wd - eps * uw)) / (2 * eps)
        p = torch.softmax(xd @ wd.t(), 1)
        p[torch.arange(M), t] -= 1
        p *= dloss.double()[:, None]
        # codes of dz: within 2^-3 of themselves; of x and W: within 2^-4; the outputs' bf16
        lost = 2.0 ** -3 + 2.0 ** -4 + 2.0 ** -8
        room_x = lost * ((p.abs() @ wd.abs()) * ux.abs()).sum()
        room_w = lost * ((p.abs().t() @ xd.abs()) * uw.abs()).sum()
        assert abs((dx.double() * ux).sum() - by_x) < room_x
        assert abs((dw.double() * uw).sum() - by_w) < room_w
        # ... and, the losses being independent, far less in a sum of thousands of them
        assert abs((dx.double() * ux).sum() - by_x) < 0.1 * room_x
        assert abs((dw.double() * uw).sum() - by_w) < 0.1 * room_w


@pytest.mark.parametrize("M,V", [(6, 100), (600, 9000)])
def test_rows_that_do_not_count(M, V):
    """Ignored rows hold NaN, rows with dloss 0 infinities: neither reaches an output."""
    t = make(M, V, 64, seed=9)
    x, wt, swt, dloss = more(t)
    a, b, sa, sb, target = t
    clean = run(t, (x, wt, swt, torch.where(torch.arange(M, device=DEV) < 2, 0.0, dloss)))
    target = target.clone()
    target[0] = -100
    dloss[1] = 0
    a.view(torch.uint8)[0] = 0x7f
    x[0], x[1] = math.nan, math.inf
    loss, lse = binding.fp8_linear_cross_entropy(a, b, sa, sb, target)
    assert lse[0].isnan() and loss[0] == 0
    dx, dw = binding.fp8_linear_cross_entropy_backward(dloss, a, b, sa, sb, target, loss, lse, x, wt, swt)
    assert (dx[:2] == 0).all() and torch.equal(dx[2:], clean[1][0][2:]) and torch.equal(dw, clean[1][1])
    none = torch.full_like(target, -100)
    dx, dw = binding.fp8_linear_cross_entropy_backward(dloss, a, b, sa, sb, none, loss, lse, x, wt, swt)
    assert (dx == 0).all() and (dw == 0).all()


@pytest.mark.parametrize("path", ["short", "whole"])
@pytest.mark.parametrize("M,V", [(1, 20), (6, 100), (600, 9000)])
def test_another_ignored_index(M, V, path, monkeypatch):
    """Entries of the vocabulary, whose rows have a loss of 0 and an lse like any other, and numbers outside it."""
    if path == "whole":
        monkeypatch.setattr(binding, "_calls", None)
    for ignore in (0, V - 1, V + 7, -1, 2 ** 40):
        t = make(M, V, 64, seed=31)
        target = t[4]
        target[M // 2::3] = ignore
        if M > 1:
            target[0] = 7
        x, wt, swt, dloss = more(t)
        loss, lse = binding.fp8_linear_cross_entropy(*t, ignore_index=ignore)
        args = (dloss, *t, loss, lse, x, wt, swt)
        got = binding.fp8_linear_cross_entropy_backward(*args, ignore_index=ignore)
        assert (got[0][target == ignore] == 0).all() and lse.isfinite().all()
        close(got, gradient64(*args, ignore=ignore), ignore)
        # (the default one is then no entry as any other)
        target[0] = -100
        assert binding.fp8_linear_cross_entropy_backward(*args, ignore_index=ignore)[0][0].isnan().all()


@pytest.mark.parametrize("M,V", [(6, 100), (600, 9000)])
def test_a_weight_of_0_hides_what_is_no_number(M, V):
    t = make(M, V, 64, seed=19)
    x, wt, swt, dloss = more(t)
    off = torch.arange(M, device=DEV) % 3 == 1
    dloss = torch.where(off, 0.0, dloss)
    _, want = run(t, (x, wt, swt, dloss))
    a, b, sa, sb, target = t
    a.view(torch.uint8)[off] = 0x7f
    x[off] = math.nan
    target = torch.where(off, V + 5, target)
    loss, lse = binding.fp8_linear_cross_entropy(a, b, sa, sb, target)
    assert loss[off].isnan().all() and lse[off].isnan().all()
    dx, dw = binding.fp8_linear_cross_entropy_backward(dloss, a, b, sa, sb, target, loss, lse, x, wt, swt)
    assert (dx[off] == 0).all() and torch.equal(dx[~off], want[0][~off]) and torch.equal(dw, want[1])


@pytest.mark.parametrize("what", ["dloss", "loss", "lse", "inf lse", "target"])
@pytest.mark.parametrize("M,V", [(6, 100), (600, 9000)])
def test_what_is_no_number_shows(M, V, what):
    t = make(M, V, 64, seed=10)
    args, (dx, dw) = run(t, more(t))
    args = [x.clone() for x in args]
    if what == "target":
        args[5][2] = V
    else:
        args[{"dloss": 0, "loss": 6}.get(what, 7)][2] = math.inf if what == "inf lse" else math.nan
    bad_dx, bad_dw = binding.fp8_linear_cross_entropy_backward(*args)
    rest = torch.arange(M, device=DEV) != 2
    assert bad_dx[2].isnan().all() and torch.equal(bad_dx[rest], dx[rest]) and bad_dw.isnan().all()


def test_a_sure_row_has_no_gradient():
    """Where the loss is 0 in fp32, h is 0 and so is the row's gradient."""
    t = make(20, 300, 64, seed=12)
    args, _ = run(t, more(t))
    args = list(args)
    args[6] = args[6].clone()
    args[6][4], args[6][5] = 0.0, -1e-7
    dx, dw = binding.fp8_linear_cross_entropy_backward(*args)
    assert (dx[4:6] == 0).all() and dw.isfinite().all()
    close((dx, dw), gradient64(*args))


def test_a_nearly_sure_row_keeps_the_shape_of_its_gradient():
    """h = 1 - p of the target is so small that 57344 / h passes the largest float."""
    a, b, sa, sb, t = make(20, 1000, 64)
    for codes, value in ((a, 1.0), (b, 0.0)):
        codes[:] = torch.full_like(codes.float(), value).to(codes.dtype)
    b[1::2] = torch.full((500, 64), -0.5, device=DEV).to(b.dtype)
    t = torch.arange(20, device=DEV) * 48
    b[t] = torch.ones(20, 64, device=DEV).to(b.dtype)
    a, sa, sb, t = a[:1], torch.full((1,), 86 / 64, device=DEV), torch.ones_like(sb), t[3:4]
    b[t.item() + 48::48] = 0
    b[:t.item():48] = 0
    t = (a.contiguous(), b, sa, sb, t)
    tensors, got = run(t, more(t, dloss=torch.full((1,), 2.0 ** 100, device=DEV)))
    assert 0 < float(tensors[6]) < 57344 / torch.finfo(torch.float32).max
    close(got, gradient64(*tensors))


@pytest.mark.parametrize("M,V,rows", [(2 ** 23 - 5, 40, None), (3, 2 ** 23 - 5, None), (130, 2 ** 23 - 5, (3, 127))])
def test_the_largest_sizes(M, V, rows):
    """All rows, or `rows` of them and the others with a weight of 0."""
    t = make(M, V, 16, seed=24)
    extra = more(t)
    if rows:
        rows = torch.tensor(rows, device=DEV)
        extra[3][torch.ones(M, dtype=torch.bool, device=DEV).index_fill(0, rows, False)] = 0
    (dloss, a, b, sa, sb, target, loss, lse, x, wt, swt), (dx, dw) = run(t, extra)
    if rows is not None:
        dloss, a, sa, target, loss, lse, x = (v[rows].contiguous() for v in (dloss, a, sa, target, loss, lse, x))
        assert int((dx != 0).any(1).sum()) == len(rows)
        dx = dx[rows]
    close((dx, dw), gradient64(dloss, a, b, sa, sb, target, loss, lse, x, wt, swt))


def test_one_dloss_for_all_rows():
    t = make(300, 5000, 128, seed=13, ignore=-100)
    x, wt, swt, _ = more(t)
    w = torch.tensor([0.25], device=DEV)
    args, want = run(t, (x, wt, swt, torch.full((300,), 0.25, device=DEV)))
    for dloss in (w, w[0], w.expand(300)):
        got = binding.fp8_linear_cross_entropy_backward(dloss, *args[1:])
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_no_rows():
    t = make(0, 100, 64)
    args, (dx, dw) = run(t, more(t, dloss=torch.ones(0, device=DEV)))
    assert dx.shape == (0, 64) and dw.shape == (100, 64) and (dw == 0).all()


@pytest.mark.parametrize("M,V,K", [(200, 3000, 1024), (1500, 9000, 256)])
def test_equal_calls_equal_bits_whatever_the_buffers_hold(M, V, K):
    t = make(M, V, K, seed=14)
    args, want = run(t, more(t))
    need = binding.lib().fp8_linear_cross_entropy_backward_workspace_size(M, V, K, 1, 1)
    for fill in (0, 0xff, 0x7f):
        ws = torch.full((need,), fill, dtype=torch.uint8, device=DEV)
        dx, dw = torch.full((M, K), math.nan, dtype=BF16, device=DEV), torch.full((V, K), math.nan, dtype=BF16, device=DEV)
        got = binding.fp8_linear_cross_entropy_backward(*args, dx=dx, dw=dw, workspace=ws)
        assert got[0] is dx and got[1] is dw and torch.equal(dx, want[0]) and torch.equal(dw, want[1])
    with pytest.raises(ValueError):
        binding.fp8_linear_cross_entropy_backward(*args, workspace=torch.empty(need - 1, dtype=torch.uint8, device=DEV))


def moved(t, align):
    """t's values, contiguous, at an address that suits `align` bytes but not twice as many."""
    size = t.element_size()
    flat = torch.empty(t.numel() * size + 512, dtype=torch.uint8, device=DEV)
    at = -flat.data_ptr() % 256 + align
    out = flat[at:at + t.numel() * size].view(t.dtype).view(t.shape)
    assert out.data_ptr() % (2 * align) == align
    return out.copy_(t)


@pytest.mark.parametrize("M,V,K", [(3, 1001, 512), (260, 9000, 272), (1500, 9000, 256), (300, 30000, 64)])
def test_odd_addresses(M, V, K):
    t = make(M, V, K, seed=25, ignore=-100)
    x, wt, swt, dloss = more(t)
    aligns = (16, 16, 4, 4, 8)
    t = tuple(moved(v.view(torch.uint8) if n == 16 else v, n).view(v.dtype) for v, n in zip(t, aligns))
    swt, dloss, x, wt = moved(swt, 4), moved(dloss, 4), moved(x, 2), moved(wt.view(torch.uint8), 16).view(wt.dtype)
    loss, lse = (moved(v, 4) for v in binding.fp8_linear_cross_entropy(*t))
    check(loss, lse, *t)
    out = [moved(torch.full(s, 7.0, dtype=BF16, device=DEV), 2) for s in ((M, K), (V, K))]
    got = binding.fp8_linear_cross_entropy_backward(dloss, *t, loss, lse, x, wt, swt, dx=out[0], dw=out[1])
    assert got[0] is out[0] and got[1] is out[1]
    close(got, gradient64(dloss, *t, loss, lse, x, wt, swt))


def test_given_buffers_count_as_written():
    t = make(40, 100, 64)
    x, wt, swt, dloss = more(t)
    loss, lse = binding.fp8_linear_cross_entropy(*t)
    dx, dw = (torch.empty(n, 64, dtype=BF16, device=DEV) for n in (40, 100))
    for kw in (dict(dx=dx), dict(dw=dw), dict(dx=dx, dw=dw), dict(dx=dx, dw=False)):
        before = dx._version, dw._version
        binding.fp8_linear_cross_entropy_backward(dloss, *t, loss, lse, x, wt, swt, **kw)
        assert (dx._version > before[0]) == (kw.get("dx") is dx) and (dw._version > before[1]) == (kw.get("dw") is dw)


def test_threads_with_streams_of_their_own():
    problems = [make(M, V, K, seed=26) for M, V, K in ((40, 5000, 256), (1200, 9000, 128), (300, 30000, 64), (1, 3000, 512))]
    extras = [more(t) for t in problems]
    want = [run(t, e) for t, e in zip(problems, extras)]
    torch.cuda.synchronize()
    got = [None] * len(problems)

    def work(i):
        with torch.cuda.stream(torch.cuda.Stream()):
            for _ in range(5):
                got[i] = run(problems[i], extras[i])
            torch.cuda.current_stream().synchronize()

    threads = [threading.Thread(target=work, args=(i,)) for i in range(len(problems))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    for (args, out), (args0, out0) in zip(got, want):
        assert torch.equal(args[6], args0[6]) and torch.equal(args[7], args0[7])
        assert torch.equal(out[0], out0[0]) and torch.equal(out[1], out0[1])


def test_captured_and_replayed():
    calls = []
    for M, V, K in ((3, 2000, 2048), (700, 9000, 256)):
        t = make(M, V, K, seed=17)
        calls.append(run(t, more(t)))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=torch.cuda.Stream()):
        outs = [binding.fp8_linear_cross_entropy_backward(*args) for args, _ in calls]
    for rep in range(3):
        for o in outs:
            for x in o:
                x.fill_(-1)
        binding.fp8_linear_cross_entropy_backward(*calls[rep % 2][0])
        graph.replay()
        torch.cuda.synchronize()
        for o, (_, w) in zip(outs, calls):
            assert all(torch.equal(x, y) for x, y in zip(o, w)), rep
