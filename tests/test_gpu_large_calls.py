"""Calls that move more than the memory-side cache holds (256 MB): their loads and
stores carry the non-temporal hint, and nothing else about them may differ.

Rows of a norm do not depend on each other, so a large call has to give the bits
of the same rows in small calls.  The products are taken of whole numbers whose
scales are powers of two, so that every sum is exact in fp32 in any order.
"""
import pytest
import torch

from precision_linear_amd import binding

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF16 = torch.bfloat16
CACHED = 256 << 20
U = 2.0 ** -24


def bits(t):
    return t.view({1: torch.uint8, 2: torch.int16, 4: torch.int32}[t.element_size()])


def chunks(rows, parts=6):
    edges = [rows * i // parts for i in range(parts + 1)]
    return list(zip(edges, edges[1:]))


@pytest.mark.parametrize("rows,cols,y,fmt", [(14001, 4096, True, "e4m3fn"), (60001, 1008, True, "e5m2"),
                                             (17000, 4097, True, None), (6100, 16384, False, "e4m3fn"),
                                             (150001, 513, True, None)])
def test_layer_norm(rows, cols, y, fmt):
    print(f"[layer_norm] {rows} x {cols} y={y} {fmt}", flush=True)
    assert rows * cols * (2 + 2 * y + (fmt is not None)) > CACHED
    g = torch.Generator(device=DEV).manual_seed(rows)
    x = (torch.randn(rows, cols, generator=g, device=DEV) * 3 + 1).to(BF16)
    w, b = (torch.randn(cols, generator=g, device=DEV) for _ in range(2))
    got = binding.fp8_layer_norm(x, w, b, y=y, fmt=fmt, stats=True)
    for r0, r1 in chunks(rows):
        assert (r1 - r0) * cols * 5 < CACHED
        want = binding.fp8_layer_norm(x[r0:r1], w, b, y=y, fmt=fmt, stats=True)
        for name, p, q in zip(got._fields, got, want):
            assert (p is None) == (q is None)
            assert p is None or torch.equal(bits(p[r0:r1]), bits(q)), (name, r0)


@pytest.mark.parametrize("rows,cols,residual", [(8300, 4104, True), (12000, 4097, False), (70000, 1000, True),
                                                (11000, 16384, False), (90001, 511, False)])
def test_layer_norm_backward(rows, cols, residual):
    print(f"[layer_norm_backward] {rows} x {cols} residual={residual}", flush=True)
    assert rows * cols * 2 * (3 + residual) > CACHED
    g = torch.Generator(device=DEV).manual_seed(rows)
    x, dy, res = (torch.randn(rows, cols, generator=g, device=DEV).to(BF16) for _ in range(3))
    res = res if residual else None
    w = torch.randn(cols, generator=g, device=DEV)
    st = binding.fp8_layer_norm(x, stats=True)
    dx, dw, db = binding.fp8_layer_norm_backward(dy, x, st.mean, st.rstd, w, residual_grad=res)
    sums = torch.zeros(4, cols, dtype=torch.float64, device=DEV)
    for r0, r1 in chunks(rows, 8):
        s = slice(r0, r1)
        want = binding.fp8_layer_norm_backward(dy[s], x[s], st.mean[s], st.rstd[s], w,
                                               residual_grad=res[s] if residual else None)[0]
        assert torch.equal(bits(dx[s]), bits(want)), r0
        d = dy[s].double()
        t = d * ((x[s].double() - st.mean[s, None].double()) * st.rstd[s, None].double())
        for i, v in enumerate((t, t.abs(), d, d.abs())):
            sums[i] += v.sum(0)
    # At most rows / 256 + 1 of 16 waves' rows in a row per partial sum, 256 of those
    # in 32 slices, and the joins; 4 roundings in a term of dw.
    bound = (rows / 256 + 80) * U
    assert ((dw.double() - sums[0]).abs() <= bound * sums[1]).all()
    assert ((db.double() - sums[2]).abs() <= bound * sums[3]).all()


def whole(g, rows, cols, most=7):
    return torch.randint(-most, most + 1, (rows, cols), generator=g, device=DEV).float()


@pytest.mark.parametrize("mode", ["rowwise", "per_tensor"])
@pytest.mark.parametrize("M,N,K", [(4100, 28672, 1040), (4096, 28680, 1040), (16392, 8200, 144)])
def test_products_of_whole_numbers(M, N, K, mode):
    print(f"[linear] {M} x {N} x {K} {mode}", flush=True)
    assert M * K + N * K + 2 * M * N > CACHED
    g = torch.Generator(device=DEV).manual_seed(M + N)
    a, b = whole(g, M, K), whole(g, N, K)
    if mode == "rowwise":
        sa, sb = (2.0 ** torch.randint(-3, 4, (n,), generator=g, device=DEV) for n in (M, N))
    else:
        sa, sb = torch.full((1,), 0.5, device=DEV), torch.full((1,), 2.0, device=DEV)
    bias, res = whole(g, 1, N, 99)[0].to(BF16), whole(g, M, N, 99).to(BF16)
    z = (a @ b.t()) * (sa[:, None] * sb if mode == "rowwise" else sa * sb)     # exact: sums under 2^17, 2^-6 steps
    qa, qb = a.to(torch.float8_e4m3fn), b.to(torch.float8_e4m3fn)
    config = len(binding.config_names()) - 1                                   # the 256 x 256 tiles
    for bi in (None, bias):
        zb = z if bi is None else z + bi.float()
        out = binding.fp8_scaled_mm(qa, qb, sa, sb, bi, mode=mode, config=config)
        assert torch.equal(bits(out), bits(zb.to(BF16)))
        pre = torch.empty(M, N, dtype=BF16, device=DEV)
        out = binding.fp8_linear(qa, qb, sa, sb, bi, res, activation="relu", preact=pre, mode=mode, config=config)
        assert torch.equal(bits(pre), bits(zb.to(BF16)))
        assert torch.equal((zb.clamp(min=0) + res.float()).to(BF16), out)
        out = binding.fp8_linear(qa, qb, sa, sb, bi, activation="relu", mode=mode, config=config)
        assert torch.equal(zb.clamp(min=0).to(BF16), out)


@pytest.mark.parametrize("M,N,K,act", [(2500, 28672, 272, "relu"), (5000, 27008, 528, "none"),
                                       (70000, 1040, 144, "relu")])
def test_gradient_of_whole_numbers(M, N, K, act):
    print(f"[linear_backward] {M} x {N} x {K} {act}", flush=True)
    assert 2 * M * ((1 + (act != "none")) * N + K) > CACHED and 49 * max(M, N) < 2 ** 24
    g = torch.Generator(device=DEV).manual_seed(M + N)
    dy, x, w = whole(g, M, N), whole(g, M, K), whole(g, K, N)
    z = torch.randn(M, N, generator=g, device=DEV).to(BF16)
    i = torch.arange(max(M, N), device=DEV)
    dy[i % M, i % N] = 7             # a 7 in every row and column: scales are powers of 2
    z[i % M, i % N] = 1
    x[i[:max(M, K)] % M, i[:max(M, K)] % K] = 7
    dx, dw, db = binding.fp8_linear_backward(dy.to(BF16), x.to(BF16), w.to(torch.float8_e4m3fn),
                                             torch.full((K,), 0.5, device=DEV), z, activation=act)
    dz = dy * (z > 0) if act == "relu" else dy
    assert torch.equal(dx, (dz @ (0.5 * w).t()).to(BF16))
    assert torch.equal(dw, (dz.t() @ x).to(BF16))
    assert torch.equal(db, dz.sum(0))
