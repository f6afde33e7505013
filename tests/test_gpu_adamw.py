"""The AdamW step over many tensors on the GPU against 64 bits.

Tolerances, with u = 2^-24.  m = b1 m0 + c1 g: the constants, the products and the sum
round once each, so m is off by dm = 3 u (b1 |m0| + c1 |g|); v likewise, with g^2
rounded too, by 4 u v.  The denominator (a square root, a product by a rounded factor
and a sum) is then off by 5 u of itself, the quotient rounds by u, lr / (1 - b1^t) by 3 u
and the products by 2 u: a step of size s is off by 12 u s + dm s / |m|, and p (its
factor 1 - lr wd off by 2 u, the sum by u) by 3 u |p| more.  With 8-bit moments the quotient is
by the hardware's reciprocal, off by 2 u, and its product rounds: 4 u more.  A bf16 output is rounded once
more (torch.finfo(bf16).eps / 2).

Moments of 8 bits.  What is rounded to a code, x / scale, is off by dm / scale (m), 3 u
(sqrt(v)), by 3 u for the scale, its reciprocal and the product, and below 2^-6 by 2^-30 of the
sum that is formed there; rounding up or down at random is monotonous, so the codes of the two
bounds are the ends.
"""
import math

import pytest
import torch

from precision_linear_amd import binding

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF16, FP32 = torch.bfloat16, torch.float32
U = 2.0 ** -24
HALF = torch.finfo(BF16).eps / 2
HYPER = dict(lr=2e-3, betas=(0.9, 0.995), eps=1e-8, weight_decay=0.05)


def make(sizes, param=FP32, grad=FP32, bits=32, master=False, seed=0, odd=0):
    """Lists of tensors; odd: elements by which their addresses are off."""
    g = torch.Generator(device=DEV).manual_seed(seed)

    def one(n, scale, dtype):
        t = torch.empty(n + odd, dtype=dtype, device=DEV)[odd:]
        return t.copy_(scale * torch.randn(n, generator=g, device=DEV))

    p = [one(n, 0.05, param) for n in sizes]
    t = dict(params=p, grads=[one(n, 1e-3, grad) for n in sizes], master=None, exp_avg_scale=None, exp_avg_sq_scale=None)
    if master:
        t["master"] = [(x.float() * (1 + 1e-3 * torch.randn(x.shape, generator=g, device=DEV))) for x in p]
    m = [one(n, 5e-4, FP32) for n in sizes]
    v = [one(n, 1e-3, FP32).square_() for n in sizes]
    if bits == 32:
        return t | dict(exp_avg=m, exp_avg_sq=v)
    for name, xs in (("exp_avg", m), ("exp_avg_sq", [x.sqrt() for x in v])):
        t[name], t[name + "_scale"] = [], []
        for x in xs:
            blocks = (x.numel() + 255) // 256
            pad = torch.zeros(blocks * 256, device=DEV)
            pad[:x.numel()] = x
            s = pad.view(-1, 256).abs().amax(1) / 448
            q = (pad.view(-1, 256) / s[:, None]).nan_to_num(0).view(-1)[:x.numel()].to(torch.float8_e4m3fn)
            t[name].append(torch.empty(x.numel() + odd, dtype=torch.uint8, device=DEV)[odd:].copy_(q.view(torch.uint8)))
            t[name + "_scale"].append(s)
    return t


def copies(t):
    return {k: None if v is None else [x.clone() for x in v] for k, v in t.items()}


def random_bits(seed, at):
    low = 0xffffffff
    x = (at * 0x6A09E667 + (seed * 0xBB67AE85 & low)) & low
    x = ((x ^ (x >> 15)) * 0x3C6EF373) & low
    x = ((x ^ (x >> 13)) * 0xA54FF53B) & low
    return x ^ (x >> 16)


def code_at_random(y, r, positive):
    """y >= 0 to e4m3fn's values, up where the part of a step and r / 2^16 make one."""
    y = y.clamp(0, 448)
    _, e = torch.frexp(y)
    powers = torch.tensor([2.0 ** i for i in range(-9, 6)], dtype=torch.float64, device=y.device)
    step = powers[(e.long() - 1).clamp(-6, 8) - 3 + 9]
    t = torch.floor(y / step + r.double() / 65536) * step
    return torch.where((y > 0) & (t == 0), 2.0 ** -9, t) if positive else t


def check(before, after, step, seed=0, gs=1.0, lr=HYPER["lr"], betas=HYPER["betas"], eps=HYPER["eps"],
          weight_decay=HYPER["weight_decay"]):
    b1, b2 = betas
    eight = before["exp_avg_scale"] is not None
    blocks_before = 0
    for i, p in enumerate(before["params"]):
        n = p.numel()
        blocks = (n + 255) // 256
        of = torch.arange(n, device=DEV) // 256
        g = before["grads"][i].double() * gs
        w0 = (p if before["master"] is None else before["master"][i]).double()
        m0, v0 = before["exp_avg"][i], before["exp_avg_sq"][i]
        if eight:
            m0 = m0.view(torch.float8_e4m3fn).double() * before["exp_avg_scale"][i].double()[of]
            v0 = (v0.view(torch.float8_e4m3fn).double() * before["exp_avg_sq_scale"][i].double()[of]).square()
        m0, v0 = m0.double(), v0.double()
        m, v = b1 * m0 + (1 - b1) * g, b2 * v0 + (1 - b2) * g * g
        extra = 4 * U if eight else 0                       # (the stored values are products, squared)
        dm = (3 * U + extra + 2 * U * (gs != 1)) * (b1 * m0.abs() + (1 - b1) * g.abs())
        rv = 4 * U + extra + 4 * U * (gs != 1)              # of v
        fast = 4 * U * eight
        den = v.sqrt() / math.sqrt(1 - b2 ** step) + eps
        rate = lr / (1 - b1 ** step)
        w = w0 * (1 - lr * weight_decay) - rate * m / den
        tol = 3 * U * w0.abs() + rate / den * (dm + (12 * U + rv + fast) * m.abs()) + 1e-44
        for x, half in ((after["params"][i], HALF if p.dtype == BF16 else 0),
                        (None if after["master"] is None else after["master"][i], 0)):
            if x is not None:
                off = (x.double() - w).abs()
                assert (off <= tol + half * (w.abs() + tol)).all(), (i, float((off / tol).max()))
        if not eight:
            assert ((after["exp_avg"][i].double() - m).abs() <= dm + 1e-44).all()
            assert ((after["exp_avg_sq"][i].double() - v).abs() <= rv * v + 1e-44).all()
            continue
        r = random_bits(seed, torch.arange(n, device=DEV) + 256 * blocks_before)
        blocks_before += blocks
        for name, x, d, bits, positive in (("exp_avg", m, dm, r & 0xffff, False),
                                           ("exp_avg_sq", v.sqrt(), (rv + fast) * v.sqrt(), r >> 16, True)):
            scale = torch.zeros(blocks, dtype=torch.float64, device=DEV).scatter_reduce(0, of, x.abs(), "amax") / 448
            most = torch.zeros(blocks, dtype=torch.float64, device=DEV).scatter_reduce(0, of, d, "amax") / 448
            got = after[name + "_scale"][i].double()
            assert ((got - scale).abs() <= 2 * U * scale + most + 1e-44).all(), name
            y = torch.where(scale[of] > 0, x.abs() / scale[of], 0.0)
            dy = torch.where(scale[of] > 0, (d + y * most[of]) / scale[of], 0.0) + 6 * U * y + 2.0 ** -30
            lo = code_at_random((y - dy).clamp(min=0), bits, False)
            hi = code_at_random(y + dy, bits, positive)
            c = after[name][i].view(torch.float8_e4m3fn).double()
            assert ((c.abs() >= lo) & (c.abs() <= hi)).all(), (name, i)
            assert ((c == 0) | (torch.sign(c) == torch.sign(x)) | (x.abs() <= d)).all()
            if positive:
                assert ((c > 0) | (x == 0)).all()


SIZES = [[1], [2, 3], [255, 256, 257], [4095, 4096, 4097, 0, 5], [100003], [1 << 20, 7]]
TYPES = [(FP32, FP32, False), (FP32, BF16, False), (BF16, BF16, False), (BF16, FP32, True), (BF16, BF16, True),
         (BF16, FP32, False)]


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("param,grad,master", TYPES)
@pytest.mark.parametrize("sizes", SIZES)
def test_step(sizes, param, grad, master, bits):
    print(f"[adamw] {sizes} {param} {grad} {master} {bits}", flush=True)
    for step, odd in ((1, 0), (1000, 1), (3, 3)):
        t = make(sizes, param, grad, bits, master, seed=step, odd=odd)
        before = copies(t)
        assert binding.adamw_step(**t, step=step, seed=step * 77, **HYPER) is None
        check(before, t, step, step * 77)
        assert all(torch.equal(a, b) for a, b in zip(t["grads"], before["grads"]))


@pytest.mark.parametrize("path", ["short", "whole"])
@pytest.mark.parametrize("master", [True, False])
@pytest.mark.parametrize("bits", [32, 8])
def test_an_empty_tensor_first(bits, master, path, monkeypatch):
    if path == "whole":
        monkeypatch.setattr(binding, "_calls", None)
    for sizes in ([0, 1000], [0, 0, 300, 0, 4097], [0]):
        t = make(sizes, BF16, BF16, bits, master)
        before = copies(t)
        binding.adamw_step(**t, step=5, seed=11, **HYPER)
        check(before, t, 5, 11)


@pytest.mark.parametrize("bits", [32, 8])
def test_many_tensors(bits):
    """More than a launch takes; positions go on through the list."""
    g = torch.Generator().manual_seed(1)
    sizes = [int(n) for n in torch.randint(0, 9000, (131,), generator=g)]
    t = make(sizes, BF16, BF16, bits, True)
    before = copies(t)
    binding.adamw_step(**t, step=7, seed=123, **HYPER)
    check(before, t, 7, 123)


@pytest.mark.parametrize("bits", [32, 8])
def test_beyond_the_memory_side_cache(bits):
    n = 40_000_001
    t = make([n, 300], FP32, BF16, bits)
    before = copies(t)
    binding.adamw_step(**t, step=2, seed=5, **HYPER)
    check(before, t, 2, 5)


def test_what_lies_around_the_tensors_stays():
    for bits in (32, 8):
        for dtype in (FP32, BF16):
            t = make([1000], dtype, dtype, bits)
            around = {}
            for name in ("params", "exp_avg", "exp_avg_sq"):
                x = t[name][0]
                whole = torch.full((x.numel() + 64,), 3, dtype=x.dtype, device=DEV)
                whole[32:-32] = x
                t[name] = [whole[32:-32]]
                around[name] = whole
            binding.adamw_step(**t, step=1, **HYPER)
            for whole in around.values():
                assert (whole[:32] == 3).all() and (whole[-32:] == 3).all()


@pytest.mark.parametrize("hyper", [dict(lr=0.0), dict(betas=(0.0, 0.0)), dict(eps=0.0), dict(weight_decay=0.0), dict(eps=1.0),
                                   dict(betas=(0.99, 0.0)), dict(weight_decay=500.0)])
@pytest.mark.parametrize("bits", [32, 8])
def test_hyperparameters(hyper, bits):
    t = make([5000], FP32, FP32, bits, seed=3)
    before = copies(t)
    binding.adamw_step(**t, step=5, **HYPER | hyper)
    check(before, t, 5, **hyper)


def test_zero_gradients_and_states():
    for bits in (32, 8):
        t = make([700, 20], FP32, FP32, bits)
        s = binding.adamw_state(t["params"], bits)
        t |= dict(exp_avg=s.exp_avg, exp_avg_sq=s.exp_avg_sq, exp_avg_scale=s.exp_avg_scale,
                  exp_avg_sq_scale=s.exp_avg_sq_scale)
        for g in t["grads"]:
            g.zero_()
        before = copies(t)
        binding.adamw_step(**t, step=1, **HYPER)
        check(before, t, 1)
        for name in ("exp_avg", "exp_avg_sq"):
            assert all((x.view(torch.uint8) == 0).all() for x in t[name])


@pytest.mark.parametrize("eps", [1e-38, 1e-40, 1e-44, 1e-60])
def test_an_eps_below_the_smallest_normal_number(eps):
    """0 over it is 0, in 8 bits too, where the quotient is by a reciprocal."""
    for bits in (32, 8):
        t = make([700, 20], FP32, FP32, bits)
        s = binding.adamw_state(t["params"], bits)
        t |= dict(exp_avg=s.exp_avg, exp_avg_sq=s.exp_avg_sq, exp_avg_scale=s.exp_avg_scale,
                  exp_avg_sq_scale=s.exp_avg_sq_scale)
        for g in t["grads"]:
            g[::2] = 0
        before = copies(t)
        binding.adamw_step(**t, step=1, **HYPER | dict(eps=eps))
        check(before, t, 1, eps=eps)


def test_small_second_moments_are_never_lost():
    """A block with one large gradient: the others' sqrt(v) would be 0 in 8 bits, and their step m / eps."""
    t = make([256], FP32, FP32, 8)
    s = binding.adamw_state(t["params"], 8)
    t |= dict(exp_avg=s.exp_avg, exp_avg_sq=s.exp_avg_sq, exp_avg_scale=s.exp_avg_scale, exp_avg_sq_scale=s.exp_avg_sq_scale)
    t["grads"][0].fill_(1e-7)
    t["grads"][0][7] = 1.0
    p0 = t["params"][0].clone()
    for step in range(1, 20):
        binding.adamw_step(**t, step=step, seed=step, **HYPER)
        assert (t["exp_avg_sq"][0].view(torch.uint8) > 0).all()
    # Each step is at most lr (1 + what m may be rounded up by: a whole code of 2^-9) / (...) of the
    # stored sqrt(v), itself at least a code: no more than a few lr, where m / eps would be 10^4 lr.
    assert (t["params"][0] - p0).abs().max() < 19 * HYPER["lr"] * 40


@pytest.mark.parametrize("bits", [32, 8])
def test_gradients_whose_squares_are_next_to_nothing(bits):
    """v down to fp32's subnormal numbers: its root is no 0."""
    t = make([256, 256, 256], FP32, FP32, bits)
    s = binding.adamw_state(t["params"], bits)
    t |= dict(exp_avg=s.exp_avg, exp_avg_sq=s.exp_avg_sq, exp_avg_scale=s.exp_avg_scale, exp_avg_sq_scale=s.exp_avg_sq_scale)
    for g, size in zip(t["grads"], (1e-14, 1e-16, 1e-18)):
        g.copy_(size * (1 + torch.rand(256, device=DEV)))
    before = copies(t)
    binding.adamw_step(**t, step=1, **HYPER | dict(eps=0.0, betas=(0.0, 0.5)))
    check(before, t, 1, eps=0.0, betas=(0.0, 0.5))


@pytest.mark.parametrize("bits", [32, 8])
def test_no_numbers_show(bits):
    t = make([1000, 600], FP32, FP32, bits)
    t["grads"][0].view(torch.int32)[300] = -1                # a NaN of all ones
    t["grads"][1][10] = math.inf
    binding.adamw_step(**t, step=2, **HYPER)
    p, q = t["params"]
    assert p[300].isnan() and p.isnan().sum() == 1
    assert q[10].isnan() and q.isnan().sum() == 1
    m = t["exp_avg"][0]
    m = m.view(torch.float8_e4m3fn).float() if bits == 8 else m
    assert m[300].isnan() and m.isnan().sum() == 1
    binding.adamw_step(**t, step=3, **HYPER)
    assert p[300].isnan() and p.isnan().sum() == 1


def test_grad_scale():
    gs = torch.tensor([0.125], device=DEV)
    for bits in (32, 8):
        t = make([3000, 11], BF16, BF16, bits, True)
        before = copies(t)
        binding.adamw_step(**t, step=4, grad_scale=gs, **HYPER)
        check(before, t, 4, gs=0.125)


def test_one_gradient_for_two_parameters():
    t = make([1000, 1000], FP32, FP32)
    t["grads"][1] = t["grads"][0]
    before = copies(t)
    binding.adamw_step(**t, step=1, **HYPER)
    check(before, t, 1)


def test_shapes_and_state_helper():
    p = [torch.randn(s, device=DEV).to(BF16) for s in ((), (3,), (4, 5, 6), (0, 3), (33, 64))]
    g = [torch.randn_like(x) for x in p]
    for bits in (32, 8):
        for master in (True, False):
            s = binding.adamw_state(p, bits, master)
            w = [x.clone() for x in p]
            t = dict(params=w, grads=g, **s._asdict())
            flat = {k: None if v is None else [x.reshape(-1).clone() for x in v] for k, v in t.items()}
            binding.adamw_step(**t, step=1, **HYPER)
            check(flat, {k: None if v is None else [x.reshape(-1) for x in v] for k, v in t.items()}, 1)


def same(a, b):
    assert a.keys() == b.keys()
    for k in a:
        assert (a[k] is None) == (b[k] is None)
        for x, y in zip(a[k] or [], b[k] or []):
            assert torch.equal(x.view(torch.uint8) if x.dtype.itemsize == 1 else x, y.view(torch.uint8) if y.dtype.itemsize == 1 else y), k


@pytest.mark.parametrize("bits", [32, 8])
def test_numbers_on_the_gpu_and_both_paths(bits, monkeypatch):
    """Tensors in place of numbers, and the binding without its extension: the same bits."""
    results = []
    for short in (True, False):
        if not short:
            monkeypatch.setattr(binding, "_calls", None)
        for tensors in (False, True):
            t = make([4097, 300, 0, 70000], BF16, BF16, bits, True)
            num = dict(step=9, lr=0.001953125, seed=(1 << 33) + 5)
            if tensors:
                num = dict(step=torch.tensor([9.0], device=DEV), lr=torch.tensor(0.001953125, device=DEV),
                           seed=torch.tensor([(1 << 33) + 5], device=DEV))
            binding.adamw_step(**t, **num, betas=(0.9, 0.995))
            results.append(t)
    for r in results[1:]:
        same(r, results[0])


def block_codes(x, r, positive):
    """The definition in fp32, as include/adamw.h has it; x is whole blocks."""
    amax = x.view(-1, 256).abs().amax(1, keepdim=True)
    scale = amax / torch.full_like(amax, 448.0)
    y = (x.view(-1, 256) * torch.where(scale > 0, 1 / scale, 0.0)).view(-1)
    t = y.abs().clamp(max=448.0)
    lift = torch.where(t < 2.0 ** -6, 2.0 ** -6, 0.0)
    t = (((t + lift).view(torch.int32) + (r << 4).to(torch.int32)) & ~0xfffff).view(torch.float32) - lift
    if positive:
        t = torch.where((y > 0) & (t == 0), 2.0 ** -9, t)
    return torch.copysign(t, y).to(torch.float8_e4m3fn).view(torch.uint8), scale[:, 0]


def test_codes_are_the_definitions_bit_for_bit():
    """Every product, sum and root of the moments is rounded as it is written, so over steps
    the codes and scales are those of fp32 arithmetic, none off by a neighbour."""
    n = 1 << 22
    t = make([n], FP32, BF16, 8)
    b1, b2 = HYPER["betas"]
    m8, v8, ms, vs = (t[k][0].clone() for k in ("exp_avg", "exp_avg_sq", "exp_avg_scale", "exp_avg_sq_scale"))
    g = torch.Generator(device=DEV).manual_seed(8)
    for step in range(1, 6):
        t["grads"][0].copy_(1e-3 * torch.randn(n, generator=g, device=DEV))
        binding.adamw_step(**t, step=step, seed=step, **HYPER)
        grad = t["grads"][0].float()
        m = b1 * (m8.view(torch.float8_e4m3fn).float().view(-1, 256) * ms[:, None]).view(-1) + (1 - b1) * grad
        v = (v8.view(torch.float8_e4m3fn).float().view(-1, 256) * vs[:, None]).view(-1)
        v = b2 * (v * v) + (1 - b2) * (grad * grad)
        r = random_bits(step, torch.arange(n, device=DEV))
        m8, ms = block_codes(m, r & 0xffff, False)
        v8, vs = block_codes(v.double().sqrt().float(), r >> 16, True)
        for name, want in (("exp_avg", m8), ("exp_avg_sq", v8), ("exp_avg_scale", ms), ("exp_avg_sq_scale", vs)):
            assert torch.equal(t[name][0], want), (step, name)


def test_equal_calls_equal_bits_and_seeds_differ():
    a, b, c = (make([50000], FP32, BF16, 8) for _ in range(3))
    binding.adamw_step(**a, step=2, seed=1, **HYPER)
    binding.adamw_step(**b, step=2, seed=1, **HYPER)
    binding.adamw_step(**c, step=2, seed=2, **HYPER)
    same(a, b)
    assert not torch.equal(a["exp_avg"][0], c["exp_avg"][0]) and torch.equal(a["params"][0], c["params"][0])


def test_moments_of_8_bits_follow_those_of_32():
    """E[sqrt(v)] over many elements.  Between codes 2^-3 to 2^-4 apart a change of
    (1 - b2) / 2 of sqrt(v) is a step with a probability of 0.04 at most, so one element's sqrt(v) wanders
    by sigma^2 = 0.04 (2^-3)^2 / (2 (1 - b2) / 2 2) < 0.07; its mean moves by up to sigma^2 / 2 (g^2 / sqrt(v) is
    convex), the mean's error over 2^16 elements is 2^-8 sigma: within 5 % in all."""
    n = 1 << 16
    a, b = make([n], FP32, FP32, 32), make([n], FP32, FP32, 8)
    for t, bits in ((a, 32), (b, 8)):
        s = binding.adamw_state(t["params"], bits)
        t |= dict(exp_avg=s.exp_avg, exp_avg_sq=s.exp_avg_sq, exp_avg_scale=s.exp_avg_scale, exp_avg_sq_scale=s.exp_avg_sq_scale)
    g = torch.Generator(device=DEV).manual_seed(5)
    scale = torch.exp(torch.randn(n, generator=g, device=DEV))
    for step in range(1, 601):
        grad = scale * torch.randn(n, generator=g, device=DEV)
        if step > 400:
            grad *= 0.25                                    # the moments have to come down again
        for t in (a, b):
            t["grads"][0].copy_(grad)
            binding.adamw_step(**t, step=step, seed=step, **HYPER)
    v = b["exp_avg_sq"][0].view(torch.float8_e4m3fn).float() * b["exp_avg_sq_scale"][0].repeat_interleave(256)
    ratio = (v / a["exp_avg_sq"][0].sqrt()).double()
    live = scale > 0.1                                      # (far below the block's largest, a code is coarse)
    assert abs(float(ratio[live].mean()) - 1) < 0.05
    m = b["exp_avg"][0].view(torch.float8_e4m3fn).float() * b["exp_avg_scale"][0].repeat_interleave(256)
    off = ((m - a["exp_avg"][0]).double() / a["exp_avg_sq"][0].double().sqrt())[live]
    assert abs(float(off.mean())) < 6 / 2 ** 8              # unbiased: within 6 sigma of its mean, sigma < 1


def test_captured_and_replayed():
    for bits in (32, 8):
        a, b = (make([5000, 300, 1], BF16, BF16, bits, True, seed=2) for _ in range(2))
        step, seed = torch.ones(1, device=DEV), torch.zeros(1, dtype=torch.int64, device=DEV)
        graph = torch.cuda.CUDAGraph()
        warm = copies(a)
        binding.adamw_step(**warm, step=step, seed=seed, **HYPER)
        with torch.cuda.graph(graph, stream=torch.cuda.Stream()):
            binding.adamw_step(**a, step=step, seed=seed, **HYPER)
            step.add_(1)
            seed.add_(1)
        step.fill_(1)
        seed.fill_(0)
        for rep in range(4):
            graph.replay()
            binding.adamw_step(**b, step=rep + 1, seed=rep, **HYPER)
            torch.cuda.synchronize()
            same(a, b)


def test_another_stream():
    a, b = (make([100000], FP32, BF16, 8) for _ in range(2))
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        for step in range(1, 5):
            binding.adamw_step(**a, step=step, seed=step, **HYPER)
    s.synchronize()
    for step in range(1, 5):
        binding.adamw_step(**b, step=step, seed=step, **HYPER)
    same(a, b)


@pytest.mark.parametrize("path", ["short", "whole"])
def test_refusals(monkeypatch, path):
    if path == "whole":
        monkeypatch.setattr(binding, "_calls", None)
    t = make([100, 50], BF16, BF16, 32, True)
    u = make([100, 50], FP32, BF16, 8)
    before = copies(t)
    bad = [(t, dict(grads=t["grads"][:1])), (t, dict(grads=[t["grads"][0].half(), t["grads"][1].half()])),
           (t, dict(grads=[g.cpu() for g in t["grads"]])), (t, dict(params=[p.cpu() for p in t["params"]])),
           (t, dict(exp_avg=[t["exp_avg"][0], t["exp_avg"][1].half()])), (t, dict(master=t["master"][:1])),
           (t, dict(params=[t["params"][0]] * 2, grads=[t["grads"][0]] * 2, exp_avg=[t["exp_avg"][0]] * 2,
                    exp_avg_sq=[t["exp_avg_sq"][0]] * 2, master=[t["master"][0]] * 2)),
           (t, dict(exp_avg_sq=t["exp_avg"])),
           (t, dict(exp_avg_scale=u["exp_avg_scale"])), (u, dict(exp_avg_scale=None)),
           (u, dict(exp_avg_scale=u["exp_avg_scale"][:1])), (u, dict(master=[p.clone() for p in u["params"]])),
           (u, dict(exp_avg_sq=[x.float() for x in u["exp_avg_sq"]])),
           (u, dict(exp_avg_scale=[torch.zeros(2, device=DEV)] * 2)),
           (t, dict(step=0)), (t, dict(step=1.5)), (t, dict(step=None)), (t, dict(lr=-1.0)), (t, dict(lr="fast")), (t, dict(seed=0.5)), (t, dict(lr=math.nan)), (t, dict(eps=-1e-8)), (t, dict(eps=math.inf)),
           (t, dict(betas=(1.0, 0.9))), (t, dict(betas=(0.9, -0.1))), (t, dict(weight_decay=-0.1)),
           (t, dict(step=torch.ones(1, dtype=torch.int64, device=DEV))), (t, dict(lr=torch.ones(2, device=DEV))),
           (t, dict(seed=torch.ones(1, device=DEV))), (t, dict(grad_scale=0.5)), (t, dict(grad_scale=torch.ones(1))),
           (t, dict(params=[p.view(10, -1).t() for p in t["params"]]))]
    for base, kw in bad:
        with pytest.raises(ValueError):
            binding.adamw_step(**{**base, "step": 1, **HYPER, **kw})
    torch.cuda.synchronize()
    same(t, before)
    binding.adamw_step([], [], [], [], step=1, lr=0.1)
    with pytest.raises(ValueError):
        binding.adamw_state(t["params"], 16)


@pytest.mark.parametrize("path", ["short", "whole"])
@pytest.mark.parametrize("bits", [32, 8])
def test_a_graph_sees_that_its_parameter_has_moved(bits, path, monkeypatch):
    """What a step writes counts as written: a backward pass that saved it before the step refuses to run
    on the new values, as after torch's own steps."""
    if path == "whole":
        monkeypatch.setattr(binding, "_calls", None)
    t = make([300, 0, 70], BF16, BF16, bits, True)
    written = [x for k, v in t.items() if k != "grads" and v is not None for x in v]
    before = [x._version for x in written], [x._version for x in t["grads"]]
    x = torch.ones(300, device=DEV, dtype=BF16, requires_grad=True)
    y = (x * t["params"][0]).sum()
    binding.adamw_step(**t, step=1, **HYPER)
    assert all(x._version > v for x, v in zip(written, before[0]))
    assert [x._version for x in t["grads"]] == before[1]
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        y.backward()
    after = [x._version for x in written]
    with pytest.raises(ValueError):                          # a refused step writes nothing
        binding.adamw_step(**t, step=0, **HYPER)
    assert [x._version for x in written] == after


@pytest.mark.parametrize("path", ["short", "whole"])
def test_tensors_of_inference_mode(path, monkeypatch):
    """They have no version counter."""
    if path == "whole":
        monkeypatch.setattr(binding, "_calls", None)
    with torch.inference_mode():
        t = make([300, 5], FP32, FP32, 8)
        before = copies(t)
        binding.adamw_step(**t, step=1, **HYPER)
    binding.adamw_step(**t, step=2, **HYPER)
    with torch.inference_mode():
        binding.adamw_step(**before, step=1, **HYPER)
        binding.adamw_step(**before, step=2, **HYPER)
        same(t, before)
