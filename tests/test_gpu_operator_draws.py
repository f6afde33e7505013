"""The operators at sizes drawn over their ranges (spread over the logarithm,
odd ones among them), each against 64 bits with its own test's bounds."""
import math
import random

import pytest

import test_gpu_layer_norm as norm
import test_gpu_linear as linear
import test_gpu_linear_backward as backward

pytestmark = pytest.mark.gpu
ACTS = ("none", "relu", "gelu", "gelu_tanh", "silu")


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _norm_shape(rng):
    while True:
        rows, cols = _log(rng, 1, 16384), _log(rng, 1, 40000)
        if rows * cols <= 3e6:
            return rows, cols


def _product_shape(rng, step_n):
    while True:
        m, n, k = _log(rng, 1, 8192), _log(rng, step_n, 28672), max(16, _log(rng, 16, 28672) // 16 * 16)
        n = max(step_n, n // step_n * step_n)
        if m * n * k <= 3e9 and m * n + n * k + m * k <= 2e7:
            return m, n, k


@pytest.mark.parametrize("seed", range(24))
def test_layer_norm(seed):
    rng = random.Random(seed)
    rows, cols = _norm_shape(rng)
    dtype = rng.choice((norm.BF16, norm.FP32))
    x, w, b = norm.make(rows, cols, dtype, seed, rng.choice((norm.BF16, norm.FP32)))
    norm.check_forward(x, w, b)
    norm.check_backward(x, w, seed, residual=rng.random() < 0.5)
    cols = max(16, cols // 16 * 16)
    x, w, b = norm.make(rows, cols, dtype, seed)
    norm.check_forward(x, w, b, y=rng.random() < 0.5, fmt=rng.choice(("e4m3fn", "e5m2")))


@pytest.mark.parametrize("seed", range(32))
def test_linear(seed):
    rng = random.Random(100 + seed)
    m, n, k = _product_shape(rng, 1)
    mode = rng.choice(("rowwise", "per_tensor"))
    make = linear.make_whole if seed % 2 else linear.make
    t = make(m, n, k, mode, seed, bias=rng.random() < 0.7, residual=rng.random() < 0.5)
    linear.check(t, rng.choice(ACTS), preact=rng.random() < 0.5, mode=mode)


@pytest.mark.parametrize("seed", range(32))
def test_linear_backward(seed):
    rng = random.Random(200 + seed)
    m, n, k = _product_shape(rng, 16)
    if seed % 2 and 49 * max(m, n) < 2 ** 24:
        backward.check(backward.make_whole(m, n, k, seed), "none", whole=True)
    backward.check(backward.make(m, n, k, seed), rng.choice(ACTS))
