"""Outputs of the linear layer's gradient asked for alone, on every path of the
quantisation: joined in 64-row and in 128-row tiles, not joined (over 64 column
blocks), with longer strips, with the slope table and without, with the
non-temporal hints and without.

What is asked for may change the plan, and with it the order of fp32 sums.  Whole
numbers (test_gpu_linear_backward's) are exact in any order, so there every output
has the same bits alone; the activations' outputs keep to that file's bounds
against 64 bits.
"""
import pytest
import torch

from precision_linear_amd import binding
from test_gpu_linear_backward import DEV, HALF, make, make_whole, reference, within

pytestmark = pytest.mark.gpu
SHAPES = [(300, 272, 144), (130, 8336, 32), (1100, 7296, 48), (700, 7984, 8208), (17000, 96, 1040), (2000, 28672, 64),
          (2400, 28672, 64)]
ASKED = [(1, 0, 0), (0, 1, 0), (0, 0, 1), (1, 1, 0), (1, 0, 1), (0, 1, 1), (1, 1, 1)]


def parts(args, act):
    """(asked, outputs) of every choice of outputs, with nothing given that they do not need."""
    dy, x, wt, sw, z = (t.to(DEV) for t in args)
    for asked in ASKED:
        dx, dw, db = map(bool, asked)
        print(f"[linear_backward] {asked} of {dy.shape[0]} x {dy.shape[1]} x {x.shape[1]} {act}", flush=True)
        got = binding.fp8_linear_backward(dy, x if dw else None, wt if dx else None, sw if dx else None,
                                          None if act == "none" else z, activation=act, dx=dx, dw=dw, dbias=db)
        assert [t is not None for t in got] == [dx, dw, db]
        yield asked, got


@pytest.mark.parametrize("act", ["none", "relu"])
@pytest.mark.parametrize("M,N,K", SHAPES)
def test_whole_numbers(M, N, K, act):
    args = make_whole(M, N, K, 5)
    if act == "relu":                                    # keep the sevens
        dy, x, wt, sw, z = args
        args = (dy, x, wt, sw, torch.where(dy == 7, z.abs() + 1, z))
    got = dict(parts(args, act))
    for asked, outs in got.items():
        for i in range(3):
            assert not asked[i] or torch.equal(outs[i], got[1, 1, 1][i]), (asked, i)


@pytest.mark.parametrize("act", ["gelu", "silu"])
@pytest.mark.parametrize("M,N,K", SHAPES)
def test_activations(M, N, K, act):
    args = make(M, N, K, 6)
    ref = reference(*args, act, False)
    for asked, outs in parts(args, act):
        for name, got, (want, err), half in zip(("dx", "dw", "dbias"), outs, ref, (HALF, HALF, 0.0)):
            if got is not None:
                within(f"{name} of {asked}", got, want, err + half * (want.abs() + err))
