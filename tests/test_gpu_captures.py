"""Graphs captured on a stream whose workspaces do not exist yet, replayed in
another order than captured and beside each other; eager calls on the capturing
stream.  Every result has the bits of the eager call."""
import pytest
import torch

from precision_linear_amd import binding
from test_gpu_layer_norm import make as make_norm
from test_gpu_linear import make as make_linear, to_dev
from test_gpu_linear_backward import make as make_grad

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF16 = torch.bfloat16


def linear(seed):
    t = to_dev(make_linear(128, 1024, 8192, "rowwise", seed))
    assert binding.select_splits(128, 1024, 8192, "rowwise", True) > 1
    return lambda: (binding.fp8_linear(**t, activation="silu"),)


def multiply(seed):
    t = to_dev(make_linear(64, 2048, 8192, "rowwise", seed, residual=False))
    del t["residual"]
    assert binding.select_splits(64, 2048, 8192, "rowwise", True) > 1
    return lambda: (binding.fp8_scaled_mm(**t, mode="rowwise"),)


def linear_backward(seed):
    args = [t.to(DEV) for t in make_grad(64, 4096, 1024, seed)]
    return lambda: binding.fp8_linear_backward(*args, activation="gelu")


def layer_norm_backward(seed):
    x, w, _ = (t.to(DEV) for t in make_norm(2000, 1000, BF16, seed))
    dy = make_norm(2000, 1000, BF16, seed + 50)[0].to(DEV)
    st = binding.fp8_layer_norm(x, stats=True)
    return lambda: binding.fp8_layer_norm_backward(dy, x, st.mean, st.rstd, w)


def quantize(seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    x = torch.randn(4099, 8192, generator=g, device=DEV).to(BF16)        # (large enough for one pass)
    return lambda: binding.fp8_quantize(x, "per_tensor")


def capture(stream, call):
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        outs = call()
    return graph, outs


def check(outs, want, what):
    torch.cuda.synchronize()
    for i, (a, b) in enumerate(zip(outs, want)):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8)), (what, i)


OPERATORS = [linear, multiply, linear_backward, layer_norm_backward, quantize]


@pytest.mark.parametrize("path", ["short", "whole"])
@pytest.mark.parametrize("make", OPERATORS)
def test_graphs_of_a_fresh_stream_replayed_in_reverse_order(monkeypatch, make, path):
    binding.lib()
    if path == "whole":
        monkeypatch.setattr(binding, "_calls", None)
    calls = [make(seed) for seed in (1, 2, 3)]
    want = [call() for call in calls]
    torch.cuda.synchronize()
    print(f"[captures] {make.__name__} {path}", flush=True)
    fresh = torch.cuda.Stream()
    graphs = [capture(fresh, call) for call in calls[:2]]
    with torch.cuda.stream(fresh):                      # an eager call there, before any replay
        check(calls[2](), want[2], "eager")
    for rep in range(3):
        for i in (1, 0):
            graph, outs = graphs[i]
            for t in outs:
                t.zero_()
            junk = torch.randn(256, 256, device=DEV) @ torch.randn(256, 256, device=DEV)
            torch.cuda.synchronize()
            graph.replay()
            check(outs, want[i], (rep, i))
            del junk
        with torch.cuda.stream(fresh):
            check(calls[2](), want[2], ("eager", rep))


@pytest.mark.parametrize("make", OPERATORS)
def test_graphs_of_one_stream_replayed_beside_each_other(make):
    calls = [make(seed) for seed in (4, 5)]
    want = [call() for call in calls]
    torch.cuda.synchronize()
    print(f"[captures] {make.__name__} side by side", flush=True)
    fresh = torch.cuda.Stream()
    graphs = [capture(fresh, call) for call in calls]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for rep in range(3):
        for _, outs in graphs:
            for t in outs:
                t.zero_()
        torch.cuda.synchronize()
        for _ in range(10):
            for (graph, _), stream in zip(graphs, streams):
                with torch.cuda.stream(stream):
                    graph.replay()
        for i in range(2):
            check(graphs[i][1], want[i], (rep, i))


def test_a_capture_of_many_calls_has_one_workspace():
    call = linear(6)
    want = call()
    fresh = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    before = torch.cuda.memory_allocated()
    with torch.cuda.graph(graph, stream=fresh):
        outs = [call() for _ in range(6)]
    grown = torch.cuda.memory_allocated() - before
    need = binding.workspace_size(128, 1024, 8192, "rowwise", True)
    assert grown < 2 * need + 6 * 2 * 128 * 1024 + (2 << 20)
    for _ in range(2):
        graph.replay()
        for o in outs:
            check(o, want, "replay")
