"""Whose workspace a call gets (CPU): the module's for the stream, or, while a
graph is captured, one of that capture's own, since its fill is then recorded
and not run and since the graph may be replayed beside other work."""
import torch

from precision_linear_amd import binding

CPU = torch.device("cpu")


def workspace(monkeypatch, capture, nbytes=1000, kind="mm", stream=1 << 50):
    monkeypatch.setattr(binding, "_capture_id", lambda device, stream: capture, raising=False)
    return binding._workspace(CPU, stream, nbytes, kind)


def test_a_capture_has_its_own(monkeypatch):
    monkeypatch.setattr(binding, "_workspaces", {})
    monkeypatch.setattr(binding, "_captured", {}, raising=False)
    for kind in ("mm", "layer_norm", "quantize"):
        first = workspace(monkeypatch, 7, kind=kind)
        assert workspace(monkeypatch, 7, kind=kind) is first              # the calls of one capture share it
        assert workspace(monkeypatch, 7, kind=kind, stream=5) is not first
        second = workspace(monkeypatch, 8, kind=kind)
        eager = workspace(monkeypatch, None, kind=kind)                   # its fill has to run
        assert first is not second and eager is not first and eager is not second
        assert workspace(monkeypatch, None, kind=kind) is eager
        third = workspace(monkeypatch, 9, kind=kind)
        assert third is not eager and third is not second
        assert workspace(monkeypatch, 9, kind=kind) is third
        larger = workspace(monkeypatch, 9, 10 << 20, kind=kind)
        assert larger.numel() >= 10 << 20 and workspace(monkeypatch, 9, kind=kind) is larger


def test_a_capture_with_an_id_of_zero_is_one(monkeypatch):
    monkeypatch.setattr(binding, "_workspaces", {})
    monkeypatch.setattr(binding, "_captured", {}, raising=False)
    assert workspace(monkeypatch, 0) is not workspace(monkeypatch, None)
