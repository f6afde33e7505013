"""The cross entropy and its gradient on every tile configuration of the multiply, with K
whole and split, against 64 bits (tolerances: test_gpu_cross_entropy and _backward)."""
import pytest
import torch

from precision_linear_amd import binding
from test_gpu_cross_entropy import check, make
from test_gpu_cross_entropy_backward import close, gradient64, more, run

pytestmark = pytest.mark.gpu

# Configuration, K split, and sizes whose automatic plan is that.
PLANS = [(0, True, 16, 1000, 16384), (1, False, 1, 16, 64), (1, True, 1, 16, 16384), (2, False, 16, 20000, 256),
         (3, False, 100, 4000, 64), (3, True, 64, 4000, 4096), (4, False, 129, 4000, 1024), (4, True, 64, 4000, 16384),
         (5, False, 64, 20000, 4096), (5, True, 300, 1000, 16384), (6, False, 1000, 1000, 4096), (7, False, 512, 4000, 4096),
         (7, True, 128, 4000, 16384), (8, False, 1000, 4000, 4096), (8, True, 256, 4000, 16384), (9, False, 1000, 4000, 256),
         (9, True, 128, 20000, 16384), (10, False, 1000, 1000, 64), (10, True, 17, 20000, 16384), (11, False, 512, 20000, 64),
         (11, True, 700, 5008, 16384), (11, True, 300, 12000, 12288)]


def test_the_list_has_every_configuration():
    assert {p[0] for p in PLANS} == set(range(len(binding.config_names())))


@pytest.mark.parametrize("config,split,M,V,K", PLANS)
def test_plan(config, split, M, V, K):
    print(f"[cross entropy plans] {config} {split} {M} x {V} x {K}", flush=True)
    n = (V + 15) // 16 * 16
    assert binding.select_config(M, n, K, "rowwise") == config
    assert (binding.select_splits(M, n, K, "rowwise") > 1) == split
    for fa, fb, v in (("e4m3fn", "e4m3fn", V), ("e5m2", "e4m3fn", V - 3 if V > 16 else V)):
        t = make(M, v, K, fa=fa, fb=fb, ignore=-100, seed=21, whole=True)
        check(*binding.fp8_linear_cross_entropy(*t), *t)
        args, got = run(t, more(t))
        close(got, gradient64(*args), (fa, v))
        # a second call on the same stream, its counters as the first left them
        again = binding.fp8_linear_cross_entropy_backward(*args)
        assert torch.equal(again[0], got[0]) and torch.equal(again[1], got[1])


@pytest.mark.parametrize("M,V,K", [(1001, 50255, 256), (300, 65536, 512), (200, 40000, 1040), (2000, 30000, 2048), (4, 40000, 64)])
def test_long_sums(M, V, K):
    """dx sums over vocabularies past the plan model's K: units joined by a second launch, and not."""
    print(f"[cross entropy plans] long sum {M} x {V} x {K}", flush=True)
    for fw in ("e4m3fn", "e5m2"):
        t = make(M, V, K, ignore=-100, seed=22, whole=True)
        args, got = run(t, more(t, fw=fw))
        close(got, gradient64(*args), fw)
        K8 = got[0].shape[1]
        # an output that allows no wide stores
        flat = torch.empty(M * K8 + 1, dtype=torch.bfloat16, device=got[0].device)[1:].view(M, K8)
        dx, _ = binding.fp8_linear_cross_entropy_backward(*args, dx=flat, dw=False)
        assert torch.equal(dx, got[0])
