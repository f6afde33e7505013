"""Host-side checks of the AdamW step's C ABI and binding: exports, structures and
every refusal before anything touches a device."""
import ctypes
import math
import os
import random
import re

import pytest
import torch

from precision_linear_amd import binding

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
P = 0x10000          # a 64 KiB-aligned fake device address, never dereferenced


@pytest.fixture(scope="module")
def L():
    if not os.path.exists(binding.library_path):
        from precision_linear_amd import build
        build.build()
    return binding.lib()


def test_exports_every_declared_function(L):
    text = open(os.path.join(ROOT, "include", "adamw.h")).read()
    text = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
    names = set(re.findall(r"\b(adamw_\w+)\s*\(", text))
    assert names == set(binding.ADAMW_EXPORTS)
    for n in names:
        assert hasattr(L, n), n


def test_status_strings(L):
    for s in range(9):
        assert L.adamw_status_string(s) != b"unknown status"
    assert L.adamw_status_string(9) == b"unknown status"


def test_structures_as_in_the_header():
    text = open(os.path.join(ROOT, "include", "adamw.h")).read()
    text = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
    for name, struct in (("adamw_tensor", binding._AdamwTensor), ("adamw_numbers", binding._AdamwNumbers)):
        body = re.search(r"struct %s \{(.*?)\}" % name, text, flags=re.S).group(1)
        fields = [f for line in body.split(";") for f in re.findall(r"\*?(\w+)(?:,|$)", line.strip())]
        assert fields == [f[0] for f in struct._fields_]


def tensor(i=0, **kw):
    at = lambda k: P * (8 * i + k + 1)                      # noqa: E731
    t = dict(param=at(0), grad=at(1), exp_avg=at(2), exp_avg_sq=at(3), master=None, exp_avg_scale=None,
             exp_avg_sq_scale=None, numel=1000)
    return binding._AdamwTensor(**{**t, **kw})


def call(L, tensors, pd=1, gd=1, bits=32, count=None, numbers=True, **kw):
    n = binding._AdamwNumbers(**{**dict(lr=1e-3, beta1=0.9, beta2=0.999, eps=1e-8, weight_decay=0.1, step=1), **kw})
    array = (binding._AdamwTensor * max(1, len(tensors)))(*tensors)
    return L.adamw_step(ctypes.byref(array), len(tensors) if count is None else count, pd, gd, bits,
                        ctypes.byref(n) if numbers else None, None)


E = binding


@pytest.mark.parametrize("t,kw,code", [
    ({}, dict(pd=2), E.ADAMW_ERR_DTYPE), ({}, dict(gd=-1), E.ADAMW_ERR_DTYPE), ({}, dict(bits=16), E.ADAMW_ERR_DTYPE),
    (dict(master=P * 7), dict(), E.ADAMW_ERR_DTYPE), ({}, dict(numbers=False), E.ADAMW_ERR_NULL),
    ({}, dict(count=-1), E.ADAMW_ERR_SHAPE), (dict(numel=-1), dict(), E.ADAMW_ERR_SHAPE),
    (dict(numel=1 << 44), dict(), E.ADAMW_ERR_SHAPE),
    (dict(param=None), dict(), E.ADAMW_ERR_NULL), (dict(grad=None), dict(), E.ADAMW_ERR_NULL),
    (dict(exp_avg=None), dict(), E.ADAMW_ERR_NULL), (dict(exp_avg_sq=None), dict(), E.ADAMW_ERR_NULL),
    (dict(exp_avg_scale=P), dict(), E.ADAMW_ERR_NULL), ({}, dict(bits=8), E.ADAMW_ERR_NULL),
    (dict(exp_avg_scale=P * 6), dict(bits=8), E.ADAMW_ERR_NULL),
    (dict(param=P + 2), dict(), E.ADAMW_ERR_ALIGN), (dict(param=P + 1), dict(pd=0), E.ADAMW_ERR_ALIGN),
    (dict(grad=P + 2), dict(), E.ADAMW_ERR_ALIGN), (dict(exp_avg=P + 2), dict(), E.ADAMW_ERR_ALIGN),
    (dict(master=P * 7 + 2), dict(pd=0), E.ADAMW_ERR_ALIGN),
    (dict(exp_avg_scale=P * 6 + 1, exp_avg_sq_scale=P * 7), dict(bits=8), E.ADAMW_ERR_ALIGN),
    (dict(exp_avg=P), dict(), E.ADAMW_ERR_ALIAS),
    ({}, dict(lr=-1.0), E.ADAMW_ERR_VALUE), ({}, dict(lr=math.inf), E.ADAMW_ERR_VALUE),
    ({}, dict(lr=math.nan), E.ADAMW_ERR_VALUE), ({}, dict(beta1=1.0), E.ADAMW_ERR_VALUE),
    ({}, dict(beta2=-0.5), E.ADAMW_ERR_VALUE), ({}, dict(beta2=math.nan), E.ADAMW_ERR_VALUE),
    ({}, dict(eps=-1.0), E.ADAMW_ERR_VALUE), ({}, dict(weight_decay=math.inf), E.ADAMW_ERR_VALUE),
    ({}, dict(step=0), E.ADAMW_ERR_VALUE), ({}, dict(lr_ptr=P + 2), E.ADAMW_ERR_ALIGN),
    ({}, dict(seed_ptr=P + 4), E.ADAMW_ERR_ALIGN),
])
def test_refusals(L, t, kw, code):
    assert call(L, [tensor(**t)], **kw) == code


def test_lists(L):
    assert call(L, [tensor(0), tensor(0)]) == E.ADAMW_ERR_ALIAS
    assert call(L, [tensor(0), tensor(1, exp_avg_sq=P * 4)]) == E.ADAMW_ERR_ALIAS
    assert call(L, [tensor(0, master=P * 7), tensor(1)], pd=0) == E.ADAMW_ERR_NULL
    if torch.cuda.is_available():
        pytest.skip("a GPU is present: these cases would launch on fake pointers")
    reached = (E.ADAMW_ERR_DEVICE, E.ADAMW_ERR_LAUNCH)
    assert call(L, [tensor(0), tensor(1)]) in reached
    assert call(L, [tensor(0, grad=P), tensor(1, grad=P)]) in reached
    assert call(L, [tensor(0)], step=0, step_ptr=P) in reached
    assert call(L, [tensor(0, exp_avg=P * 3 + 1, exp_avg_scale=P * 6, exp_avg_sq_scale=P * 7)], bits=8) in reached


@pytest.mark.parametrize("first,second,kw", [
    ({}, dict(param=P + 3996), {}), ({}, dict(exp_avg=P * 3 + 400), {}), (dict(exp_avg_sq=P * 3 + 3996), {}, {}),
    (dict(numel=1 << 20), dict(numel=4), {}),
    (dict(master=P * 7), dict(master=P * 7), dict(pd=0)), (dict(master=P * 7), dict(master=P * 7 + 3996), dict(pd=0)),
    (dict(exp_avg_scale=P * 6, exp_avg_sq_scale=P * 7), dict(exp_avg_scale=P * 6, exp_avg_sq_scale=P * 15), dict(bits=8)),
    (dict(exp_avg_scale=P * 6, exp_avg_sq_scale=P * 7), dict(exp_avg_scale=P * 14, exp_avg_sq_scale=P * 7 + 12), dict(bits=8)),
    (dict(exp_avg_scale=P * 6, exp_avg_sq_scale=P * 6 + 12), dict(exp_avg_scale=P * 14, exp_avg_sq_scale=P * 15), dict(bits=8)),
])
def test_what_overlaps_is_refused(L, first, second, kw):
    """1000 elements are 4000 bytes of fp32 and 16 of scales."""
    tensors = [tensor(0, **first), tensor(1, **second)]
    assert call(L, tensors, **kw) == E.ADAMW_ERR_ALIAS
    assert call(L, tensors[::-1], **kw) == E.ADAMW_ERR_ALIAS


def test_neighbours_are_taken(L):
    if torch.cuda.is_available():
        pytest.skip("a GPU is present: these cases would launch on fake pointers")
    reached = (E.ADAMW_ERR_DEVICE, E.ADAMW_ERR_LAUNCH)
    assert call(L, [tensor(0), tensor(1, param=P + 4000, exp_avg=P * 3 + 4000, exp_avg_sq=P * 4 + 4000)]) in reached
    assert call(L, [tensor(0), tensor(1, param=P, exp_avg=P, exp_avg_sq=P, numel=0)]) in reached


@pytest.mark.parametrize("empty", [{}, dict(param=None, grad=None, exp_avg=None, exp_avg_sq=None),
                                   dict(master=P * 7, exp_avg_scale=P * 6, exp_avg_sq_scale=P * 7)])
@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("master", [True, False])
def test_empty_tensors_anywhere(L, empty, bits, master):
    """Pointers of empty tensors (torch's are NULL) count neither for nor against masters, wherever they are."""
    if torch.cuda.is_available():
        pytest.skip("a GPU is present: these cases would launch on fake pointers")
    reached = (E.ADAMW_ERR_DEVICE, E.ADAMW_ERR_LAUNCH)
    more = dict(exp_avg_scale=P * 6, exp_avg_sq_scale=P * 7) if bits == 8 else {}
    full = tensor(0, **more, **(dict(master=P * 8) if master else {}))
    none = tensor(1, numel=0, **empty)
    for tensors in ([none, full], [full, none], [none, none, full, none], [none]):
        assert call(L, tensors, pd=0, bits=bits) in reached
    if master:
        assert call(L, [none, full], pd=1, bits=bits) == E.ADAMW_ERR_DTYPE
        assert call(L, [none, full, tensor(2, **more)], pd=0, bits=bits) == E.ADAMW_ERR_NULL


@pytest.mark.parametrize("kinds", ["bits 32", "masters", "bits 8", "bits 8, masters"])
@pytest.mark.parametrize("order", ["tensor by tensor", "kind by kind", "kinds side by side", "shuffled", "each kind shuffled"])
@pytest.mark.parametrize("count", [1, 2, 7, 40, 64, 131, 300])
def test_overlaps_among_many(L, count, order, kinds):
    """Ranges that touch are taken, one byte more is refused, whatever the order of the list."""
    rng = random.Random(f"{count} {order} {kinds}")
    bits, master = 8 if "8" in kinds else 32, "masters" in kinds
    names = ["param", "exp_avg", "exp_avg_sq"] + ["master"] * master + ["exp_avg_scale", "exp_avg_sq_scale"] * (bits == 8)
    numel = [rng.choice((1, 3, 256, 257, rng.randrange(1, 5000))) for _ in range(count)]
    size = lambda i, k: {"param": 2 * numel[i], "master": 4 * numel[i], "exp_avg": numel[i] * bits // 8,        # noqa: E731
                         "exp_avg_sq": numel[i] * bits // 8}.get(k, 4 * ((numel[i] + 255) // 256))
    spots = [(i, k) for i in range(count) for k in names]
    if order == "kinds side by side":              # one kind's between another's
        spots = [(i, k) for ks in (names[:2], names[2:]) for i in range(count) for k in ks]
    elif order != "tensor by tensor":
        spots.sort(key=lambda s: names.index(s[1]))
    if order == "each kind shuffled":
        rng.shuffle(spots)
    at, starts = 1 << 44, {}
    for i, k in spots:
        at = (at + 3) // 4 * 4 + rng.choice((0, 0, 4, 512, 1 << 30))
        starts[i, k] = at
        at += size(i, k)
    ranges = sorted((starts[s], starts[s] + size(*s), s) for s in spots)
    perm = list(range(count))
    if order == "shuffled":
        rng.shuffle(perm)

    def status(starts):
        return call(L, [tensor(0, numel=numel[i], **{k: starts[i, k] for k in names}) for i in perm], pd=0, bits=bits)

    if not torch.cuda.is_available():              # (a launch on these addresses would fault)
        assert status(starts) in (E.ADAMW_ERR_DEVICE, E.ADAMW_ERR_LAUNCH)
    for _ in range(30):
        (a, b, s), (c, d, t) = rng.choice([(x, y) for x, y in zip(ranges, ranges[1:])])
        if rng.random() < 0.5:                     # the later one begins in the earlier one's last bytes
            c = (b - 1) // 4 * 4
            assert status(starts | {t: c}) == E.ADAMW_ERR_ALIAS
        else:                                      # any two begin at one address
            x, y = rng.sample(spots, 2)
            assert status(starts | {x: starts[y]}) == E.ADAMW_ERR_ALIAS


def test_binding_refuses_before_the_library():
    p, g = [torch.zeros(4)], [torch.zeros(4)]
    for args in ((p, g, g, g), (p, [], g, g), ([3], g, g, g), (p, g, [], g)):
        with pytest.raises(ValueError):
            binding.adamw_step(*args, step=1, lr=0.1)
    with pytest.raises(ValueError):
        binding.adamw_state(p)
    assert binding.adamw_step([], [], [], [], step=1, lr=0.1) is None
