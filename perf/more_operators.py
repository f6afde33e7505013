"""The operators of a training step behind the blocks, as cases that can be timed
and compared: the softmax cross entropy of an FP8 linear layer over a large
vocabulary, its gradient, the AdamW step over many tensors, and the codes of a
weight in the two layouts that the next step's products take.

Formulas (M rows, a vocabulary of V, K features):

  loss       z = s sum_k A[m, k] B[j, k]
             lse = log sum_j exp(z), loss = lse - z[target] (0 for ignored rows)
  loss_grad  p = exp(z - lse), h = 1 - p[target] = -expm1(-loss)
             q = e5m2(57344 p / h), -57344 at the target, 0 in ignored rows
             dx = dloss h / 57344 * sum_j q W          (W in e4m3, a scale a column)
             xr = x dloss h, in e4m3 with one scale a column
             dw = sum_m q xr / 57344
  adamw      m = b1 m + (1 - b1) g, v = b2 v + (1 - b2) g^2
             p = p (1 - lr wd) - lr / (1 - b1^t) m / (sqrt(v / (1 - b2^t)) + eps)
             with the moments in 32 bits, or m and sqrt(v) in e4m3, one scale
             for each block of 256 elements of a tensor, rounded to one of the
             two neighbours at random (sqrt(v) > 0 never to 0)
  codes      scale = max |w| / 448 for each row, q = e4m3(w / scale), and the
             same for each column, transposed

`own` selects what run() calls: the plain form below, or the package.
"""
import math

import torch

own = False

E4M3_MAX = 448.0
E5M2_MAX = 57344.0
IGNORE = -100
BLOCK = 256
BETA1, BETA2, EPS, DECAY, RATE = 0.9, 0.999, 1e-8, 0.1, 1e-3
DTYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}


# ------------------------------------------------------------------ cases ---

def listed():
    return [
        # Scoring the next token of one sequence: latency.
        dict(name="loss_token", op="loss", m=1, v=32000, k=2048, mode="rowwise", ignored=False),
        # An evaluation batch over a vocabulary of no round size, padded rows ignored.
        dict(name="loss_odd", op="loss", m=1000, v=50255, k=2048, mode="per_tensor", ignored=True),
        # A training step's tokens over a large vocabulary.
        dict(name="loss_train", op="loss", m=8192, v=131072, k=4096, mode="rowwise", ignored=False),
        # A short fine-tuning batch of a small model.
        dict(name="loss_grad_short", op="loss_grad", m=100, v=32000, k=1024, mode="rowwise", ignored=False),
        # The evaluation batch's sizes in training: odd vocabulary, odd rows, some of them ignored.
        dict(name="loss_grad_odd", op="loss_grad", m=1001, v=50255, k=2048, mode="rowwise", ignored=True),
        # A training step's tokens over a large vocabulary.
        dict(name="loss_grad_train", op="loss_grad", m=8192, v=131072, k=4096, mode="rowwise", ignored=True),
        # The norms and biases of one block: latency.
        dict(name="adamw_vectors", op="adamw", tensors=6, largest=28672, param="fp32", grad="fp32", master=False,
             bits=32),
        # All the small and middling tensors of a model, of any size: bf16 weights with fp32 masters.
        dict(name="adamw_many", op="adamw", tensors=150, largest=1500000, param="bf16", grad="bf16", master=True,
             bits=32),
        # Both matrices of a large feed-forward block, fp32 weights, bf16 gradients.
        dict(name="adamw_block", op="adamw", tensors=2, largest=28672 * 8192, param="fp32", grad="bf16",
             master=False, bits=32),
        # The same with the moments in 8 bits.
        dict(name="adamw_block_8bit", op="adamw", tensors=2, largest=28672 * 8192, param="fp32", grad="bf16",
             master=False, bits=8),
        # A projection of a small model, bf16 weights, rows that end inside a tile.
        dict(name="codes_odd", op="codes", n=1000, k=4160, dtype="bf16"),
        # The up projection of a large block, from its fp32 master.
        dict(name="codes_block", op="codes", n=28672, k=8192, dtype="fp32"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("loss", "loss_grad", "adamw", "codes"))
    if op in ("loss", "loss_grad"):
        while True:
            m, v, k = _log(rng, 1, 16384), _log(rng, 1000, 262144), max(64, _log(rng, 64, 8192) // 16 * 16)
            if rng.random() < 0.5:
                v = v // 16 * 16
            if m * v <= 8192 * 131072 and m * v * k <= 8192 * 131072 * 4096:
                break
        return dict(op=op, m=m, v=v, k=k, mode=rng.choice(("rowwise", "rowwise", "per_tensor")),
                    ignored=rng.random() < 0.5)
    if op == "adamw":
        while True:
            tensors, largest = _log(rng, 1, 300), _log(rng, 1, 28672 * 8192)
            if tensors * largest <= 2 * 28672 * 8192:
                break
        param = rng.choice(("fp32", "bf16"))
        return dict(op=op, tensors=tensors, largest=largest, param=param, grad=rng.choice(("bf16", "fp32")),
                    master=param == "bf16" and rng.random() < 0.7, bits=rng.choice((8, 32)))
    while True:
        n, k = _log(rng, 1, 65536), max(16, _log(rng, 16, 28672) // 16 * 16)
        if n * k <= 28672 * 8192:
            break
    return dict(op=op, n=n, k=k, dtype=rng.choice(("bf16", "fp32")))


def _sizes(case):
    """Elements of each tensor: the largest first, the others spread below it, most of them odd."""
    n, largest = case["tensors"], case["largest"]
    if largest >= 1 << 24:
        return [largest] * n
    return [max(1, int(largest * ((i * 0.6180339887498949) % 1.0 if i else 1.0))) for i in range(n)]


def _up(n, to):
    return -(-n // to) * to


def work(case):
    op = case["op"]
    if op in ("loss", "loss_grad"):
        m, v, k = case["m"], case["v"], case["k"]
        scales = 4 * (m + v) if case["mode"] == "rowwise" else 8
        read = m * k + v * k + scales + 8 * m
        if op == "loss":
            return {"bytes": read + 8 * m, "flops": 2 * m * v * k}
        return {"bytes": read + 12 * m + v * k + 4 * k + 2 * m * k + 2 * m * k + 2 * v * k, "flops": 6 * m * v * k}
    if op == "adamw":
        n = sum(_sizes(case))
        size = {"bf16": 2, "fp32": 4}
        param = size[case["param"]] + 8 if case["master"] else 2 * size[case["param"]]
        states = 16 if case["bits"] == 32 else 4 + 16 / BLOCK
        return {"bytes": n * (param + size[case["grad"]] + states), "flops": 16 * n}
    n, k = case["n"], case["k"]
    return {"bytes": n * k * ({"bf16": 2, "fp32": 4}[case["dtype"]] + 2) + 4 * (n + k), "flops": 4 * n * k}


# ----------------------------------------------------------------- inputs ---

def _generator(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    return g


def _normal(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda", dtype=torch.float32)


def _codes(x, qmax, dtype, axis):
    """(codes, scale) of x with one scale for each row (axis 1), column (axis 0) or tensor (None)."""
    amax = x.abs().amax() if axis is None else x.abs().amax(dim=axis, keepdim=True)
    scale = amax / torch.full_like(amax, qmax)      # (a division by a number may multiply by its reciprocal)
    q = torch.where(scale > 0, x / scale, torch.zeros_like(x)).clamp(-qmax, qmax)
    return q.to(dtype), scale.reshape(-1)


def _prepare_loss(case, g):
    m, v, k = case["m"], case["v"], case["k"]
    w = 0.02 * _normal(g, v, k)
    target = torch.randint(0, v, (m,), generator=g, device="cuda")
    x = _normal(g, m, k)
    # What the model has learnt: the target's logit is higher by 0 (the first row's, so
    # that no batch has losses next to 0 alone, where 32 bits of a logit are few) to 18.
    rise = 18.0 * torch.rand(m, 1, generator=g, device="cuda")
    rise[0] = 0.0
    x += w[target] * (rise / (0.0004 * k))
    if case["ignored"]:
        out = torch.rand(m, generator=g, device="cuda") < 0.1
        out[0] = False
        target[out] = IGNORE
    x = x.bfloat16()
    axis = 1 if case["mode"] == "rowwise" else None
    s = {"target": target, "case": case, "op": case["op"]}
    s["a"], s["sa"] = _codes(x.float(), E4M3_MAX, torch.float8_e4m3fn, axis)
    s["b"], s["sb"] = _codes(w, E4M3_MAX, torch.float8_e4m3fn, axis)
    if case["op"] == "loss":
        return s
    s["x"] = x
    # W transposed (k x v, rows of whole 16 bytes), laid out once for each update of the weights.
    wt, s["swt"] = _codes(w.t(), E4M3_MAX, torch.float8_e4m3fn, 1)
    s["wt"] = torch.zeros(k, _up(v, 16), dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)
    s["wt"].view(torch.uint8)[:, :v] = wt.view(torch.uint8)
    del w, wt
    # Of the mean over the rows that count, by weights of about 1.
    s["dloss"] = (0.5 + torch.rand(m, generator=g, device="cuda")) / m
    z = _logits(s)
    s["lse"] = torch.logsumexp(z, 1)
    s["loss"] = _pick(s["lse"][:, None] - z, target)
    return s


def _prepare_adamw(case, g):
    sizes = _sizes(case)
    starts = [0]
    for n in sizes:
        starts.append(starts[-1] + _up(n, BLOCK))
    total = starts[-1]
    live = torch.zeros(total, dtype=torch.bool, device="cuda")
    for at, n in zip(starts, sizes):
        live[at:at + n] = True
    # Tensors lie in flat buffers, each from a whole block on.
    p = torch.where(live, 0.02 * _normal(g, total), 0.0)
    # Gradients of rows that learn at different speeds.
    grad = torch.where(live, 1e-3 * _normal(g, total) * torch.exp(_normal(g, total // BLOCK)).repeat_interleave(BLOCK), 0.0)
    mean = 0.3 * grad + torch.where(live, 2e-4 * _normal(g, total), 0.0)
    square = torch.where(live, (1e-3 * _normal(g, total)) ** 2 + 0.5 * grad * grad, 0.0)
    del live
    s = {"case": case, "op": "adamw", "step": 100, "seed": int(torch.randint(0, 1 << 31, (), generator=g, device="cuda"))}
    s["p"] = p.to(DTYPES[case["param"]])
    s["master"] = p if case["master"] else None
    s["grad"] = grad.to(DTYPES[case["grad"]])
    if case["bits"] == 32:
        s["m"], s["v"] = mean, square
    else:
        s["m"], s["m_scale"] = _codes(mean.view(-1, BLOCK), E4M3_MAX, torch.float8_e4m3fn, 1)
        s["v"], s["v_scale"] = _codes(square.sqrt().view(-1, BLOCK), E4M3_MAX, torch.float8_e4m3fn, 1)
        s["m"], s["v"] = s["m"].view(-1), s["v"].view(-1)
    views = lambda t: None if t is None else [t[a:a + n] for a, n in zip(starts, sizes)]  # noqa: E731
    blocks = lambda t: None if t is None else [t[a // BLOCK:b // BLOCK] for a, b in zip(starts, starts[1:])]  # noqa: E731
    s["lists"] = {k: views(s[k]) for k in ("p", "grad", "m", "v", "master")}
    s["lists"] |= {k: blocks(s.get(k)) for k in ("m_scale", "v_scale")}
    return s


def prepare(case, seed):
    g = _generator(seed)
    if case["op"] in ("loss", "loss_grad"):
        return _prepare_loss(case, g)
    if case["op"] == "adamw":
        return _prepare_adamw(case, g)
    # Rows and columns of different size.
    w = 0.02 * _normal(g, case["n"], case["k"]) * torch.exp(0.3 * _normal(g, case["n"], 1))
    return {"op": "codes", "case": case, "w": (w * torch.exp(0.3 * _normal(g, 1, case["k"]))).to(DTYPES[case["dtype"]])}


# ------------------------------------------------------------- plain form ---

def _logits(s):
    z = s["a"].float() @ s["b"].float().t()
    return z * (s["sa"][:, None] * s["sb"][None, :] if s["case"]["mode"] == "rowwise" else s["sa"] * s["sb"])


def _pick(rows, target):
    """rows[m, target[m]], 0 for ignored rows."""
    kept = target != IGNORE
    return torch.where(kept, rows.gather(1, torch.where(kept, target, 0)[:, None])[:, 0], 0.0)


def _plain_loss(s):
    z = _logits(s)
    most = z.amax(1, keepdim=True)
    lse = torch.exp(z - most).sum(1, keepdim=True).log() + most
    return {"loss": _pick(lse - z, s["target"]), "lse": lse[:, 0]}


def _plain_loss_grad(s):
    target, v = s["target"], s["case"]["v"]
    kept = target != IGNORE
    h = torch.where(kept, -torch.expm1(-s["loss"]), 0.0)
    q = torch.exp(_logits(s) - s["lse"][:, None])
    q *= torch.where(h > 0, E5M2_MAX / h, 0.0)[:, None]
    q.clamp_(max=E5M2_MAX)
    rows = torch.arange(len(target), device=target.device)
    q[rows, torch.where(kept, target, 0)] = torch.where(kept & (h > 0), -E5M2_MAX, 0.0)
    q = q.to(torch.float8_e5m2).float()
    r = s["dloss"] * h
    dx = (q @ s["wt"][:, :v].float().t()) * ((r / E5M2_MAX)[:, None] * s["swt"][None, :])
    xc, sx = _codes(s["x"].float() * r[:, None], E4M3_MAX, torch.float8_e4m3fn, 0)
    dw = (q.t() @ xc.float()) * (sx / E5M2_MAX)
    return {"dx": dx.bfloat16(), "dw": dw.bfloat16()}


def _random(seed, n):
    """n numbers of 32 bits (in int64)."""
    low = 0xffffffff
    x = (torch.arange(n, device="cuda") * 0x6A09E667 + seed * 0xBB67AE85 % (1 << 32)) & low
    x = ((x ^ (x >> 15)) * 0x3C6EF373) & low
    x = ((x ^ (x >> 13)) * 0xA54FF53B) & low
    return x ^ (x >> 16)


def _codes_at_random(x, r, positive):
    """(codes, scales) of x in e4m3, a scale for each block; rounded up where the part
    of the step that x reaches, and r / 2^16, make a whole one."""
    b = x.view(-1, BLOCK)
    amax = b.abs().amax(1, keepdim=True)
    scale = amax / torch.full_like(amax, E4M3_MAX)
    scale = torch.where(scale < 2.0 ** -100, 0.0, scale)
    y = (b * torch.where(scale > 0, 1 / scale, 0.0)).view(-1)
    t = y.abs().clamp(max=E4M3_MAX)
    lift = torch.where(t < 2.0 ** -6, 2.0 ** -6, 0.0)       # (below, the steps are those of 2^-6)
    t = (((t + lift).view(torch.int32) + (r << 4).to(torch.int32)) & ~0xfffff).view(torch.float32) - lift
    if positive:
        t = torch.where((y > 0) & (t == 0), 2.0 ** -9, t)
    return torch.copysign(t, y).to(torch.float8_e4m3fn), scale[:, 0]


def _plain_adamw(s):
    case = s["case"]
    s["step"] += 1
    g = s["grad"].float()
    if case["bits"] == 32:
        m, v = s["m"], s["v"]
    else:
        m = (s["m"].float().view(-1, BLOCK) * s["m_scale"][:, None]).view(-1)
        v = (s["v"].float().view(-1, BLOCK) * s["v_scale"][:, None]).view(-1).square()
    m = BETA1 * m + (1 - BETA1) * g
    v = BETA2 * v + (1 - BETA2) * (g * g)
    p = (s["p"] if s["master"] is None else s["master"]).float()
    root = v.sqrt()
    p = p * (1 - RATE * DECAY) - (RATE / (1 - BETA1 ** s["step"])) * (
        m / (root * (1 / math.sqrt(1 - BETA2 ** s["step"])) + EPS))
    if case["bits"] == 32:
        s["m"].copy_(m)
        s["v"].copy_(v)
    else:
        r = _random(s["seed"] + s["step"], p.numel())
        for name, x, bits in (("m", m, r & 0xffff), ("v", root, r >> 16)):
            q, scale = _codes_at_random(x, bits, name == "v")
            s[name].view(torch.uint8).copy_(q.view(torch.uint8))
            s[name + "_scale"].copy_(scale)
    s["p"].copy_(p)
    if s["master"] is not None:
        s["master"].copy_(p)
    return _adamw_outputs(s)


def _adamw_outputs(s):
    return {k: s[k] for k in ("p", "m", "v", "master", "m_scale", "v_scale") if s.get(k) is not None}


def _plain_codes(s):
    w = s["w"].float()
    q, scale = _codes(w, E4M3_MAX, torch.float8_e4m3fn, 1)
    qt, scale_t = _codes(w.t(), E4M3_MAX, torch.float8_e4m3fn, 1)
    return {"q": q, "scale": scale, "qt": qt, "scale_t": scale_t}


def _own_run(s):
    from precision_linear_amd import binding
    op, case = s["op"], s["case"]
    if op == "loss":
        loss, lse = binding.fp8_linear_cross_entropy(s["a"], s["b"], s["sa"], s["sb"], s["target"],
                                                     ignore_index=IGNORE, mode=case["mode"])
        return {"loss": loss, "lse": lse}
    if op == "loss_grad":
        dx, dw = binding.fp8_linear_cross_entropy_backward(
            s["dloss"], s["a"], s["b"], s["sa"], s["sb"], s["target"], s["loss"], s["lse"], s["x"], s["wt"], s["swt"],
            ignore_index=IGNORE, mode=case["mode"])
        return {"dx": dx, "dw": dw}
    if op == "adamw":
        s["step"] += 1
        t = s["lists"]
        binding.adamw_step(t["p"], t["grad"], t["m"], t["v"], step=s["step"], lr=RATE, betas=(BETA1, BETA2), eps=EPS,
                           weight_decay=DECAY, master=t["master"], exp_avg_scale=t["m_scale"],
                           exp_avg_sq_scale=t["v_scale"], seed=s["seed"] + s["step"])
        return _adamw_outputs(s)
    q, scale, qt, scale_t = binding.fp8_quantize_weight(s["w"])
    qt = qt[:, :case["n"]]          # (rows of qt are whole 16 bytes)
    return {"q": q.view(torch.float8_e4m3fn), "scale": scale, "qt": qt.view(torch.float8_e4m3fn), "scale_t": scale_t}


def run(state):
    if own:
        return _own_run(state)
    return {"loss": _plain_loss, "loss_grad": _plain_loss_grad, "adamw": _plain_adamw,
            "codes": _plain_codes}[state["op"]](state)


# ---------------------------------------------------------------- 64 bits ---

def _nearest_float8(v, mantissa, least, qmax):
    """Nearest value with `mantissa` fraction bits and exponents from `least` on, ties to even."""
    v = v.clamp(-qmax, qmax)
    _, e = torch.frexp(v)
    step = torch.ldexp(torch.ones_like(v), (e - 1).clamp(min=least) - mantissa)
    return torch.round(v / step) * step


def _exact_scaled(v, axis):
    """(values of v's e4m3 codes, their scale).  Scale and quotient are rounded to
    32 bits, as the codes are defined: inputs of few bits put many quotients
    next to a tie between two codes."""
    s = (v.abs().amax(axis, keepdim=True) / E4M3_MAX).float().double()
    t = torch.where(s > 0, v / s, torch.zeros_like(v)).float().double()
    return _nearest_float8(t, 3, -6, E4M3_MAX), s


def _exact_logits(s):
    wide = (slice(None), None) if s["case"]["mode"] == "rowwise" else (None, slice(None))
    a = s["a"].double().mul_(s["sa"].double()[wide])
    return torch.mm(a, s["b"].double().mul_(s["sb"].double()[wide]).t())


def _exact_loss(s):
    z = _exact_logits(s)
    lse = torch.logsumexp(z, 1)
    at = s["target"].clamp(min=0)
    loss = lse - z[torch.arange(len(at), device=at.device), at]
    return {"loss": loss * (s["target"] != IGNORE), "lse": lse}


def _exact_loss_grad(s):
    kept = s["target"] != IGNORE
    h = (1 - torch.exp(-s["loss"].double())) * kept
    q = _exact_logits(s).sub_(s["lse"].double()[:, None]).exp_()
    q *= torch.where(h > 0, E5M2_MAX / h, torch.zeros_like(h))[:, None]
    hot = torch.nn.functional.one_hot(s["target"][kept], s["case"]["v"]).bool()
    q[kept] = torch.where(hot, -E5M2_MAX * (h[kept] > 0).double()[:, None], q[kept])
    del hot
    q = _nearest_float8(q, 2, -14, E5M2_MAX)
    r = s["dloss"].double() * h
    wt = s["wt"][:, :s["case"]["v"]].double().mul_(s["swt"].double()[:, None])
    dx = torch.mm(q, wt.t()) * (r / E5M2_MAX)[:, None]
    del wt
    xc, sx = _exact_scaled(s["x"].double() * r[:, None], 0)
    return {"dx": dx, "dw": torch.mm(q.t(), xc * (sx / E5M2_MAX))}


def _exact_state(x, r, positive):
    b = x.view(-1, BLOCK)
    scale = b.abs().amax(1, keepdim=True) / E4M3_MAX
    y = torch.where(scale > 0, b / scale, torch.zeros_like(b)).view(-1)
    t = y.abs().clamp(max=E4M3_MAX)
    _, e = torch.frexp(t)
    step = torch.ldexp(torch.ones_like(t), (e - 1).clamp(min=-6) - 3)
    t = torch.floor(t / step + r.double() / 65536) * step
    if positive:
        t = torch.where(y > 0, t.clamp(min=2.0 ** -9), t)
    return t * torch.sign(y), scale[:, 0]


def _exact_adamw(s):
    case, t = s["case"], s["step"] + 1
    m, v = s["m"].double(), s["v"].double()
    if case["bits"] == 8:
        m = (m.view(-1, BLOCK) * s["m_scale"].double()[:, None]).view(-1)
        v = (v.view(-1, BLOCK) * s["v_scale"].double()[:, None]).view(-1).square_()
    g = s["grad"].double()
    m = torch.lerp(g, m, BETA1)
    v = torch.lerp(g.square(), v, BETA2)
    del g
    p = (s["p"] if s["master"] is None else s["master"]).double()
    down = (v / (1 - BETA2 ** t)).sqrt_().add_(EPS)
    p = p - RATE * (DECAY * p + m / (1 - BETA1 ** t) / down)
    del down
    out = {"p": p}
    if case["master"]:
        out["master"] = p
    if case["bits"] == 32:
        return out | {"m": m, "v": v}
    r = _random(s["seed"] + t, p.numel())
    out["m"], out["m_scale"] = _exact_state(m, r & 0xffff, False)
    out["v"], out["v_scale"] = _exact_state(v.sqrt_(), r >> 16, True)
    return out


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "codes":
        w = s["w"].double()
        q, scale = _exact_scaled(w, 1)
        qt, scale_t = _exact_scaled(w.t(), 1)
        return {"q": q, "scale": scale[:, 0], "qt": qt, "scale_t": scale_t[:, 0]}
    return {"loss": _exact_loss, "loss_grad": _exact_loss_grad, "adamw": _exact_adamw}[case["op"]](s)
