"""Workloads of what surrounds the 8-bit linear layer where it serves and learns: the root-mean-square
norm with the residual's addition, its gradient, the low-rank adapters of many requests beside the
layer, their gradients, and the AdamW step over many tensors.

Each case is one call a program makes.  ``run`` computes it with elementary torch operations, or,
where ``own`` is true, through the package's binding; ``exact`` restates it in 64 bits.
"""
import math

import torch

own = False

EPS = 1e-6
TINY = 2.0 ** -100  # a row or block whose largest magnitude is below this is quantised as if it were this
DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
BLOCK = 256         # values of an 8-bit state that share a scale
MOST_8 = 448.0      # the largest value of float8_e4m3fn
BETA1, BETA2, ADAM_EPS, DECAY = 0.9, 0.999, 1e-8, 0.01
MOST_NORM = 16384 * 4096                # elements of a norm case
MOST_ADAPTED = 8192 * (4096 + 16384)    # rows times channels read and written of an adapter case
MOST_WEIGHTS = 64 * 16 * 8192           # elements of its adapters
MOST_STEPPED = 96 << 20                 # elements of an AdamW case

_capi = None


def _binding():
    global _capi
    if _capi is None:
        from conv2d_batchnorm_silu_gb300 import capi
        _capi = capi
    return _capi


def listed():
    return [
        # One decoding step of a batch: the residual's addition, the norm, and its rows both as int8 for the shared
        # projection and in 16 bits for the adapters beside it.
        {"name": "add norm both 64x4096", "op": "rms_norm", "rows": 64, "c": 4096, "dtype": "bf16", "pad": 0,
         "residual": True, "out": "both"},
        # An odd channel count in column slices of wider tensors: rows without 16-byte alignment.
        {"name": "add norm 3001x777 slice", "op": "rms_norm", "rows": 3001, "c": 777, "dtype": "f16", "pad": 23,
         "residual": True, "out": "y"},
        # A long prompt's wide tokens: memory traffic alone counts.
        {"name": "add norm 16384x4096", "op": "rms_norm", "rows": 16384, "c": 4096, "dtype": "bf16", "pad": 0,
         "residual": True, "out": "y"},
        # The gradient at the pixels of a 16x40x40x256 feature map.
        {"name": "norm grad 25600x256", "op": "rms_norm_backward", "rows": 25600, "c": 256, "dtype": "bf16", "pad": 0,
         "residual": False},
        # The gradient of a long batch of wide tokens, with the one that arrives past the norm added.
        {"name": "add norm grad 16384x4096", "op": "rms_norm_backward", "rows": 16384, "c": 4096, "dtype": "bf16", "pad": 0,
         "residual": True},
        # One token of one request: latency alone.
        {"name": "adapters 1x4096x4096", "op": "adapters", "m": 1, "k": 4096, "n": 4096, "rank": 16, "adapters": 8,
         "requests": 0, "dtype": "bf16", "pad": 0, "base": True, "hidden": False},
        # One decoding step of a batch whose requests each have one of 64 adapters: the adapters' bytes count.
        {"name": "adapters 128x4096x4096 of 64", "op": "adapters", "m": 128, "k": 4096, "n": 4096, "rank": 16, "adapters": 64,
         "requests": 0, "dtype": "bf16", "pad": 0, "base": True, "hidden": False},
        # The prompts of a few requests through the widest projection: its input and output count.
        {"name": "adapters 8192x4096x16384", "op": "adapters", "m": 8192, "k": 4096, "n": 16384, "rank": 64, "adapters": 8,
         "requests": 12, "dtype": "bf16", "pad": 0, "base": True, "hidden": False},
        # Odd in every size, in slices, full precision, as the forward pass of training: no base, hidden rows kept.
        {"name": "adapters 777x1001x515 f32", "op": "adapters", "m": 777, "k": 1001, "n": 515, "rank": 12, "adapters": 5,
         "requests": 9, "dtype": "f32", "pad": 7, "base": False, "hidden": True},
        # The gradients of a few adapters trained side by side on their own batches.
        {"name": "adapters grad 8192x4096x4096", "op": "adapters_backward", "m": 8192, "k": 4096, "n": 4096, "rank": 16,
         "adapters": 4, "requests": 8, "dtype": "bf16", "pad": 0, "base": True},
        # The step of those adapters and norms: many small tensors, 16-bit parameters, states in 8 bits.
        {"name": "adamw 8-bit 192 tensors", "op": "adamw", "tensors": 192, "size": 65536, "dtype": "bf16", "grad": "f32",
         "bits": 8, "odd": False},
        # The step of a whole model's part: memory traffic alone counts.
        {"name": "adamw 32-bit 64M", "op": "adamw", "tensors": 24, "size": 4 << 20, "dtype": "f32", "grad": "f32",
         "bits": 32, "odd": False},
    ]


def _spread(rng, low, high):
    """A whole number spread over the logarithm of [low, high]; one in two a multiple of 8 or 64 where it can be."""
    v = int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))
    step = rng.choice((1, 1, 8, 64))
    return max(low, min(high, v // step * step if v >= step else v))


def draw(rng):
    kind = rng.random()
    dtype, pad = rng.choice(("bf16", "bf16", "f16", "f32")), rng.choice((0, 0, 8, 23))
    if kind < 0.4:
        while True:
            rows, c = _spread(rng, 1, 32768), _spread(rng, 16, 8192)
            if rows * c <= MOST_NORM:
                break
        case = {"op": "rms_norm" if kind < 0.25 else "rms_norm_backward", "rows": rows, "c": c, "dtype": dtype, "pad": pad,
                "residual": rng.random() < 0.6}
        if kind < 0.25:
            case["out"] = rng.choice(("y", "q", "both"))
        return case
    if kind < 0.8:
        grad = kind >= 0.65
        while True:
            m, k, n = _spread(rng, 1, 16384), _spread(rng, 32, 16384), _spread(rng, 16, 16384)
            rank, adapters = rng.choice((4, 8, 8, 12, 16, 16, 32, 64)), _spread(rng, 1, 64)
            if m * (k + n) <= MOST_ADAPTED // (3 if grad else 1) and adapters * rank * (k + n) <= MOST_WEIGHTS // (2 if grad else 1):
                break
        case = {"op": "adapters_backward" if grad else "adapters", "m": m, "k": k, "n": n, "rank": rank, "adapters": adapters,
                "requests": rng.choice((0, 1, 7, 40)), "dtype": dtype, "pad": pad, "base": rng.random() < 0.7}
        if not grad:
            case["hidden"] = rng.random() < 0.5
        return case
    while True:
        tensors, size = _spread(rng, 1, 400), _spread(rng, 256, 16 << 20)
        if tensors * size <= MOST_STEPPED:
            break
    return {"op": "adamw", "tensors": tensors, "size": size, "dtype": rng.choice(("f32", "f32", "bf16", "f16")),
            "grad": rng.choice(("f32", "bf16")), "bits": rng.choice((8, 32)), "odd": rng.random() < 0.4}


def _rows(gen, rows, c, pad, dtype, size=1.0):
    """Activations as layers see them: each channel with its own offset, a few with a much larger spread; a
    column slice of a wider tensor where `pad` is not 0."""
    dev = gen.device
    x = torch.randn(rows, c + pad, generator=gen, device=dev)
    spread = 0.5 + torch.rand(c + pad, generator=gen, device=dev)
    spread[torch.randint(0, c, (max(1, c // 100),), generator=gen, device=dev)] *= 8.0
    x = (x * spread + 0.3 * torch.randn(c + pad, generator=gen, device=dev)) * size
    return x.to(dtype)[:, :c]


def _index(gen, m, adapters, requests):
    """The adapter of each row: one at random (a step of decoding), or the same along each of `requests` runs of rows
    (prompts); about one in sixteen has none."""
    dev = gen.device
    of = torch.randint(0, adapters, (requests or m,), generator=gen, device=dev)
    of[torch.rand(requests or m, generator=gen, device=dev) < 1 / 16] = -1
    if requests:
        cuts = torch.sort(torch.randint(0, m, (requests - 1,), generator=gen, device=dev)).values
        of = of[torch.bucketize(torch.arange(m, device=dev), cuts, right=True)]
    return of.to(torch.int32)


def _sizes(case):
    """Elements of each tensor: three in four as large as the case says or a little less, the others vectors."""
    n = case["size"]
    return [max(1, (n // 64 if i % 4 == 3 else n - (n // 8) * (i % 3)) - (i % 7 if case["odd"] else 0))
            for i in range(case["tensors"])]


def _cut(flat, starts, sizes):
    return [flat[a:a + n] for a, n in zip(starts, sizes)]


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(dev)
    gen.manual_seed(seed)
    dtype, op = DTYPES[case["dtype"]], case["op"]
    s = {"case": case}
    if op.startswith("rms_norm"):
        rows, c, pad = case["rows"], case["c"], case["pad"]
        s["x"] = _rows(gen, rows, c, pad, dtype)
        s["gamma"] = 0.5 + torch.rand(c, generator=gen, device=dev)
        s["residual"] = _rows(gen, rows, c, pad, dtype, 0.01 if op == "rms_norm_backward" else 2.0) if case["residual"] else None
        if op == "rms_norm_backward":
            s["dy"] = _rows(gen, rows, c, pad, dtype, 0.01)
            s["rstd"] = s["x"].float().square().mean(dim=1).add(EPS).rsqrt()
        return s
    if op.startswith("adapters"):
        m, k, n, g, r, pad = (case[name] for name in ("m", "k", "n", "adapters", "rank", "pad"))
        s["x"] = _rows(gen, m, k, pad, dtype)
        s["index"] = _index(gen, m, g, case["requests"])
        s["a"] = (torch.randn(g, r, k, generator=gen, device=dev) / math.sqrt(k)).to(dtype)
        s["b"] = (0.3 * torch.randn(g, n, r, generator=gen, device=dev) / math.sqrt(r)).to(dtype)
        s["scale"] = 0.5 + 1.5 * torch.rand(g, generator=gen, device=dev)
        if op == "adapters":
            s["base"] = torch.randn(m, n + pad, generator=gen, device=dev).to(dtype)[:, :n] if case["base"] else None
        else:
            s["dy"] = _rows(gen, m, n, pad, dtype, 0.01)
            s["base"] = (0.01 * torch.randn(m, k + pad, generator=gen, device=dev)).to(dtype)[:, :k] if case["base"] else None
            s["hidden"] = _picked(s["x"].float() @ s["a"].float().flatten(0, 1).t(), s["index"], g)[0]
        return s
    sizes, starts, total = _sizes(case), [], 0
    for n in sizes:  # each tensor on a block of the 8-bit states of its own
        starts.append(total)
        total += -(-n // BLOCK) * BLOCK
    inside = torch.zeros(total, dtype=torch.bool, device=dev)
    for part in _cut(inside, starts, sizes):
        part.fill_(True)
    p = 0.05 * torch.randn(total, generator=gen, device=dev)
    spread = torch.exp(torch.randn(total // BLOCK, generator=gen, device=dev)).repeat_interleave(BLOCK)
    g = 1e-3 * spread * torch.randn(total, generator=gen, device=dev)
    m = 4e-4 * spread * torch.randn(total, generator=gen, device=dev)
    v = (1e-3 * spread * (0.3 + torch.rand(total, generator=gen, device=dev))).square()
    p, g, m, v = ((t * inside).to(d) for t, d in ((p, dtype), (g, DTYPES[case["grad"]]), (m, torch.float32), (v, torch.float32)))
    s.update(p=p, g=g, m=m, v=v, step=100, lr=1e-3, grad_scale=torch.full((1,), 0.5, device=dev))
    if case["bits"] == 8:
        s["m_scale"], s["v_scale"] = (torch.clamp(t.view(-1, BLOCK).amax(dim=1), min=TINY) / MOST_8 for t in (m.abs(), v.sqrt()))
        s["m"] = (m.view(-1, BLOCK) / s["m_scale"][:, None]).clamp(-MOST_8, MOST_8).view(-1).to(torch.float8_e4m3fn)
        least = torch.where(v > 0, 2.0 ** -9, 0.0)
        s["v"] = torch.maximum((v.sqrt().view(-1, BLOCK) / s["v_scale"][:, None]).clamp(0, MOST_8).view(-1), least).to(torch.float8_e4m3fn)
    for name in ("p", "g", "m", "v"):
        s[name + "s"] = _cut(s[name], starts, sizes)
    if case["bits"] == 8:
        first = torch.zeros(total, dtype=torch.int64, device=dev)
        for a, part in zip(starts, _cut(first, starts, [-(-n // BLOCK) * BLOCK for n in sizes])):
            part.fill_(a)
        s["place"] = (torch.arange(total, device=dev) - first).view(-1, BLOCK)  # in each tensor
        blocks = [-(-n // BLOCK) for n in sizes]
        for name in ("m_scale", "v_scale"):
            s[name + "s"] = _cut(s[name], [a // BLOCK for a in starts], blocks)
    return s


def _picked(all_hidden, index, adapters):
    """Of products with every adapter [rows, adapters * rank], those of each row's own; and the same with zeros in the
    place of the others."""
    rows = all_hidden.view(len(index), adapters, -1)
    mine = (index[:, None] == torch.arange(adapters, device=index.device))[:, :, None]
    kept = torch.where(mine, rows, torch.zeros((), dtype=rows.dtype, device=rows.device))
    return kept.sum(dim=1), kept.flatten(1)


def _spread_out(hidden, index, adapters):
    """[rows, rank] at the place of each row's adapter in [rows, adapters * rank]."""
    mine = (index[:, None] == torch.arange(adapters, device=index.device))[:, :, None]
    return (hidden[:, None, :] * mine).flatten(1)


def _row_scale(s):
    index = s["index"].long()
    return torch.where(index >= 0, s["scale"][index.clamp(min=0)], 0.0)[:, None]


def _quantised(v):
    most = torch.clamp(v.abs().amax(dim=1, keepdim=True), min=TINY)
    return torch.round(v * (127.0 / most)), (most / 127.0)[:, 0]


def _dither(place, step):
    """Two numbers in [0, 1) for each place of a tensor and step: the halves of the mixed bits (Appleby's 32-bit
    finaliser) of place + step * 0x9E3779B9."""
    z = (place + step * 0x9E3779B9) & 0xFFFFFFFF
    z = ((z ^ (z >> 16)) * 0x85EBCA6B) & 0xFFFFFFFF
    z = ((z ^ (z >> 13)) * 0xC2B2AE35) & 0xFFFFFFFF
    z = z ^ (z >> 16)
    return (z >> 16).float() / 65536, (z & 0xFFFF).float() / 65536


def _eighth(x, u):
    """Magnitudes up to 448 to one of the two e4m3 values around them, by u in [0, 1)."""
    grid = torch.exp2(torch.clamp(torch.frexp(x).exponent - 1, min=-6) - 3).to(x.dtype)
    return torch.clamp(torch.floor(x / grid + u) * grid, max=MOST_8)


def _held(x, u):
    """Non-negative values [blocks, BLOCK] as e4m3 values and a scale for each block."""
    most = torch.clamp(x.amax(dim=1, keepdim=True), min=TINY)
    return _eighth(x * (MOST_8 / most), u), (most / MOST_8)[:, 0]


def _step_all(s):
    """The AdamW step of all tensors, which lie in one buffer, into the buffers."""
    p, m, v, eight = s["p"], s["m"], s["v"], s["case"]["bits"] == 8
    g = s["g"].float() * s["grad_scale"]
    m1, v1 = m, v
    if eight:
        m1 = (m.float().view(-1, BLOCK) * s["m_scale"][:, None]).view(-1)
        v1 = (v.float().view(-1, BLOCK) * s["v_scale"][:, None]).square().view(-1)
    m1 = BETA1 * m1 + (1 - BETA1) * g
    v1 = BETA2 * v1 + (1 - BETA2) * g * g
    root = torch.sqrt(v1)
    c1, c2 = 1 - BETA1 ** s["step"], math.sqrt(1 - BETA2 ** s["step"])
    p.copy_(p.float() * (1 - s["lr"] * DECAY) - s["lr"] / c1 * m1 / (root / c2 + ADAM_EPS))
    if not eight:
        m.copy_(m1)
        v.copy_(v1)
        return
    um, uv = _dither(s["place"], s["step"])
    m1, root = m1.view(-1, BLOCK), root.view(-1, BLOCK)
    held, scale = _held(m1.abs(), um)
    m.copy_(torch.copysign(held, m1).view(-1))
    s["m_scale"].copy_(scale)
    held, scale = _held(root, uv)
    v.copy_(torch.maximum(held, torch.where(root > 0, 2.0 ** -9, 0.0)).view(-1))
    s["v_scale"].copy_(scale)


def _state_of(s):
    names = ("p", "m", "v", "m_scale", "v_scale") if s["case"]["bits"] == 8 else ("p", "m", "v")
    return {name: s[name] for name in names}


def _plain(s):
    case, op = s["case"], s["case"]["op"]
    dtype = DTYPES[case["dtype"]]
    if op == "rms_norm":
        x, out = s["x"], {}
        if s["residual"] is not None:
            x = out["total"] = (x.float() + s["residual"].float()).to(dtype)
        x = x.float()
        y = x * (1.0 / torch.sqrt((x * x).sum(dim=1, keepdim=True) / x.shape[1] + EPS)) * s["gamma"]
        if case["out"] != "q":
            out["y"] = y.to(dtype)
        if case["out"] != "y":
            q, out["scale"] = _quantised(y)
            out["q"] = q.to(torch.bfloat16)
        return out
    if op == "rms_norm_backward":
        x, g, rstd = s["x"].float(), s["dy"].float() * s["gamma"], s["rstd"][:, None]
        h = x * rstd
        dx = rstd * (g - h * ((g * h).sum(dim=1, keepdim=True) / x.shape[1]))
        if s["residual"] is not None:
            dx = dx + s["residual"].float()
        return {"dx": dx.to(dtype), "dgamma": (s["dy"].float() * h).sum(dim=0)}
    if op == "adapters":
        index, g = s["index"], case["adapters"]
        hidden, mine = _picked(s["x"].float() @ s["a"].float().flatten(0, 1).t(), index, g)
        y = _row_scale(s) * (mine @ s["b"].float().transpose(1, 2).flatten(0, 1))
        if s["base"] is not None:
            y = y + s["base"].float()
        return {"y": y.to(dtype), "hidden": hidden} if case["hidden"] else {"y": y.to(dtype)}
    if op == "adapters_backward":
        index, g, x = s["index"], case["adapters"], s["x"].float()
        dy = s["dy"].float() * _row_scale(s)
        _, dh = _picked(dy @ s["b"].float().transpose(1, 2).flatten(0, 1).t(), index, g)
        dx = dh @ s["a"].float().flatten(0, 1)
        if s["base"] is not None:
            dx = dx + s["base"].float()
        da = (dh.t() @ x).view(g, -1, x.shape[1])
        db = (dy.t() @ _spread_out(s["hidden"], index, g)).view(dy.shape[1], g, -1).transpose(0, 1).contiguous()
        return {"dx": dx.to(dtype), "da": da, "db": db}
    _step_all(s)
    return _state_of(s)


def _called(s):
    capi, case, op = _binding(), s["case"], s["case"]["op"]
    if op == "rms_norm":
        if case["out"] == "y":
            out = capi.rms_norm(s["x"], s["gamma"], EPS, residual=s["residual"])
            names = ("y", "total")
        else:
            out = capi.rms_norm_quantize(s["x"], s["gamma"], EPS, residual=s["residual"], return_y=case["out"] == "both")
            names = ("q", "scale") + (("total",) if s["residual"] is not None else ()) + ("y",)
        out = dict(zip(names, out if isinstance(out, tuple) else (out,)))
        if "q" in out:  # as values: next to a half, the sum over a row decides, whose order is open
            out["q"] = out["q"].to(torch.bfloat16)
        return out
    if op == "rms_norm_backward":
        dx, dgamma = capi.rms_norm_backward(s["dy"], s["x"], s["gamma"], s["rstd"], residual=s["residual"])
        return {"dx": dx, "dgamma": dgamma}
    if op == "adapters":
        out = capi.linear_adapters(s["x"], s["index"], s["a"], s["b"], s["scale"], base=s["base"], return_hidden=case["hidden"])
        return {"y": out[0], "hidden": out[1]} if case["hidden"] else {"y": out}
    if op == "adapters_backward":
        dx, da, db = capi.linear_adapters_backward(s["dy"], s["x"], s["index"], s["a"], s["b"], s["scale"], s["hidden"],
                                                   base=s["base"])
        return {"dx": dx, "da": da, "db": db}
    scales = {"exp_avg_scale": s["m_scales"], "exp_avg_sq_scale": s["v_scales"]} if case["bits"] == 8 else {}
    capi.adamw_step(s["ps"], s["gs"], s["ms"], s["vs"], step=s["step"], lr=s["lr"], betas=(BETA1, BETA2), eps=ADAM_EPS,
                    weight_decay=DECAY, grad_scale=s["grad_scale"], **scales)
    return _state_of(s)


def run(state):
    return _called(state) if own else _plain(state)


def exact(case, seed):
    """The definitions in 64 bits: the norm through its sum of squares, its gradient as the chain rule gives it term by
    term, adapters one after the other over the rows that they have, the step from the moments' recurrences."""
    s, op = prepare(case, seed), case["op"]
    dtype = DTYPES[case["dtype"]]
    if op == "rms_norm":
        x, out = s["x"].double(), {}
        if case["residual"]:
            out["total"] = x + s["residual"].double()
            x = out["total"].to(dtype).double()
        y = torch.einsum("rc,r,c->rc", x, (torch.linalg.vector_norm(x, dim=1).square() / x.shape[1] + EPS) ** -0.5, s["gamma"].double())
        if case["out"] != "q":
            out["y"] = y
        if case["out"] != "y":
            out["scale"] = torch.maximum(y.amax(dim=1), -y.amin(dim=1)).clamp(min=TINY) / 127.0
            out["q"] = torch.round(y / out["scale"][:, None])
        return out
    if op == "rms_norm_backward":
        x, dy, rstd, gamma = s["x"].double(), s["dy"].double(), s["rstd"].double(), s["gamma"].double()
        # y depends on x directly and through rstd, whose derivative is -rstd^3 x / c.
        drstd = torch.einsum("rc,rc,c->r", dy, x, gamma)
        dx = dy * gamma * rstd[:, None] - (drstd * rstd ** 3 / x.shape[1])[:, None] * x
        if case["residual"]:
            dx = dx + s["residual"].double()
        return {"dx": dx, "dgamma": torch.einsum("rc,rc,r->c", dy, x, rstd)}
    if op.startswith("adapters"):
        x, a, b, scale = s["x"].double(), s["a"].double(), s["b"].double(), s["scale"].double()
        if op == "adapters":
            hidden, y = x.new_zeros(case["m"], case["rank"]), x.new_zeros(case["m"], case["n"])
        else:
            dx, da, db = torch.zeros_like(x), torch.zeros_like(a), torch.zeros_like(b)
            dy, hidden = s["dy"].double(), s["hidden"].double()
        for j in range(case["adapters"]):
            at = (s["index"] == j).nonzero()[:, 0]
            if op == "adapters":
                hidden[at] = torch.einsum("mk,rk->mr", x[at], a[j])
                y[at] = scale[j] * torch.einsum("mr,nr->mn", hidden[at], b[j])
            else:
                dh = scale[j] * torch.einsum("mn,nr->mr", dy[at], b[j])
                dx[at] = torch.einsum("mr,rk->mk", dh, a[j])
                da[j] = torch.einsum("mr,mk->rk", dh, x[at])
                db[j] = scale[j] * torch.einsum("mn,mr->nr", dy[at], hidden[at])
        base = s["base"].double() if case["base"] else 0.0
        if op == "adapters":
            return {"y": y + base, "hidden": hidden} if case["hidden"] else {"y": y + base}
        return {"dx": dx + base, "da": da, "db": db}
    p, g, eight = s["p"].double(), s["g"].double() * s["grad_scale"].double(), case["bits"] == 8
    m, v = s["m"].double(), s["v"].double()
    if eight:
        m = m * s["m_scale"].double().repeat_interleave(BLOCK)
        v = (v * s["v_scale"].double().repeat_interleave(BLOCK)).square()
    m = torch.lerp(g, m, BETA1)
    v = torch.lerp(g * g, v, BETA2)
    mean, variance = m / (1 - BETA1 ** s["step"]), v / (1 - BETA2 ** s["step"])
    out = {"p": p - s["lr"] * DECAY * p - s["lr"] * mean / (variance.sqrt() + ADAM_EPS)}
    if not eight:
        return {**out, "m": m, "v": v}
    tops = [t.view(-1, BLOCK).amax(dim=1).clamp(min=TINY) / MOST_8 for t in (m.abs(), v.sqrt())]
    # The values themselves, which the held ones are within a step of the format of, have no one rounding in 64 bits.
    return {**out, "m": None, "v": None, "m_scale": tops[0], "v_scale": tops[1]}


def work(case):
    op, size = case["op"], DTYPES[case["dtype"]].itemsize
    if op.startswith("rms_norm"):
        rows, c, more = case["rows"], case["c"], 1 if case["residual"] else 0
        if op == "rms_norm_backward":
            return {"bytes": (3 + more) * rows * c * size + 8 * c + 4 * rows, "flops": 9 * rows * c}
        wide = 1 + 2 * more + (0 if case["out"] == "q" else 1)
        narrow = 0 if case["out"] == "y" else rows * (c + 4)
        return {"bytes": wide * rows * c * size + narrow + 4 * c, "flops": 5 * rows * c}
    if op.startswith("adapters"):
        m, k, n, g, r = (case[name] for name in ("m", "k", "n", "adapters", "rank"))
        # Adapters that some row has, as many as are expected.
        drawn = (case["requests"] or m) * 15 / 16
        used = int(round(g * (1 - (1 - 1 / g) ** drawn))) if g > 1 else 1
        weights, base = used * r * (k + n) * size + 4 * m + 4 * g, 1 if case["base"] else 0
        if op == "adapters":
            return {"bytes": m * (k + n * (1 + base)) * size + weights + (4 * m * r if case["hidden"] else 0),
                    "flops": 2 * m * r * (k + n)}
        return {"bytes": m * (n + k * (2 + base)) * size + weights + 4 * m * r + 4 * g * r * (k + n), "flops": 4 * m * r * (k + n)}
    n = sum(_sizes(case))
    state = 16 if case["bits"] == 32 else 4 + 16 / BLOCK
    return {"bytes": int(n * (2 * size + DTYPES[case["grad"]].itemsize + state)), "flops": 14 * n}
