"""Workloads of the token-wise operators: layer norm, its gradient, and the linear layer in
8-bit integers.

Each case is one call a program makes: ``layer_norm`` (the rows normalised, with the statistics
its gradient needs), ``layer_norm_backward`` (the gradients of the input and of both parameters)
or ``linear`` (a product of int8 rows with int8 weights, scales for each row and each output
channel, bias, activation and residual; the rows come quantised, are quantised by the call, or
are normalised and quantised by it).  ``run`` computes a case with elementary torch operations,
or, where ``own`` is true, through the package's binding; ``exact`` restates it in 64 bits.
"""
import math

import torch

own = False

EPS = 1e-5
TINY = 2.0 ** -100  # a row whose largest magnitude is below this is quantised as if it were this
DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
MOST_ELEMENTS = 16384 * 4096            # of a layer norm case
MOST_PRODUCTS = 8192 * 4096 * 16384     # multiply-adds of a linear case

_capi = None


def _binding():
    global _capi
    if _capi is None:
        from conv2d_batchnorm_silu_gb300 import capi
        _capi = capi
    return _capi


def listed():
    return [
        # The pixels of one small feature map, normalised over few channels: a call whose launch counts.
        {"name": "norm 1024x32", "op": "layer_norm", "rows": 1024, "c": 32, "dtype": "bf16", "pad": 0},
        # An odd channel count, in a column slice of a wider tensor: rows without 16-byte alignment.
        {"name": "norm 3001x777 slice", "op": "layer_norm", "rows": 3001, "c": 777, "dtype": "f16", "pad": 23},
        # A long batch of wide tokens, as in training: memory traffic alone counts.
        {"name": "norm 16384x4096", "op": "layer_norm", "rows": 16384, "c": 4096, "dtype": "bf16", "pad": 0},
        # The gradient at the pixels of a 16x40x40x256 feature map.
        {"name": "norm grad 25600x256", "op": "layer_norm_backward", "rows": 25600, "c": 256, "dtype": "bf16", "pad": 0},
        # The gradient in full precision at odd sizes.
        {"name": "norm grad 999x1537 f32", "op": "layer_norm_backward", "rows": 999, "c": 1537, "dtype": "f32", "pad": 0},
        # The gradient of a long batch of wide tokens.
        {"name": "norm grad 16384x4096", "op": "layer_norm_backward", "rows": 16384, "c": 4096, "dtype": "bf16", "pad": 0},
        # One step of serving a few sequences: norm, quantisation and product of eight tokens.
        {"name": "linear norm 8x4096x4096", "op": "linear", "quant": "norm", "m": 8, "k": 4096, "n": 4096,
         "dtype": "bf16", "bias": True, "act": "identity", "residual": False, "pad": 0},
        # The expansion of a token block over the pixels of a 16x40x40x256 feature map, with SiLU.
        {"name": "linear norm 25600x256x1024", "op": "linear", "quant": "norm", "m": 25600, "k": 256, "n": 1024,
         "dtype": "bf16", "bias": True, "act": "silu", "residual": False, "pad": 0},
        # A single token through a wide layer: the weights' bytes alone count.
        {"name": "linear rows 1x8192x8192", "op": "linear", "quant": "rows", "m": 1, "k": 8192, "n": 8192,
         "dtype": "bf16", "bias": False, "act": "identity", "residual": False, "pad": 0},
        # A batch of single tokens, already quantised, added to the residual stream.
        {"name": "linear 64x8192x8192", "op": "linear", "quant": "none", "m": 64, "k": 8192, "n": 8192,
         "dtype": "bf16", "bias": True, "act": "identity", "residual": True, "pad": 0},
        # Odd in every size, rows in a slice, 32-bit input and output.
        {"name": "linear rows 333x1001x777 f32", "op": "linear", "quant": "rows", "m": 333, "k": 1001, "n": 777,
         "dtype": "f32", "bias": True, "act": "relu", "residual": False, "pad": 7},
        # A prompt through the widest layer: the tensor cores alone count.
        {"name": "linear 8192x4096x16384", "op": "linear", "quant": "none", "m": 8192, "k": 4096, "n": 16384,
         "dtype": "bf16", "bias": True, "act": "silu", "residual": False, "pad": 0},
    ]


def _spread(rng, low, high):
    """A whole number spread over the logarithm of [low, high]; one in two a multiple of 8 or 64 where it can be."""
    v = int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))
    step = rng.choice((1, 1, 8, 64))
    return max(low, min(high, v // step * step if v >= step else v))


def draw(rng):
    if rng.random() < 0.4:
        while True:
            rows, c = _spread(rng, 1, 32768), _spread(rng, 16, 8192)
            if rows * c <= MOST_ELEMENTS:
                break
        return {"op": rng.choice(("layer_norm", "layer_norm_backward")), "rows": rows, "c": c,
                "dtype": rng.choice(("bf16", "bf16", "f16", "f32")), "pad": rng.choice((0, 0, 8, 23))}
    while True:
        m, k, n = _spread(rng, 1, 32768), _spread(rng, 32, 16384), _spread(rng, 16, 16384)
        if m * k * n <= MOST_PRODUCTS and m * max(k, n) <= 4 * MOST_ELEMENTS:
            break
    quant = rng.choice(("none", "rows", "norm"))
    # Normalised values are rounded to 8 bits from 32-bit sums whose order is open: 16-bit outputs there.
    dtype = rng.choice(("bf16", "bf16", "f16") if quant == "norm" else ("bf16", "bf16", "f16", "f32"))
    return {"op": "linear", "quant": quant, "m": m, "k": k, "n": n, "dtype": dtype, "bias": rng.random() < 0.7,
            "act": rng.choice(("identity", "silu", "relu")), "residual": rng.random() < 0.3, "pad": rng.choice((0, 0, 16, 7))}


def _rows(gen, rows, c, pad, dtype):
    """Activations as layers see them: each channel with its own offset, a few with a much larger spread; a
    column slice of a wider tensor where `pad` is not 0."""
    dev = gen.device
    x = torch.randn(rows, c + pad, generator=gen, device=dev)
    spread = 0.5 + torch.rand(c + pad, generator=gen, device=dev)
    spread[torch.randint(0, c, (max(1, c // 100),), generator=gen, device=dev)] *= 8.0
    x = x * spread + 0.3 * torch.randn(c + pad, generator=gen, device=dev)
    return x.to(dtype)[:, :c]


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(dev)
    gen.manual_seed(seed)
    dtype, pad = DTYPES[case["dtype"]], case["pad"]
    s = {"case": case}
    if case["op"] == "linear":
        m, k, n = case["m"], case["k"], case["n"]
        if case["quant"] == "none":
            a = (torch.randn(m, k + pad, generator=gen, device=dev) * 32.0).round_().clamp_(-127, 127)
            s["a"] = a.to(torch.int8)[:, :k]
            s["a_scale"] = (0.5 + torch.rand(m, generator=gen, device=dev)) / 32.0
        else:
            s["x"] = _rows(gen, m, k, pad, dtype)
        if case["quant"] == "norm":
            s["gamma"] = 0.5 + torch.rand(k, generator=gen, device=dev)
            s["beta"] = 0.1 * torch.randn(k, generator=gen, device=dev)
        s["w"] = (torch.randn(n, k, generator=gen, device=dev) * 32.0).round_().clamp_(-127, 127).to(torch.int8)
        s["w_scale"] = (0.5 + torch.rand(n, generator=gen, device=dev)) / (32.0 * math.sqrt(k))
        s["bias"] = 0.1 * torch.randn(n, generator=gen, device=dev) if case["bias"] else None
        s["residual"] = torch.randn(m, n, generator=gen, device=dev).to(dtype) if case["residual"] else None
        return s
    rows, c = case["rows"], case["c"]
    s["x"] = _rows(gen, rows, c, pad, dtype)
    s["gamma"] = 0.5 + torch.rand(c, generator=gen, device=dev)
    s["beta"] = 0.1 * torch.randn(c, generator=gen, device=dev)
    if case["op"] == "layer_norm_backward":
        s["dy"] = (0.01 * torch.randn(rows, c, generator=gen, device=dev)).to(dtype)
        x = s["x"].float()
        mean = x.mean(dim=1, keepdim=True)
        s["stats"] = torch.stack((mean[:, 0], (x - mean).square().mean(dim=1).add(EPS).rsqrt()))
    return s


def _normalised(x, gamma, beta):
    mean = x.sum(dim=1, keepdim=True) / x.shape[1]
    d = x - mean
    rstd = 1.0 / torch.sqrt((d * d).sum(dim=1, keepdim=True) / x.shape[1] + EPS)
    return d * rstd * gamma + beta, mean, rstd


def _quantised(v):
    most = torch.clamp(v.abs().amax(dim=1, keepdim=True), min=TINY)
    return torch.round(v * (127.0 / most)), most / 127.0


def _activated(z, act):
    if act == "silu":
        return z / (1.0 + torch.exp(-z))
    return torch.clamp(z, min=0.0) if act == "relu" else z


def _plain(s):
    case = s["case"]
    dtype = DTYPES[case["dtype"]]
    if case["op"] == "layer_norm":
        y, mean, rstd = _normalised(s["x"].float(), s["gamma"], s["beta"])
        return {"y": y.to(dtype), "stats": torch.stack((mean[:, 0], rstd[:, 0]))}
    if case["op"] == "layer_norm_backward":
        x, dy, (mean, rstd) = s["x"].float(), s["dy"].float(), s["stats"]
        h = (x - mean[:, None]) * rstd[:, None]
        g = dy * s["gamma"]
        c = x.shape[1]
        dx = rstd[:, None] * (g - g.sum(dim=1, keepdim=True) / c - h * ((g * h).sum(dim=1, keepdim=True) / c))
        return {"dx": dx.to(dtype), "dgamma": (dy * h).sum(dim=0), "dbeta": dy.sum(dim=0)}
    if case["quant"] == "none":
        a, a_scale = s["a"].float(), s["a_scale"][:, None]
    else:
        v = s["x"].float()
        if case["quant"] == "norm":
            v = _normalised(v, s["gamma"], s["beta"])[0]
        a, a_scale = _quantised(v)
    z = (a @ s["w"].float().t()) * (a_scale * s["w_scale"])
    if s["bias"] is not None:
        z = z + s["bias"]
    z = _activated(z, case["act"])
    if s["residual"] is not None:
        z = z + s["residual"].float()
    out = {"y": z.to(dtype)}
    if case["quant"] != "none":
        out["scale"] = a_scale[:, 0]
    return out


def _called(s):
    capi, case = _binding(), s["case"]
    if case["op"] == "layer_norm":
        y, stats = capi.layer_norm(s["x"], s["gamma"], s["beta"], EPS, return_stats=True)
        return {"y": y, "stats": stats}
    if case["op"] == "layer_norm_backward":
        dx, dgamma, dbeta = capi.layer_norm_backward(s["dy"], s["x"], s["gamma"], s["stats"])
        return {"dx": dx, "dgamma": dgamma, "dbeta": dbeta}
    if case["quant"] == "none":
        a, a_scale = s["a"], s["a_scale"]
    elif case["quant"] == "rows":
        a, a_scale = capi.quantize_rows(s["x"])
    else:
        a, a_scale = capi.layer_norm_quantize(s["x"], s["gamma"], s["beta"], EPS)
    out = {"y": capi.linear_int8(a, s["w"], a_scale, s["w_scale"], bias=s["bias"], activation=case["act"],
                                 residual=s["residual"], out_dtype=DTYPES[case["dtype"]])}
    if case["quant"] != "none":
        out["scale"] = a_scale
    return out


def run(state):
    return _called(state) if own else _plain(state)


def exact(case, seed):
    """The definitions in 64 bits: moments from the raw values, the gradient as the chain rule gives it term by
    term, integers summed as such (every sum of the cases is below 2**53)."""
    s = prepare(case, seed)
    if case["op"] == "linear":
        if case["quant"] == "none":
            q, t = s["a"].double(), s["a_scale"].double()
        else:
            v = s["x"].double()
            if case["quant"] == "norm":
                var, mean = torch.var_mean(v, dim=1, unbiased=False, keepdim=True)
                v = torch.addcmul(s["beta"].double(), (v - mean) / torch.sqrt(var + EPS), s["gamma"].double())
            t = torch.maximum(v.amax(dim=1), -v.amin(dim=1)).clamp(min=TINY) / 127.0
            q = torch.round(v / t[:, None])
        z = torch.einsum("mk,nk->mn", q, s["w"].double()) * t[:, None] * s["w_scale"].double()[None, :]
        if case["bias"]:
            z = z + s["bias"].double()
        if case["act"] == "silu":
            z = z * torch.sigmoid(z)
        elif case["act"] == "relu":
            z = torch.relu(z)
        if case["residual"]:
            z = z + s["residual"].double()
        return {"y": z} if case["quant"] == "none" else {"y": z, "scale": t}
    x, gamma = s["x"].double(), s["gamma"].double()
    if case["op"] == "layer_norm":
        var, mean = torch.var_mean(x, dim=1, unbiased=False)
        rstd = (var + EPS) ** -0.5
        y = torch.addcmul(s["beta"].double(), (x - mean[:, None]) * rstd[:, None], gamma)
        return {"y": y, "stats": torch.stack((mean, rstd))}
    dy, (mean, rstd) = s["dy"].double(), s["stats"].double()
    c = x.shape[1]
    d = x - mean[:, None]
    dh = dy * gamma
    # y depends on x directly, through the variance and through the mean.
    dvar = (dh * d).sum(1) * -0.5 * rstd ** 3
    dmean = -(dh.sum(1) * rstd) - 2.0 / c * dvar * d.sum(1)
    dx = dh * rstd[:, None] + (2.0 / c) * dvar[:, None] * d + dmean[:, None] / c
    return {"dx": dx, "dgamma": torch.einsum("rc,rc,r->c", dy, d, rstd), "dbeta": dy.sum(0)}


def work(case):
    size = DTYPES[case["dtype"]].itemsize
    if case["op"] == "linear":
        m, k, n = case["m"], case["k"], case["n"]
        rows_in = m * k + 4 * m if case["quant"] == "none" else m * k * size + 4 * m
        params = n * k + 4 * n + (4 * n if case["bias"] else 0) + (8 * k if case["quant"] == "norm" else 0)
        return {"bytes": rows_in + params + m * n * size * (2 if case["residual"] else 1), "flops": 2 * m * n * k}
    rows, c = case["rows"], case["c"]
    if case["op"] == "layer_norm":
        return {"bytes": 2 * rows * c * size + 8 * c + 8 * rows, "flops": 8 * rows * c}
    return {"bytes": 3 * rows * c * size + 12 * c + 8 * rows, "flops": 14 * rows * c}
