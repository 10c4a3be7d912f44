"""The convolution layer followed by a token-wise block on its pixels, in int8.

A feature map that the fused layer leaves as [n, h, w, c] is n*h*w tokens of c channels in memory
already.  On them runs, with a hidden width of its own,

    y = h + W2 SiLU(W1 LN(h) + b1) + b2

as four calls: ``layer_norm_quantize`` (the norm's output as int8 with a scale per token),
``linear_int8`` with SiLU, ``quantize_rows`` of the hidden rows, ``linear_int8`` with the residual.
The weights are quantised once, by ``quantize_rows`` too: a scale per output channel.

``TokenBlock.tune_norm`` trains the norm's gamma and beta towards given rows with ``layer_norm`` and
``layer_norm_backward``.

``AdaptedProjection`` is what requests with low-rank adapters of their own share on a residual stream,

    total = h + residual,  z = W RMSNorm(total) + bias + s_g B_g A_g RMSNorm(total)

as three calls: ``rms_norm_quantize`` (the total, and its norm as int8 and as it is), ``linear_int8`` with the
projection that all share, ``linear_adapters`` with each row's adapter, added in place.  ``tune`` trains the adapters
with ``linear_adapters_backward`` and ``adamw_step``, the projection staying as it is.

    python -m conv2d_batchnorm_silu_gb300.token_block [--n 16] [--size 40] [--channels 256] [--hidden 1024]

prints how far the int8 block is from the same block in fp32, its time and the loss of a short tuning, and the time and
tuning of a projection with four adapters on the same pixels.
Needs a GPU.
"""
from __future__ import annotations

import argparse

import torch

from . import capi


def _current(stream):
    """A call's stream (torch.cuda.Stream or a handle; None: the current one) as PyTorch's current one."""
    if stream is not None and not isinstance(stream, torch.cuda.Stream):
        handle = capi._stream_handle(stream)
        # 0 and 1 are the default stream's; as an ExternalStream, 0 would be one of PyTorch's own.
        stream = torch.cuda.default_stream() if handle in (0, 1) else torch.cuda.ExternalStream(handle)
    return torch.cuda.stream(stream)


class TokenBlock:
    """gamma, beta [c] and b1 [hidden], b2 [c] in fp32; w1 [hidden][c] and w2 [c][hidden] of any float type."""

    def __init__(self, gamma, beta, w1, b1, w2, b2, eps=1e-5):
        self.gamma, self.beta, self.b1, self.b2, self.eps = gamma, beta, b1, b2, eps
        self.w1, self.w1_scale = capi.quantize_rows(w1)
        self.w2, self.w2_scale = capi.quantize_rows(w2)

    def __call__(self, h, stream=None):
        """h [..., c], f32, bf16 or f16 -> the block's output in the same type and shape."""
        q, scale = capi.layer_norm_quantize(h, self.gamma, self.beta, self.eps, stream=stream)
        u = capi.linear_int8(q, self.w1, scale, self.w1_scale, self.b1, "silu", out_dtype=h.dtype, stream=stream)
        q, scale = capi.quantize_rows(u, stream=stream)
        return capi.linear_int8(q, self.w2, scale, self.w2_scale, self.b2, "identity", h, h.dtype, stream=stream)

    def tune_norm(self, h, target, steps=20, rate=0.2):
        """Gradient steps on gamma and beta for the mean over tokens of |LN(h) - target|^2 / 2; the losses."""
        tokens = h.numel() // h.shape[-1]
        losses = []
        for _ in range(steps):
            y, stats = capi.layer_norm(h, self.gamma, self.beta, self.eps, return_stats=True)
            off = y.float() - target
            losses.append(float(off.square().sum() / (2 * tokens)))
            # The gradient of the sum over tokens, so that 16-bit types do not lose errors divided by their number.
            _, dgamma, dbeta = capi.layer_norm_backward(off.to(h.dtype), h, self.gamma, stats)
            self.gamma = self.gamma - rate / tokens * dgamma
            self.beta = self.beta - rate / tokens * dbeta
        return losses


class AdaptedProjection:
    """gamma [c] in fp32, w [n][c] of any float type (quantised here), bias [n] in fp32 or None; a [adapters][rank][c] and
    b [adapters][n][rank] in fp32, used in h's type; scale [adapters] in fp32 or None."""

    def __init__(self, gamma, w, bias, a, b, scale=None, eps=1e-6):
        self.gamma, self.bias, self.a, self.b, self.scale, self.eps = gamma, bias, a, b, scale, eps
        self.w, self.w_scale = capi.quantize_rows(w)

    def __call__(self, h, residual, index, stream=None):
        """h and residual [..., c], index int32 for each row (outside the adapters: none) -> (z [..., n], total [..., c])."""
        with _current(stream):  # PyTorch's casts too, whose memory is then the stream's
            q, q_scale, total, y = capi.rms_norm_quantize(h, self.gamma, self.eps, residual=residual, return_y=True)
            z = capi.linear_int8(q, self.w, q_scale, self.w_scale, self.bias, out_dtype=h.dtype)
            a, b = self.a.to(h.dtype), self.b.to(h.dtype)
            return capi.linear_adapters(y, index, a, b, self.scale, base=z, y=z), total

    def tune(self, h, residual, index, target, steps=20, lr=1e-2, bits=8):
        """AdamW steps on the adapters for the mean over rows of |z - target|^2 / 2, with moments of so many bits; the
        losses."""
        rows, losses, state = index.numel(), [], capi.adamw_state([self.a, self.b], bits)
        q, q_scale, _, y = capi.rms_norm_quantize(h, self.gamma, self.eps, residual=residual, return_y=True)
        shared = capi.linear_int8(q, self.w, q_scale, self.w_scale, self.bias, out_dtype=h.dtype)
        for step in range(1, steps + 1):
            a, b = self.a.to(h.dtype), self.b.to(h.dtype)
            z, hidden = capi.linear_adapters(y, index, a, b, self.scale, base=shared, return_hidden=True)
            off = z.float() - target
            losses.append(float(off.square().sum() / (2 * rows)))
            # The gradient of the sum over rows, so that 16-bit types do not lose errors divided by their number.
            _, da, db = capi.linear_adapters_backward(off.to(h.dtype), y, index, a, b, self.scale, hidden)
            capi.adamw_step([self.a, self.b], [da, db], step=step, lr=lr, weight_decay=0.0, grad_scale=1.0 / rows, **state)
        return losses


def _main():
    p = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    p.add_argument("--n", type=int, default=16)
    p.add_argument("--size", type=int, default=40, help="pixels of a side of the feature map")
    p.add_argument("--channels", type=int, default=256)
    p.add_argument("--hidden", type=int, default=1024)
    args = p.parse_args()
    n, c, hidden = args.n, args.channels, args.hidden
    g = torch.Generator(device="cuda").manual_seed(0)

    def rand(*shape):
        return torch.randn(*shape, generator=g, device="cuda")

    x = rand(n, args.size, args.size, c).bfloat16()
    w = (rand(c, 3, 3, c) * (2 / (9 * c)) ** 0.5).bfloat16()
    scale, bias = 1 + 0.1 * rand(c), 0.1 * rand(c)
    w1, w2 = rand(hidden, c) / c ** 0.5, rand(c, hidden) / hidden ** 0.5
    gamma, beta, b1, b2 = 1 + 0.1 * rand(c), 0.1 * rand(c), 0.1 * rand(hidden), 0.1 * rand(c)
    block = TokenBlock(gamma, beta, w1, b1, w2, b2)

    def step():
        return block(capi.forward(x, w, scale, bias, stride=1, pad=1))

    h = capi.forward(x, w, scale, bias, stride=1, pad=1)
    branch = (step().float() - h.float())
    f = torch.nn.functional
    want = f.linear(f.silu(f.linear(f.layer_norm(h.float(), (c,), gamma, beta, 1e-5), w1, b1)), w2, b2)
    print(f"int8 branch against fp32: {float((branch - want).norm() / want.norm()):.4f} of its norm")
    for _ in range(3):
        step()
    start, stop = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    start.record()
    for _ in range(50):
        step()
    stop.record()
    stop.synchronize()
    print(f"convolution and block on {n * args.size ** 2} tokens: {start.elapsed_time(stop) * 20:.1f} us")
    losses = block.tune_norm(h, f.layer_norm(h.float(), (c,), 1 + 0.1 * rand(c), 0.1 * rand(c), 1e-5))
    print(f"tuning the norm: loss {losses[0]:.4f} -> {losses[-1]:.6f} in {len(losses)} steps")
    adapters, rank = 4, 16
    index = (torch.arange(h.numel() // c, device="cuda") * adapters // (h.numel() // c)).int()
    shared = AdaptedProjection(gamma, w1, b1, rand(adapters, rank, c) / c ** 0.5, 0.1 * rand(adapters, hidden, rank))
    wanted = AdaptedProjection(gamma, w1, b1, rand(adapters, rank, c) / c ** 0.5, 0.1 * rand(adapters, hidden, rank))
    for _ in range(3):
        shared(h, x, index)
    start.record()
    for _ in range(50):
        shared(h, x, index)
    stop.record()
    stop.synchronize()
    print(f"projection with {adapters} adapters of rank {rank}: {start.elapsed_time(stop) * 20:.1f} us")
    losses = shared.tune(h, x, index, wanted(h, x, index)[0].float())
    print(f"tuning the adapters: loss {losses[0]:.4f} -> {losses[-1]:.6f} in {len(losses)} steps")
    capi.check()


if __name__ == "__main__":
    _main()
