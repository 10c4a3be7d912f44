"""The convolution layer followed by a token-wise block on its pixels, in int8.

A feature map that the fused layer leaves as [n, h, w, c] is n*h*w tokens of c channels in memory
already.  On them runs, with a hidden width of its own,

    y = h + W2 SiLU(W1 LN(h) + b1) + b2

as four calls: ``layer_norm_quantize`` (the norm's output as int8 with a scale per token),
``linear_int8`` with SiLU, ``quantize_rows`` of the hidden rows, ``linear_int8`` with the residual.
The weights are quantised once, by ``quantize_rows`` too: a scale per output channel.

``TokenBlock.tune_norm`` trains the norm's gamma and beta towards given rows with ``layer_norm`` and
``layer_norm_backward``.

    python -m conv2d_batchnorm_silu_gb300.token_block [--n 16] [--size 40] [--channels 256] [--hidden 1024]

prints how far the int8 block is from the same block in fp32, its time and the loss of a short tuning.
Needs a GPU.
"""
from __future__ import annotations

import argparse

import torch

from . import capi


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
    capi.check()


if __name__ == "__main__":
    _main()
