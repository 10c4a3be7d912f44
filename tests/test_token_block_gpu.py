"""The token-wise block behind the convolution layer against the same block in 64 bits.  The bound follows
each rounding through the block: half a step for a quantised element, and the types' roundings."""
import numpy as np
import pytest
import torch

from oracle import token_ops as ref

pytestmark = pytest.mark.gpu
E32 = 2.0 ** -24


def host(t):
    return t.detach().double().cpu().numpy()


def rand(seed, *shape):
    return torch.randn(*shape, generator=torch.Generator().manual_seed(seed)).cuda()


def feature_map(n, size, c):
    from conv2d_batchnorm_silu_gb300 import capi
    x, w = rand(1, n, size, size, c).bfloat16(), (rand(2, c, 3, 3, c) * (2 / (9 * c)) ** 0.5).bfloat16()
    return capi.forward(x, w, 1 + 0.1 * rand(3, c), 0.1 * rand(4, c), stride=1, pad=1)


def product(a, da, w, dw):
    """a w^T, and how far it may be off when the factors are off by up to da and dw."""
    return a @ w.T, da @ np.abs(w).T + np.abs(a) @ dw.T + da @ dw.T


@pytest.mark.parametrize("n,size,c,hidden", [(2, 12, 64, 192), (1, 1, 128, 512), (3, 20, 256, 1024)])
def test_block(n, size, c, hidden):
    from conv2d_batchnorm_silu_gb300 import capi
    from conv2d_batchnorm_silu_gb300.token_block import TokenBlock
    h = feature_map(n, size, c)
    gamma, beta, b1, b2 = 1 + 0.1 * rand(5, c), 0.1 * rand(6, c), 0.1 * rand(7, hidden), 0.1 * rand(8, c)
    w1, w2 = rand(9, hidden, c) / c ** 0.5, rand(10, c, hidden) / hidden ** 0.5
    y = TokenBlock(gamma, beta, w1, b1, w2, b2)(h)
    assert y.shape == h.shape and y.dtype == h.dtype
    capi.check()

    def step(v, dv):  # a row's quantised elements are off by dv and by half a step of its largest, plus roundings
        return dv + (np.abs(v).max(-1, keepdims=True) + dv.max(-1, keepdims=True)) / 127 * (0.5 + 127 * 8 * E32)

    rows = host(h).reshape(-1, c)
    v, mean, rstd = ref.layer_norm(rows, host(gamma), host(beta), 1e-5)
    dv = 1e-5 * (np.abs(v) + rstd[:, None] * np.abs(rows).max(1, keepdims=True) + 1)  # fp32, rows of at most 256
    z, dz = product(v, step(v, dv), host(w1), step(host(w1), 0 * host(w1)))
    u, du = ref.activate(z + host(b1), "silu"), 1.1 * dz
    du = du + 2.0 ** -8 * (np.abs(u) + du) + 1e-5  # bf16
    out, dout = product(u, step(u, du), host(w2), step(host(w2), 0 * host(w2)))
    want = rows + out + host(b2)
    off = np.abs(host(y).reshape(-1, c) - want)
    assert (off <= dout + 2.0 ** -8 * 1.001 * (np.abs(want) + dout) + 1e-5 * (1 + np.abs(out))).all()


def test_tuning_the_norm_follows_the_gradient():
    from conv2d_batchnorm_silu_gb300.token_block import TokenBlock
    c = 64
    h = feature_map(2, 12, c).float()
    gamma, beta = 1 + 0.1 * rand(5, c), 0.1 * rand(6, c)
    block = TokenBlock(gamma, beta, rand(9, 96, c), rand(7, 96), rand(10, c, 96), rand(8, c))
    target = torch.nn.functional.layer_norm(h, (c,), 1 + 0.1 * rand(11, c), 0.1 * rand(12, c), 1e-5)
    losses = block.tune_norm(h, target, steps=3)
    # the same steps in 64 bits
    rows, t = host(h).reshape(-1, c), host(target).reshape(-1, c)
    hat = (rows - rows.mean(1, keepdims=True)) / np.sqrt(rows.var(1, keepdims=True) + 1e-5)
    g, b = host(gamma), host(beta)
    for loss in losses:
        off = hat * g + b - t
        assert abs(loss - np.square(off).sum() / (2 * len(rows))) <= 1e-4 * loss + 1e-6
        g, b = g - 0.2 * (off * hat).sum(0) / len(rows), b - 0.2 * off.sum(0) / len(rows)
    assert np.abs(host(block.gamma) - g).max() <= 1e-4 and np.abs(host(block.beta) - b).max() <= 1e-4
    assert losses[2] < losses[1] < losses[0]


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
def test_tuning_over_many_tokens_in_16_bits(dtype):
    # The error of a token divided by a million of them is nothing in f16, so the gradient has to be of its sum.
    from conv2d_batchnorm_silu_gb300.token_block import TokenBlock
    tokens, c, steps = 1 << 20, 16, 60
    h = torch.randn(tokens, c, generator=torch.Generator("cuda").manual_seed(1), device="cuda").to(dtype)
    want_gamma, want_beta = 1 + 0.1 * rand(11, c), 0.1 * rand(12, c)
    block = TokenBlock(torch.ones(c).cuda(), torch.zeros(c).cuda(), rand(9, 32, c), rand(7, 32), rand(10, c, 32), rand(8, c))
    target = torch.nn.functional.layer_norm(h.float(), (c,), want_gamma, want_beta, 1e-5)
    losses = block.tune_norm(h, target, steps=steps)
    # Each step leaves 0.8 of an error of at most 0.4, and takes 0.2 of the mean of what rounding y to the type adds
    # (at most a unit roundoff of |y| times |h|, both of mean square 1.3 and 1), so at most one such mean remains.
    unit = 2.0 ** -11 if dtype == torch.float16 else 2.0 ** -8
    left = 0.4 * 0.8 ** steps + 1.3 * unit
    assert float((block.gamma - want_gamma).abs().max()) <= left and float((block.beta - want_beta).abs().max()) <= left
    assert losses[-1] < losses[0]
