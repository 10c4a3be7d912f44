"""The norm, the projection in int8, the adapters and the AdamW step used together, against the same in 64 bits."""
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


def made(c, n, rank, adapters):
    from conv2d_batchnorm_silu_gb300.token_block import AdaptedProjection
    return AdaptedProjection(1 + 0.1 * rand(1, c), rand(2, n, c) / c ** 0.5, 0.1 * rand(3, n), rand(4, adapters, rank, c) / c ** 0.5,
                             0.3 * rand(5, adapters, n, rank), 0.5 + torch.rand(adapters, generator=torch.Generator().manual_seed(6)).cuda())


@pytest.mark.parametrize("rows,c,n,rank,adapters", [(1, 64, 96, 8, 2), (48, 256, 512, 16, 5), (700, 128, 192, 16, 3), (2600, 64, 128, 16, 2)])
def test_projection(rows, c, n, rank, adapters):
    from conv2d_batchnorm_silu_gb300 import capi
    block = made(c, n, rank, adapters)
    h, residual = rand(7, rows, c).bfloat16(), rand(8, rows, c).bfloat16()
    index = torch.randint(-1, adapters, (rows,), generator=torch.Generator().manual_seed(9)).int().cuda()
    z, total = block(h, residual, index)
    capi.check()
    assert torch.equal(total, (h.float() + residual.float()).bfloat16()) and z.shape == (rows, n)
    y, _ = ref.rms_norm(host(total), host(block.gamma), block.eps)
    # The int8 rows and weights are off by half a step of their largest (and fp32's roundings); the shared product is
    # rounded to bf16, its output again with the adapters', whose y, hidden rows and weights are bf16 as well.
    half = 0.5 + 127 * 16 * E32
    dy, dw = np.abs(y).max(1, keepdims=True) / 127 * half, host(block.w_scale)[:, None] * half
    w = host(block.w) * host(block.w_scale)[:, None]
    shared = y @ w.T + host(block.bias)
    off = dy * np.abs(w).sum(1)[None, :] + 1e-5 * (np.abs(y) @ np.abs(w).T)
    off = off + 2.0 ** -8 * 1.01 * (np.abs(shared) + off)
    a, b = block.a.bfloat16(), block.b.bfloat16()
    delta, _, terms = ref.linear_adapters(y, index.cpu().numpy(), host(a), host(b), host(block.scale))
    off = off + 3 * 2.0 ** -8 * terms
    want = shared + delta
    assert (np.abs(host(z) - want) <= off + 2.0 ** -8 * 1.01 * (np.abs(want) + off) + 1e-6).all() and dw.max() > 0


def test_a_training_step_follows_the_chain_rule():
    """Norm with residual, adapters, a squared error, the gradients back to x and every parameter, and AdamW: in fp32,
    against PyTorch's autograd in 64 bits.  Values are of order 1 to 30 and pass some 10 sums of up to 160 terms, each
    within 2^-20 of its terms; AdamW's first step is lr times a sign, where gradients stay off zero."""
    from conv2d_batchnorm_silu_gb300 import capi
    rows, c, n, rank, adapters = 90, 96, 64, 8, 3
    x, residual, target = rand(1, rows, c), rand(2, rows, c), rand(3, rows, n)
    gamma, a, b = 1 + 0.1 * rand(4, c), rand(5, adapters, rank, c) / c ** 0.5, 0.3 * rand(6, adapters, n, rank)
    scale = torch.tensor([0.5, 1.0, 2.0], device="cuda")
    index = torch.randint(-1, adapters, (rows,), generator=torch.Generator().manual_seed(7)).int().cuda()
    y, total, rstd = capi.rms_norm(x, gamma, 1e-6, residual=residual, return_rstd=True)
    z, hidden = capi.linear_adapters(y, index, a, b, scale, return_hidden=True)
    dz = z - target
    dy, da, db = capi.linear_adapters_backward(dz, y, index, a, b, scale, hidden)
    past = rand(8, rows, c)
    dx, dgamma = capi.rms_norm_backward(dy, total, gamma, rstd, residual=past)

    leaves = [t.double().requires_grad_() for t in (x, gamma, a, b)]
    xd, gd, ad, bd = leaves
    t = xd + residual.double()
    yd = t * (t.square().mean(1, keepdim=True) + 1e-6).rsqrt() * gd
    at = index.long().clamp(min=0)
    s = torch.where(index >= 0, scale.double()[at], torch.zeros((), dtype=torch.float64, device="cuda"))
    zd = s[:, None] * torch.einsum("mnr,mr->mn", bd[at], torch.einsum("mrk,mk->mr", ad[at], yd))
    ((zd - target.double()).square().sum() / 2 + (t * past.double()).sum()).backward()
    for got, leaf in zip((dx, dgamma, da, db), leaves):
        assert (got.double() - leaf.grad).abs().max() <= 2e-5 * leaf.grad.abs().max()

    params, before = [gamma, a, b], [host(p) for p in (gamma, a, b)]
    capi.adamw_step(params, [dgamma, da, db], step=1, lr=1e-3, weight_decay=0.1, **capi.adamw_state(params))
    for p, old, leaf in zip(params, before, leaves[1:]):
        grad = leaf.grad.cpu().numpy()
        want, _, _ = ref.adamw(old, grad, 0 * grad, 0 * grad, 1, 1e-3, 0.9, 0.999, 1e-8, 0.1)
        clear = np.abs(grad) > 1e-3
        assert (np.abs(host(p) - want)[clear] <= 1e-6).all() and clear.mean() > 0.5


@pytest.mark.parametrize("dtype,bits", [(torch.float32, 32), (torch.bfloat16, 8), (torch.float16, 8)])
def test_tuning_runs_in_every_type(dtype, bits):
    from conv2d_batchnorm_silu_gb300 import capi
    block = made(64, 80, 8, 3)
    h, residual = rand(7, 300, 64).to(dtype), rand(8, 300, 64).to(dtype)
    index = torch.randint(-1, 3, (300,), generator=torch.Generator().manual_seed(9)).int().cuda()
    start = [block.a.clone(), block.b.clone()]
    losses = block.tune(h, residual, index, rand(10, 300, 80), steps=4, bits=bits)
    capi.check()
    assert len(losses) == 4 and all(np.isfinite(losses))
    for p, old in zip((block.a, block.b), start):
        moved = (p - old).abs()
        assert p.isfinite().all() and 0 < float(moved.max()) <= 4 * 1e-2 * 1.5  # lr a step, and no more than some of it beyond


def test_a_captured_training_step():
    """The whole step in one graph, its step number on the device, gives what the calls give one by one."""
    from conv2d_batchnorm_silu_gb300 import capi
    rows, c, n, rank, adapters = 600, 64, 48, 8, 2
    x, target = rand(1, rows, c).bfloat16(), rand(2, rows, n).bfloat16()
    index = torch.randint(-1, adapters, (rows,), generator=torch.Generator().manual_seed(3)).int().cuda()

    def parts():
        a, b = (rand(4, adapters, rank, c) / c ** 0.5).bfloat16(), (0.3 * rand(5, adapters, n, rank)).bfloat16()
        return a, b, capi.adamw_state([a, b], 8)

    def one(a, b, state, step):
        z, hidden = capi.linear_adapters(x, index, a, b, None, return_hidden=True)
        _, da, db = capi.linear_adapters_backward(z - target, x, index, a, b, None, hidden)
        capi.adamw_step([a, b], [da, db], step=step, lr=1e-2, grad_scale=1.0 / rows, **state)

    a, b, state = parts()
    number = torch.ones(1, dtype=torch.int64, device="cuda")
    one(*parts(), 1)  # loads everything before the capture
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        one(a, b, state, number)
        number.add_(1)
    a2, b2, state2 = parts()
    for t in range(1, 6):
        graph.replay()
        one(a2, b2, state2, torch.full((1,), t, dtype=torch.int64, device="cuda"))
    assert int(number) == 6
    for p, q in ((a, a2), (b, b2)):
        assert torch.equal(p, q)
    for name in state:
        for p, q in zip(state[name], state2[name]):
            assert torch.equal(p.view(torch.uint8), q.view(torch.uint8))
