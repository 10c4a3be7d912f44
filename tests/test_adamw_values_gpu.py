"""Values of the AdamW step that its other tests' bounds leave room for, against the 64-bit oracle."""
import numpy as np
import pytest
import torch

from oracle import token_ops as ref

pytestmark = pytest.mark.gpu
E32 = 2.0 ** -24


@pytest.fixture(scope="module")
def capi():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from conv2d_batchnorm_silu_gb300 import capi
    return capi


def host(t):
    return t.detach().double().cpu().numpy().reshape(-1)


def made(seed, n, size=1.0):
    return (torch.randn(n, generator=torch.Generator().manual_seed(seed)) * size).cuda()


@pytest.mark.parametrize("bits", [8, 32])
@pytest.mark.parametrize("on_device", [False, True])
@pytest.mark.parametrize("lr", [1e-3, 1e-4, 1e-5, 2e-6])
def test_small_decays_are_kept(capi, lr, on_device, bits):
    """A fp32 parameter is within half a step of its type, and the roundings of what it loses, of the 64-bit result:
    a decay of lr * 0.01, some steps of the type or a fraction of one, is neither lost nor rounded by itself."""
    n, rates = 20000, dict(betas=(0.9, 0.999), eps=1e-8, weight_decay=0.01)
    p, g = [made(1, n)], [made(2, n, 0.1)]
    before, state = host(p[0]), capi.adamw_state(p, bits)
    capi.adamw_step(p, g, step=1, lr=torch.full((1,), lr, device="cuda") if on_device else lr, **rates, **state)
    zero = np.zeros(n)
    want, _, _ = ref.adamw(before, host(g[0]), zero, zero, 1, lr, 0.9, 0.999, 1e-8, 0.01)
    # lr and the products, the moments, the root, the quotient and 1 - beta^step
    lost = 40 * E32 * (lr * 0.01 * np.abs(before) + lr)
    half = np.spacing(np.maximum(np.abs(want), np.abs(before)).astype(np.float32)).astype(np.float64) / 2
    off = host(p[0]) - want
    assert (np.abs(off) <= half + lost).all()
    # The roundings of p have no side: of n elements, off by up to half a step each, the mean is within some sigmas.
    relative = off / np.abs(before) * np.sign(before)
    assert abs(relative.mean()) <= 6 * (2 * half / np.abs(before)).std() / 12 ** 0.5 / n ** 0.5 + 6 * (half / np.abs(before)).mean() / n ** 0.5 + lost.mean()


def test_decay_alone_over_many_steps(capi):
    """Steps without gradients, so that the decay is all there is: at lr * decay = 1e-5 a step is some 100 steps of
    the type, each rounded to half of one, 2^-25 to 2^-24 of p; 500 of them leave p within 500 * 2^-24."""
    p = [made(1, 4096)]
    before, g, state = host(p[0]), [torch.zeros(4096, device="cuda")], capi.adamw_state(p)
    for step in range(1, 501):
        capi.adamw_step(p, g, step=step, lr=1e-3, weight_decay=0.01, **state)
    want = before * (1 - 1e-5) ** 500
    ratio = host(p[0]) / want - 1
    assert np.abs(ratio).max() <= 500 * E32
    assert abs(ratio.mean()) <= 50 * E32  # the roundings fall on both sides


@pytest.mark.parametrize("bits", [8, 32])
@pytest.mark.parametrize("eps", [1e-30, 1e-39, 1e-44, 1e-50, 1e-300])
def test_the_smallest_eps_keeps_elements_without_gradients(capi, eps, bits):
    """m = v = 0: the update is 0 / eps, and the decay, of half a step of the type and its own roundings, is all."""
    p, g = [made(1, 3000)], [torch.zeros(3000, device="cuda")]
    g[0][1::3] = 0.5
    before, state = host(p[0]), capi.adamw_state(p, bits)
    capi.adamw_step(p, g, step=1, lr=1e-3, eps=eps, weight_decay=0.1, **state)
    want = before * (1 - 1e-4) - 1e-3 * (host(g[0]) > 0)  # the first step's update is the gradient's sign
    assert (np.abs(host(p[0]) - want) <= E32 * np.abs(want) + 40 * E32 * (1e-4 * np.abs(before) + 1e-3)).all()


def test_the_spread_of_8_bit_roots_under_steady_gradients(capi):
    """4000 steps of normal gradients from their own moments on, four times as long as beta2 = 0.999 remembers.  Of a
    root r between values d apart, a step's change of 0.48 * 0.001 r on average is rounded with a variance of that times
    d, which v gains and forgets by a thousandth a step: v ends at 1 + 0.48 d / r, the root with half of that as its
    variance.  d / r is 1/16 to 1/8: the mean square 1.03 to 1.06, the mean 1.007 to 1.015, the spread 0.12 to 0.175, each
    with some room for 4096 elements (0.17 / 64 = 0.003 a sigma) and for where in the binades the roots lie."""
    p = [torch.zeros(4096, device="cuda")]
    state = capi.adamw_state(p, bits=8)
    state["exp_avg_sq"][0].copy_(torch.full((4096,), 256.0, device="cuda"))
    state["exp_avg_sq_scale"][0].fill_(1 / 256)
    gen = torch.Generator("cuda").manual_seed(5)
    for step in range(10001, 14001):
        capi.adamw_step(p, [torch.randn(4096, generator=gen, device="cuda")], step=step, lr=1e-4, weight_decay=0.0, **state)
    root = host(state["exp_avg_sq"][0].float()) * np.repeat(host(state["exp_avg_sq_scale"][0]), 256)
    assert 1.0 < root.mean() < 1.025 and 0.11 < root.std() < 0.19 and 1.02 < (root ** 2).mean() < 1.07
