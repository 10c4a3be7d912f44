"""Low-rank adapters without a GPU: the 64-bit oracle against a hand case and difference quotients, and the C entry
points' refusals (each returns its status before any CUDA call)."""
import numpy as np
import pytest

from oracle import token_ops as ref


@pytest.fixture(scope="module")
def capi():
    from conv2d_batchnorm_silu_gb300 import _build
    _build.build()
    from conv2d_batchnorm_silu_gb300 import capi
    return capi


def test_by_hand():
    y, hidden, total = ref.linear_adapters([[1.0, 2.0], [3.0, 4.0], [5.0, 6.0]], [1, -1, 2], [[[1.0, 0.0]], [[2.0, -1.0]]],
                                           [[[1.0], [1.0]], [[3.0], [-4.0]]], [1.0, 0.5], [[1.0, 1.0]] * 3)
    # row 0: hidden 2 - 2 = 0; the others have no adapter
    assert hidden.tolist() == [[0.0], [0.0], [0.0]] and y.tolist() == [[1.0, 1.0]] * 3 and total[0].tolist() == [7.0, 9.0]


def test_gradient_by_difference_quotients():
    rng = np.random.default_rng(1)
    x, a, b, dy = rng.normal(size=(4, 5)), rng.normal(size=(2, 3, 5)), rng.normal(size=(2, 6, 3)), rng.normal(size=(4, 6))
    index, scale, step = [1, 0, 7, 1], [0.5, 2.0], 1e-5
    hidden = ref.linear_adapters(x, index, a, b, scale)[1]
    grads, terms = ref.linear_adapters_backward(dy, x, index, a, b, scale, hidden)

    def loss(x, a, b):
        return float((ref.linear_adapters(x, index, a, b, scale)[0] * dy).sum())

    for which, grad in enumerate(grads):
        assert (np.abs(grad) <= terms[which] + 1e-12).all()
        for i in np.ndindex(grad.shape):
            up, down = [v.copy() for v in (x, a, b)], [v.copy() for v in (x, a, b)]
            up[which][i] += step
            down[which][i] -= step
            # central differences: truncation ~ step^2, rounding ~ 2^-52 / step, of values of order 100
            assert abs((loss(*up) - loss(*down)) / (2 * step) - grad[i]) < 1e-7


P, Q = 1 << 20, 1 << 21  # stand-ins for device pointers: refused calls never touch them


def test_forward_refusals(capi):
    bad, mis = capi.CBS_ERR_INVALID_ARG, capi.CBS_ERR_MISALIGNED

    def status(x=P, sx=16, index=P, a=P, b=P, scale=None, base=None, sb=24, y=Q, sy=24, hidden=None, m=4, k=16, n=24, rank=8,
               adapters=2, dtype=1, work=Q, size=1 << 30):
        return capi.raw_status("conv_bn_silu_linear_adapters", x, sx, index, a, b, scale, base, sb, y, sy, hidden, m, k, n, rank,
                               adapters, dtype, work, size, None)

    assert status(m=0) == capi.CBS_OK and status(m=0, x=None) == capi.CBS_OK
    for name in ("x", "index", "a", "b", "y"):
        assert status(**{name: None}) == bad, name
    assert status(m=-1) == bad and status(m=(1 << 20) + 1) == bad and status(k=0) == bad and status(n=0) == bad
    assert status(rank=0) == bad and status(rank=129) == bad and status(adapters=0) == bad and status(adapters=4097) == bad
    assert status(k=(1 << 22) + 1) == bad and status(dtype=3) == bad and status(dtype=-1) == bad
    assert status(sx=-1) == bad and status(sy=23) == bad and status(base=P, sb=-1) == bad and status(base=Q, sb=32) == bad
    assert status(x=P + 1) == mis and status(index=P + 2) == mis and status(a=P + 1) == mis and status(b=P + 1) == mis
    assert status(scale=P + 2) == mis and status(hidden=P + 2) == mis and status(y=Q + 1) == mis and status(work=Q + 8) == mis
    for sizes in ((-1, 16, 24, 8, 2), (4, 0, 24, 8, 2), (4, 16, 24, 129, 2), (4, 16, 24, 8, 4097)):
        assert capi.raw_status("conv_bn_silu_linear_adapters_workspace", *sizes) == -1
        assert capi.raw_status("conv_bn_silu_linear_adapters_backward_workspace", *sizes) == -1


def test_backward_refusals(capi):
    bad, mis = capi.CBS_ERR_INVALID_ARG, capi.CBS_ERR_MISALIGNED

    def status(dy=P, sdy=24, x=P, sx=16, index=P, a=P, b=P, scale=None, hidden=P, base=None, sb=16, dx=Q, sdx=16, da=Q, db=Q, m=4,
               k=16, n=24, rank=8, adapters=2, dtype=1, work=Q, size=1 << 30):
        return capi.raw_status("conv_bn_silu_linear_adapters_backward", dy, sdy, x, sx, index, a, b, scale, hidden, base, sb, dx,
                               sdx, da, db, m, k, n, rank, adapters, dtype, work, size, None)

    for name in ("dy", "x", "index", "a", "b", "hidden", "dx", "da", "db", "work"):
        assert status(**{name: None}) == bad, name
    assert status(m=-1) == bad and status(rank=0) == bad and status(adapters=0) == bad and status(dtype=9) == bad
    assert status(sdy=-1) == bad and status(sdx=15) == bad and status(base=Q, sb=24) == bad
    for name in ("dy", "x", "a", "b", "dx"):
        assert status(**{name: P + 1}) == mis, name
    for name in ("index", "scale", "hidden", "da", "db", "work"):
        assert status(**{name: P + 2}) == mis, name
