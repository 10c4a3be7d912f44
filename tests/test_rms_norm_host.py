"""The RMS norm and the AdamW step without a GPU: the 64-bit oracle against hand cases and difference
quotients, and the C entry points' refusals (each returns its status before any CUDA call)."""
import ctypes

import numpy as np
import pytest

from oracle import token_ops as ref


@pytest.fixture(scope="module")
def capi():
    from conv2d_batchnorm_silu_gb300 import _build
    _build.build()
    from conv2d_batchnorm_silu_gb300 import capi
    return capi


def test_rms_norm_by_hand():
    y, rstd = ref.rms_norm([[1.0, 7.0]], [2.0, 3.0], eps=0.0)  # mean square 25
    assert np.allclose(rstd, 0.2) and np.allclose(y, [[0.4, 4.2]])


def test_rms_norm_gradient_by_difference_quotients():
    rng = np.random.default_rng(1)
    x, dy, gamma, eps, step = rng.normal(size=(3, 7)), rng.normal(size=(3, 7)), rng.uniform(0.5, 1.5, 7), 1e-3, 1e-5

    def loss(x, gamma):
        return float((ref.rms_norm(x, gamma, eps)[0] * dy).sum())

    dx, dgamma = ref.rms_norm_backward(dy, x, gamma, ref.rms_norm(x, gamma, eps)[1])
    for array, grad, which in ((x, dx, 0), (gamma, dgamma, 1)):
        for i in np.ndindex(array.shape):
            up, down = array.copy(), array.copy()
            up[i] += step
            down[i] -= step
            pair = [(up, gamma), (down, gamma)] if which == 0 else [(x, up), (x, down)]
            # central differences: truncation ~ step^2, rounding ~ 2^-52 / step, of values of order 10
            assert abs((loss(*pair[0]) - loss(*pair[1])) / (2 * step) - grad[i]) < 1e-8


def test_adamw_by_hand():
    # the first step from zero moments: m / c1 = g, v / c2 = g^2, so the update is lr times the sign
    p, m, v = ref.adamw([1.0, -2.0], [0.5, -4.0], [0.0, 0.0], [0.0, 0.0], 1, 0.1, 0.9, 0.999, 0.0, 0.5, 2.0)
    assert np.allclose(p, [1.0 * 0.95 - 0.1, -2.0 * 0.95 + 0.1]) and np.allclose(m, [0.1, -0.8]) and np.allclose(v, [1e-3, 64e-3])


def test_the_dither_keeps_the_mean():
    a, b = ref.dither(1 << 16, 3)
    # 65536 numbers evenly spread: their mean within 6 of its own spread 0.289 / 256
    assert abs(a.mean() - 0.5) < 0.007 and abs(b.mean() - 0.5) < 0.007 and a.max() < 1 and len(np.unique(a)) > 30000
    assert ref.e4m3_distance(np.array([448.0, 16.0, 15.9, 1.0, 2.0 ** -6, 2.0 ** -9, 0.0])).tolist() == [
        32.0, 2.0, 1.0, 0.125, 2.0 ** -9, 2.0 ** -9, 2.0 ** -9]


P, Q = 1 << 20, 1 << 21  # stand-ins for device pointers: refused calls never touch them


@pytest.mark.parametrize("quantise", [False, True])
def test_rms_norm_refusals(capi, quantise):
    bad, mis = capi.CBS_ERR_INVALID_ARG, capi.CBS_ERR_MISALIGNED

    def status(x=P, sx=8, res=None, sres=8, gamma=None, eps=1e-6, total=None, st=8, y=Q, sy=8, q=Q, sq=8, scale=Q,
               rstd=None, rows=4, c=8, dtype=1):
        if quantise:
            return capi.raw_status("conv_bn_silu_rms_norm_quantize", x, sx, res, sres, gamma, eps, total, st, y, sy, q, sq,
                                   scale, rstd, rows, c, dtype, None)
        return capi.raw_status("conv_bn_silu_rms_norm", x, sx, res, sres, gamma, eps, total, st, y, sy, rstd, rows, c,
                               dtype, None)

    assert status(rows=0) == capi.CBS_OK and status(rows=0, q=None) == capi.CBS_OK
    assert status(x=None) == bad and status(rows=-1) == bad and status(c=0) == bad and status(dtype=3) == bad
    assert status(c=(1 << 29) + 1) == bad and status(sx=-1) == bad and status(sy=7) == bad
    assert status(eps=-1.0) == bad and status(eps=float("nan")) == bad and status(eps=float("inf")) == bad
    assert status(res=P) == bad and status(res=P, total=Q, st=7) == bad and status(res=P, total=Q, sres=-1) == bad
    assert status(res=P, total=P, sres=8, st=9) == bad  # in place, but row by row elsewhere
    assert status(x=P + 1) == mis and status(y=Q + 1) == mis and status(rstd=Q + 2) == mis and status(gamma=P + 2) == mis
    assert status(res=P + 1, total=Q) == mis and status(res=P, total=Q + 1) == mis
    if quantise:
        assert status(q=None) == bad and status(scale=None) == bad and status(sq=7) == bad and status(scale=Q + 1) == mis
    else:
        assert status(y=None) == bad


def test_rms_norm_backward_refusals(capi):
    bad, mis = capi.CBS_ERR_INVALID_ARG, capi.CBS_ERR_MISALIGNED
    ok = [P, 8, P, 8, None, P, None, 8, Q, 8, Q, 4, 8, 1, Q, 1 << 20, None]

    def status(**change):
        args = list(ok)
        for i, v in change.items():
            args[int(i[1:])] = v
        return capi.raw_status("conv_bn_silu_rms_norm_backward", *args)

    for i in (0, 2, 5, 8, 10, 14):
        assert status(**{f"_{i}": None}) == bad, i
    assert status(_11=-1) == bad and status(_12=0) == bad and status(_13=7) == bad and status(_9=7) == bad
    assert status(_6=Q, _7=16) == bad and status(_6=P, _7=-1) == bad
    for i in (0, 2, 6, 8, 10, 14):
        assert status(**{f"_{i}": Q + 1}) == mis, i
    assert capi.raw_status("conv_bn_silu_rms_norm_backward_workspace", -1, 8) == -1
    assert capi.raw_status("conv_bn_silu_rms_norm_backward_workspace", 1, 0) == -1


def test_adamw_refusals(capi):
    bad, mis = capi.CBS_ERR_INVALID_ARG, capi.CBS_ERR_MISALIGNED

    def status(tensors=((),), count=None, null=False, **options):
        table = (capi.AdamWTensor * max(1, len(tensors)))()
        for t, change in zip(table, tensors):
            values = dict(param=P, grad=Q, exp_avg=P, exp_avg_sq=P, exp_avg_scale=P, exp_avg_sq_scale=P, n=16, param_dtype=1,
                          grad_dtype=0)
            for name, value in {**values, **dict(change)}.items():
                setattr(t, name, value)
        o = capi.AdamWOptions(lr=1e-3, beta1=0.9, beta2=0.999, eps=1e-8, weight_decay=0.1, grad_scale=1.0, step=1, state_bits=8)
        for name, value in options.items():
            setattr(o, name, value)
        return capi.raw_status("conv_bn_silu_adamw_step", None if null else table, len(tensors) if count is None else count,
                               ctypes.byref(o), None)

    assert status(tensors=()) == capi.CBS_OK and status(tensors=(dict(n=0, param=None),)) == capi.CBS_OK
    assert status(null=True) == bad and status(count=-1) == bad
    assert capi.raw_status("conv_bn_silu_adamw_step", None, 0, None, None) == bad
    for name in ("param", "grad", "exp_avg", "exp_avg_sq", "exp_avg_scale", "exp_avg_sq_scale"):
        assert status(tensors=({name: None},)) == bad, name
    assert status(tensors=(dict(n=-1),)) == bad and status(tensors=(dict(n=(1 << 40) + 1),)) == bad
    assert status(tensors=(dict(param_dtype=3),)) == bad and status(tensors=(dict(grad_dtype=-1),)) == bad
    assert status(tensors=(dict(param=P + 1),)) == mis and status(tensors=(dict(grad=Q + 2),)) == mis
    assert status(tensors=(dict(exp_avg_scale=P + 2),)) == mis and status(tensors=(dict(exp_avg=P + 2),), state_bits=32) == mis
    assert status(tensors=((), ())) == bad and status(tensors=((), dict(param=P + 30))) == bad  # parameters that overlap
    for change in (dict(lr=float("nan")), dict(beta1=1.0), dict(beta2=-0.1), dict(eps=-1.0), dict(eps=float("inf")),
                   dict(weight_decay=float("inf")), dict(grad_scale=float("nan")), dict(step=0), dict(state_bits=16)):
        assert status(**change) == bad, change
    assert status(lr_device=P + 2) == mis and status(step_device=P + 4, step=0) == mis
