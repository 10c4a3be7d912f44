"""Token-wise operators without a GPU: the 64-bit oracle against hand cases and difference
quotients, and the C entry points' refusals (each returns its status before any CUDA call)."""
import numpy as np
import pytest

from oracle import token_ops as ref


@pytest.fixture(scope="module")
def capi():
    from conv2d_batchnorm_silu_gb300 import _build
    _build.build()
    from conv2d_batchnorm_silu_gb300 import capi
    return capi


def test_layer_norm_by_hand():
    # mean 2, deviations -1 and 1, variance 1
    y, mean, rstd = ref.layer_norm([[1.0, 3.0]], [2.0, 3.0], [0.5, -0.5], eps=0.0)
    assert mean[0] == 2.0 and rstd[0] == 1.0
    assert y.tolist() == [[-1.5, 2.5]]


def test_layer_norm_gradient_by_difference_quotients():
    rng = np.random.default_rng(1)
    x, dy = rng.normal(size=(3, 7)), rng.normal(size=(3, 7))
    gamma, beta, eps, step = rng.uniform(0.5, 1.5, 7), rng.normal(size=7), 1e-3, 1e-5

    def loss(x, gamma, beta):
        return float((ref.layer_norm(x, gamma, beta, eps)[0] * dy).sum())

    def quotient(arrays, which):
        out = np.zeros_like(arrays[which])
        for i in np.ndindex(out.shape):
            up, down = [a.copy() for a in arrays], [a.copy() for a in arrays]
            up[which][i] += step
            down[which][i] -= step
            out[i] = (loss(*up) - loss(*down)) / (2 * step)
        return out

    mean, rstd = ref.moments(x, eps)
    got = ref.layer_norm_backward(dy, x, gamma, mean, rstd)
    for which, g in enumerate(got):
        # central differences: truncation ~ step^2, rounding ~ 2^-52 / step, of values of order 10
        assert np.abs(g - quotient([x, gamma, beta], which)).max() < 1e-8


def test_quantisation_by_hand():
    q, scale = ref.quantize_rows_f32([[0.0, 0.0], [-127.0, 63.5], [1.0, -0.25]])
    assert q.tolist() == [[0, 0], [-127, 64], [127, -32]]
    assert scale[1] == 1.0 and scale[0] > 0
    assert np.allclose(ref.row_scales([[1.0, -2.0]]), 2.0 / 127.0)


def test_linear_by_hand():
    y, z, total = ref.linear_int8([[1, -2]], [[3, 4], [-5, 6]], [0.5], [2.0, 1.0], [1.0, 0.0], "relu", [[0.25, 0.25]])
    assert z.tolist() == [[-4.0, -8.5]] and y.tolist() == [[0.25, 0.25]] and total.tolist() == [[11.0, 17.0]]


P, Q = 1 << 20, 1 << 21  # stand-ins for device pointers: refused calls never touch them


def test_layer_norm_refusals(capi):
    bad, mis = capi.CBS_ERR_INVALID_ARG, capi.CBS_ERR_MISALIGNED
    ok = [P, 8, None, None, 1e-5, Q, 8, None, 4, 8, 1, None]

    def status(**change):
        args = list(ok)
        for i, v in change.items():
            args[int(i[1:])] = v
        return capi.raw_status("conv_bn_silu_layer_norm", *args)

    assert status(_8=0) == capi.CBS_OK                     # no rows: nothing to do
    assert status(_0=None) == bad and status(_5=None) == bad
    assert status(_8=-1) == bad and status(_9=0) == bad and status(_9=-3) == bad
    assert status(_1=-1) == bad and status(_6=7) == bad    # negative distance; rows of y overlap
    assert status(_4=-1.0) == bad and status(_4=float("nan")) == bad and status(_4=float("inf")) == bad
    assert status(_10=3) == bad and status(_10=-1) == bad
    assert status(_0=P + 1) == mis and status(_5=Q + 1) == mis and status(_2=P + 2) == mis and status(_7=P + 2) == mis


def test_layer_norm_backward_refusals(capi):
    bad, mis = capi.CBS_ERR_INVALID_ARG, capi.CBS_ERR_MISALIGNED
    ok = [P, 8, P, 8, None, P, Q, 8, Q, Q, 4, 8, 1, Q, 1 << 20, None]

    def status(**change):
        args = list(ok)
        for i, v in change.items():
            args[int(i[1:])] = v
        return capi.raw_status("conv_bn_silu_layer_norm_backward", *args)

    for i in (0, 2, 5, 6, 8, 9, 13):
        assert status(**{f"_{i}": None}) == bad, i
    assert status(_10=-1) == bad and status(_11=0) == bad and status(_12=7) == bad and status(_7=7) == bad
    for i in (0, 2, 6, 8, 9, 13):
        assert status(**{f"_{i}": Q + 1}) == mis, i
    assert capi.raw_status("conv_bn_silu_layer_norm_backward_workspace", -1, 8) == -1
    assert capi.raw_status("conv_bn_silu_layer_norm_backward_workspace", 1, 0) == -1


@pytest.mark.parametrize("name", ["conv_bn_silu_quantize_rows", "conv_bn_silu_layer_norm_quantize"])
def test_quantise_refusals(capi, name):
    bad, mis = capi.CBS_ERR_INVALID_ARG, capi.CBS_ERR_MISALIGNED
    norm = name.endswith("norm_quantize")

    def status(x=P, sx=8, eps=1e-5, q=Q, sq=8, scale=Q, rows=4, c=8, dtype=1):
        mid = (None, None, eps) if norm else ()
        return capi.raw_status(name, x, sx, *mid, q, sq, scale, rows, c, dtype, None)

    assert status(rows=0) == capi.CBS_OK and status(rows=0, q=None) == capi.CBS_OK
    assert status(x=None) == bad and status(q=None) == bad and status(scale=None) == bad
    assert status(rows=-1) == bad and status(c=0) == bad and status(dtype=4) == bad
    assert status(sx=-1) == bad and status(sq=7) == bad
    assert status(x=P + 1) == mis and status(scale=Q + 2) == mis
    if norm:
        assert status(eps=-1e-5) == bad


def test_linear_refusals(capi):
    bad, mis = capi.CBS_ERR_INVALID_ARG, capi.CBS_ERR_MISALIGNED

    def status(a=P, sa=8, w=P, sw=8, a_scale=P, w_scale=P, bias=None, residual=None, sr=8, y=Q, sy=8, m=4, n=8, k=8,
               act=1, out=1, work=None, work_bytes=0):
        return capi.raw_status("conv_bn_silu_linear_int8", a, sa, w, sw, a_scale, w_scale, bias, residual, sr, y, sy,
                               m, n, k, act, out, work, work_bytes, None)

    assert status(m=0) == capi.CBS_OK and status(n=0) == capi.CBS_OK
    for name in ("a", "w", "a_scale", "w_scale", "y"):
        assert status(**{name: None}) == bad, name
    assert status(m=-1) == bad and status(n=-1) == bad and status(k=-1) == bad
    assert status(k=131072) == bad and status(n=(1 << 22) + 1) == bad
    assert status(act=3) == bad and status(act=-1) == bad and status(out=3) == bad
    assert status(sa=-1) == bad and status(sw=-1) == bad and status(sy=7) == bad
    assert status(y=Q + 1) == mis and status(a_scale=P + 1) == mis and status(w_scale=P + 2) == mis
    assert status(bias=P + 1) == mis and status(residual=P + 1) == mis and status(work=Q + 8) == mis
    assert capi.raw_status("conv_bn_silu_linear_int8_workspace", -1, 8, 8) == -1
    assert capi.raw_status("conv_bn_silu_linear_int8_workspace", 8, 8, 131072) == -1
