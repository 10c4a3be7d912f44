"""Widths at which the index arithmetic of the token-wise kernels would leave 32 bits are refused before any CUDA call."""
import pytest


@pytest.fixture(scope="module")
def capi():
    from conv2d_batchnorm_silu_gb300 import _build
    _build.build()
    from conv2d_batchnorm_silu_gb300 import capi
    return capi


P, Q = 1 << 20, 1 << 21  # stand-ins for device pointers: refused calls never touch them


@pytest.mark.parametrize("c", [(1 << 29) + 1, 1 << 30, (1 << 31) - 256, (1 << 31) - 1])
def test_rows_that_are_too_wide(capi, c):
    bad = capi.CBS_ERR_INVALID_ARG
    for rows in (0, 1):
        assert capi.raw_status("conv_bn_silu_layer_norm", P, c, None, None, 1e-5, Q, c, None, rows, c, 1, None) == bad
        assert capi.raw_status("conv_bn_silu_quantize_rows", P, c, Q, c, Q, rows, c, 1, None) == bad
        assert capi.raw_status("conv_bn_silu_layer_norm_quantize", P, c, None, None, 1e-5, Q, c, Q, rows, c, 1, None) == bad
        assert capi.raw_status("conv_bn_silu_layer_norm_backward", P, c, P, c, None, P, Q, c, Q, Q, rows, c, 1, Q,
                               1 << 60, None) == bad
        assert capi.raw_status("conv_bn_silu_layer_norm_backward_workspace", rows, c) == -1
