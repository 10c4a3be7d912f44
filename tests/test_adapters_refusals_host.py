"""Memory that the adapters' gradients may not share, without a GPU: dx is written before the weights' gradients read dy
and x, so that a gradient in place of either would spoil them."""
import pytest

P, Q = 1 << 20, 1 << 21  # stand-ins for device pointers: refused calls never touch them


@pytest.mark.parametrize("m", [1, 4, 2000])
def test_dx_in_place_of_what_is_read_again(m):
    from conv2d_batchnorm_silu_gb300 import _build
    _build.build()
    from conv2d_batchnorm_silu_gb300 import capi

    def status(dy=P, x=P, dx=Q, base=None):
        return capi.raw_status("conv_bn_silu_linear_adapters_backward", dy, 16, x, 16, P, P, P, None, P, base, 16, dx, 16, Q, Q, m, 16,
                               16, 8, 2, 1, Q, 1 << 30, None)

    assert status(dx=P) == status(dy=Q) == status(x=Q) == status(dy=Q, base=Q) == capi.CBS_ERR_INVALID_ARG
