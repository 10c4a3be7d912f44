"""The shared projection's weights as AdaptedProjection and TokenBlock keep them."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
def test_weights_are_within_half_a_step_of_their_rows_largest(dtype):
    """An integer is off by half a step and the roundings of its product with 127 / most; a step is most / 127."""
    from conv2d_batchnorm_silu_gb300.token_block import AdaptedProjection
    w = (torch.randn(96, 130, generator=torch.Generator().manual_seed(1)) / 11).to(dtype).cuda()
    block = AdaptedProjection(torch.ones(130, device="cuda"), w, None, torch.zeros(1, 4, 130, device="cuda"),
                              torch.zeros(1, 96, 4, device="cuda"))
    most = w.double().abs().amax(1, keepdim=True)
    assert (block.w_scale.double()[:, None] * 127 / most - 1).abs().max() <= 2.0 ** -22
    off = (block.w.double() * block.w_scale.double()[:, None] - w.double()).abs()
    assert (off <= most / 127 * (0.5 + 127 * 4 * 2.0 ** -24)).all() and off.max() > 0
