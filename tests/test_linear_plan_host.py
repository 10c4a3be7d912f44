"""Which of the int8 linear layer's kernels runs for which sizes, without a GPU."""
import pytest

from linear_cases import LONG, SHORT


@pytest.fixture(scope="module")
def capi():
    from conv2d_batchnorm_silu_gb300 import _build
    _build.build()
    from conv2d_batchnorm_silu_gb300 import capi
    return capi


@pytest.mark.parametrize("case", SHORT + LONG, ids=str)
def test_the_kernel_of_each_case(capi, case):
    plan = capi.linear_int8_plan(*case[5])
    assert tuple(plan[name] for name in ("kernel", "turned", "tile_rows", "tile_channels", "align")) == case[:5]
    m, n, k, _ = case[5]
    assert plan["tiles"] >= -(-m // plan["tile_rows"]) * -(-n // plan["tile_channels"])
    if case in LONG:
        assert plan["tiles"] > 3 * plan["workers"]


def test_each_form_has_a_case():
    assert {case[:5] for case in LONG} <= {case[:5] for case in SHORT}
    # Tiles of 256 with rows off 16-byte boundaries are not chosen for many tiles: both widened before are faster.
    assert {case[:5] for case in SHORT} - {case[:5] for case in LONG} == {
        ("few", 0, 1, 32, 16), ("few", 0, 2, 8, 1), ("few", 0, 4, 4, 16), ("few", 0, 8, 16, 1), ("tile", 0, 32, 64, 16),
        ("tile", 0, 32, 64, 1), ("stream", 0, 256, 128, 1), ("stream", 0, 256, 128, 4), ("stream", 1, 128, 256, 1),
        ("stream", 1, 128, 256, 4)}


def test_refusals_and_empty_layers(capi):
    for bad in ((-1, 8, 8, 16, 152), (8, (1 << 22) + 1, 8, 16, 152), (8, 8, 131072, 16, 152), (8, 8, 8, 8, 152),
                (8, 8, 8, 0, 152), (8, 8, 8, 16, 0)):
        with pytest.raises(capi.CbsError) as e:
            capi.linear_int8_plan(*bad)
        assert e.value.status == capi.CBS_ERR_INVALID_ARG
    assert capi.raw_status("conv_bn_silu_linear_int8_plan", 8, 8, 8, 16, 152, None) == capi.CBS_ERR_INVALID_ARG
    for m, n in ((0, 8), (8, 0)):
        assert capi.linear_int8_plan(m, n, 8)["tiles"] == 0
    assert capi.linear_int8_plan(300, 300, 0)["kernel"] in ("tile", "gemm")  # the streamed kernels have no K of 0
