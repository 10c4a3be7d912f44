"""The int8 linear layer in every form of its kernels, and with several tiles for each worker, against the product in 64
bits.  Which kernel runs is asserted.  The bounds follow the arithmetic, as the layer's other tests derive them."""
import pytest
import torch

from linear_cases import LONG, SHORT

pytestmark = pytest.mark.gpu

TYPES = {torch.float32: (2.0 ** -24, 2.0 ** -149), torch.bfloat16: (2.0 ** -8, 2.0 ** -133), torch.float16: (2.0 ** -11, 2.0 ** -24)}
E32 = 2.0 ** -24


@pytest.fixture(scope="module")
def capi():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from conv2d_batchnorm_silu_gb300 import capi
    return capi


def generator(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def ints(seed, rows, k, align):
    """[rows][k] whose rows start at multiples of align and of no more."""
    pad = {16: 16, 4: 4, 1: 1}[align]
    store = torch.randint(-128, 128, (rows, k + pad), generator=generator(seed), dtype=torch.int8, device="cuda")
    return store[:, pad:]


@pytest.mark.parametrize("case", SHORT + LONG, ids=str)
def test_against_64_bits(capi, case):
    m, n, k, align = case[5]
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    plan = capi.linear_int8_plan(m, n, k, align, sms)
    assert tuple(plan[name] for name in ("kernel", "turned", "tile_rows", "tile_channels", "align")) == case[:5]
    a, w = ints(1, m, k, align), ints(2, n, k, align)
    a_scale = (torch.rand(m, generator=generator(3), device="cuda") + 0.5) / 64
    w_scale = (torch.rand(n, generator=generator(4), device="cuda") + 0.5) / (64 * k ** 0.5)
    bias = torch.randn(n, generator=generator(5), device="cuda")
    res32 = torch.randn(m, n, generator=generator(6), device="cuda")
    scales = a_scale.double()[:, None] * w_scale.double()
    wt = w.double().t()
    z = (a.double() @ wt) * scales + bias.double()
    total = a.double().abs() @ wt.abs()
    # sums below 2^24 are exact; beyond, each of the k/16 additions of a tensor-core sum (or the one rounding of an
    # integer sum) errs by up to 2^-23 of the largest partial sum
    zerr = scales * torch.where(total < 2.0 ** 24, 0.0, (k / 16 + 1) * 2.0 ** -23 * total) + 4 * E32 * (z.abs() + scales * total)
    silu = z * torch.sigmoid(z)
    for out, (unit, least) in TYPES.items():
        res = res32.to(out)
        for activation, residual in (("identity", None), ("silu", res)):
            want, tol = (z, 1.1 * zerr) if activation == "identity" else (silu, 1.1 * zerr + silu.abs() * (6 + 1.2 * z.abs())
                                                                          * 2 * E32 + 1e-36)
            if residual is not None:
                want = want + residual.double()
            tol = tol + 2 * E32 * want.abs() + unit * 1.001 * want.abs() + least
            y = capi.linear_int8(a, w, a_scale, w_scale, bias, activation, residual, out)
            assert ((y.double() - want).abs() <= tol).all(), (out, activation)
    # y off 16-byte boundaries, in place of its residual, what stands beside it untouched
    store = torch.full((m, n + 3), 7.0, dtype=torch.float16, device="cuda")
    inside = store[:, 1:n + 1]
    inside.copy_(res)
    assert torch.equal(capi.linear_int8(a, w, a_scale, w_scale, bias, "silu", inside, torch.float16, y=inside), y)
    assert (store[:, 0] == 7).all() and (store[:, n + 1:] == 7).all()
    capi.check()
