"""Values of the token-wise operators that their definitions give exactly, and SiLU in fp32 to the last places."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
E32 = 2.0 ** -24


@pytest.fixture(scope="module")
def capi():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from conv2d_batchnorm_silu_gb300 import capi
    return capi


def vector(seed, c):
    return torch.randn(c, generator=torch.Generator().manual_seed(seed)).cuda()


def inexact_reciprocal(low, high, step=1):
    """The first width above low, a multiple of step, whose reciprocal is rounded so that 3 c (1/c) is not 3 in fp32."""
    f = np.float32
    return next(c for c in range(-(-low // step) * step, high, step) if f(f(3 * c) * f(f(1) / f(c))) != f(3))


# Aligned and other widths for each number of threads that share a row.
WIDTHS = sorted({inexact_reciprocal(low, 9 * low, step) for low in (7, 33, 65, 129, 257, 513, 1025, 2049, 4097, 8193)
                 for step in (1, 8)})


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("pad", [0, 1])
@pytest.mark.parametrize("c", WIDTHS)
def test_layer_norm_of_one_value(capi, c, pad, dtype):
    # Sums of c equal whole numbers are exact (below 2^24), so the mean is the value and what is left is beta.
    for value in (3.0, -7.0, 1000.0):
        if abs(value) * c >= 2 ** 24:
            continue
        x = torch.full((5, c + pad), value, dtype=TYPES[dtype], device="cuda")[:, :c]
        gamma, beta = vector(1, c), vector(2, c)
        y, stats = capi.layer_norm(x, gamma, beta, 1e-5, return_stats=True)
        assert torch.equal(stats[0], torch.full((5,), value, device="cuda"))
        assert torch.equal(y, beta.to(x.dtype).expand(5, c))
        q, scale = capi.layer_norm_quantize(x, gamma, beta, 1e-5)
        wq, ws = capi.quantize_rows(beta[None])
        assert torch.equal(q, wq.expand(5, c)) and torch.equal(scale, ws.expand(5))
        assert capi.layer_norm(x, gamma, beta, 0.0).isnan().all()


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("pad", [0, 1])
@pytest.mark.parametrize("c", WIDTHS)
def test_layer_norm_gradient_of_one_value(capi, c, pad, dtype):
    # h is 1, -1, 1, ... (0 in an odd last place): its sums with a constant gradient vanish, and the mean of that
    # gradient is its one value, so nothing is left for the input.
    rows = 5
    store = torch.zeros(rows, c + pad, dtype=TYPES[dtype], device="cuda")
    x = store[:, :c]
    x[:, : c // 2 * 2] = torch.tensor([1.0, -1.0], dtype=x.dtype, device="cuda").repeat(c // 2)
    dy = torch.full((rows, c + pad), 3.0, dtype=x.dtype, device="cuda")[:, :c]
    stats = torch.stack((torch.zeros(rows), torch.ones(rows))).cuda()
    dx, dgamma, dbeta = capi.layer_norm_backward(dy, x, None, stats)
    assert not dx.any()
    assert torch.equal(dgamma, 3.0 * rows * x[0].float()) and torch.equal(dbeta, torch.full_like(dbeta, 3.0 * rows))


# Few rows, the one-launch tile, sums joined after streamed weights at each row tile, streamed rows, and the widened
# product in each of its tiles.
SIZES = [(3, 300, 16), (8, 300, 1000), (24, 300, 64), (20, 300, 4096), (40, 712, 2048), (100, 712, 2048), (300, 300, 4096),
         (700, 1300, 400), (1500, 1300, 400), (2300, 2000, 1040), (1500, 9, 4096), (9000, 100, 2048), (100, 712, 2051)]


@pytest.mark.parametrize("m,n,k", SIZES)
def test_linear_silu_in_fp32(capi, m, n, k):
    # One product in each sum and scales of powers of two: z is exact, from -112 to 112 in steps of 1/8.
    a, w = torch.zeros(m, k, dtype=torch.int8, device="cuda"), torch.zeros(n, k, dtype=torch.int8, device="cuda")
    where = k // 2
    a[:, where] = (torch.arange(m, device="cuda") * 29 % 257 - 128).to(torch.int8)
    w[:, where] = (torch.arange(n, device="cuda") % 7 + 1).to(torch.int8)
    a_scale, w_scale = torch.full((m,), 0.25, device="cuda"), torch.full((n,), 0.5, device="cuda")
    z = a[:, where].double()[:, None] * w[:, where].double() / 8
    want = z * torch.sigmoid(z)
    y = capi.linear_int8(a, w, a_scale, w_scale, activation="silu", out_dtype=torch.float32).double()
    # The exponential errs by 2 units in the last place, the sum, the quotient (or a reciprocal of two sums'
    # product and two products) by half a unit each: 5 + 5 roundings.  Beyond -88.7 the exponential leaves the range and
    # the result is -0, at most 88.8 * 2^-128 off.
    tol = 10 * E32 * want.abs() + torch.where(z < -88.7, 2.7e-37, 0.0)
    assert ((y - want).abs() <= tol).all(), float(((y - want).abs() / want.abs().clamp(min=1e-37)).max())
    # The residual is added to that, and the 16-bit types see the same value but for what their rounding hides.
    res = torch.full((m, n), 1.0, device="cuda")
    y = capi.linear_int8(a, w, a_scale, w_scale, None, "silu", res, torch.float32).double()
    assert ((y - want - 1.0).abs() <= tol + E32 * 1.001 * (want + 1.0).abs()).all()
    for out, unit in ((torch.bfloat16, 2.0 ** -8), (torch.float16, 2.0 ** -11)):
        y = capi.linear_int8(a, w, a_scale, w_scale, activation="silu", out_dtype=out).double()
        tiny = 1e-36 if out == torch.bfloat16 else 2.0 ** -24
        assert ((y - want).abs() <= unit * 1.01 * want.abs() + tiny).all()
    capi.check()
