"""Layer norm, its gradient and the quantisations at numbers of rows that take every block round its ring of rows
more than twice, with a remainder, for each number of threads that share a row; each row against its definition in
64 bits.  The bounds follow the arithmetic: unit roundoffs, and the additions a thread makes in a row."""
import pytest
import torch

pytestmark = pytest.mark.gpu

TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
ROUND = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8, "f16": 2.0 ** -11}
LEAST = {"f32": 2.0 ** -149, "bf16": 2.0 ** -133, "f16": 2.0 ** -24}
E32 = 2.0 ** -24
EPS = 1e-5


@pytest.fixture(scope="module")
def capi():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from conv2d_batchnorm_silu_gb300 import capi
    return capi


def rows_of(seed, rows, c, dtype, pad, shift=0.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn(rows, c + pad, generator=g, device="cuda")
    x = x * (0.25 + 2 * torch.rand(rows, 1, generator=g, device="cuda")) + shift
    return x.to(TYPES[dtype])[:, :c]


def vector(seed, c, low=None):
    g = torch.Generator(device="cuda").manual_seed(seed)
    v = torch.randn(c, generator=g, device="cuda")
    return v if low is None else low + torch.rand(c, generator=g, device="cuda")


def summing(c):
    """Relative error of a row sum: at most c/32 + 32 additions after one another."""
    return (c / 32 + 32) * E32


def normalised(x, gamma, beta):
    """(y, mean, rstd, bound of what fp32 may be off) in 64 bits."""
    c, x, gamma, beta = x.shape[1], x.double(), gamma.double(), beta.double()
    mean = x.sum(1, keepdim=True) / c
    rstd = 1.0 / torch.sqrt(((x - mean) ** 2).sum(1, keepdim=True) / c + EPS)
    h = (x - mean) * rstd
    y = h * gamma + beta
    s = summing(c)
    off = s * x.abs().mean(1, keepdim=True)  # of the mean
    g, h = gamma.abs(), h.abs()
    bound = (g * rstd * off + g * h * (2 * s + 8 * E32) + g * rstd * x.abs() * 2 * E32 + 4 * E32 * (y.abs() + g * h))
    return y, mean, rstd, off, bound


# (type, elements a slice leaves over, channels for t threads a row, ring slots).  Threads hold 32 elements of 16-bit
# rows on 16-byte boundaries, and 16 of f32 rows; of 16-bit rows off them 16, and 32 beyond 2048 channels.
FORMS = {
    "bf16": ("bf16", 0, lambda t: 24 * t, 3),
    "f32": ("f32", 0, lambda t: 12 * t, 3),
    "f32 anywhere": ("f32", 1, lambda t: 12 * t + 1, 3),
    "f16 anywhere": ("f16", 1, lambda t: (12 if t <= 128 else 20) * t + 1, 4),
    "f16 anywhere, 32": ("f16", 1, lambda t: 20 * t + 1, 4),
}
CASES = [(t, form) for form in list(FORMS)[:4] for t in (4, 8, 16, 32, 64, 128, 256, 512)] + [(128, "f16 anywhere, 32")]


def rows_for(threads, rounds):
    # 512 threads an SM, in blocks that hold one row or several.
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    return rounds * sms * 512 // threads + 3


@pytest.mark.parametrize("threads,form", CASES)
def test_norm_and_quantisation(capi, threads, form):
    dtype, pad, width, slots = FORMS[form]
    c, rows = width(threads), rows_for(threads, 2 * slots + 1)
    if form == "f16 anywhere" and threads == 512:
        c = 10001
    x, gamma, beta = rows_of(threads, rows, c, dtype, pad, shift=0.5), vector(1, c, 0.5), vector(2, c)
    want, mean, rstd, off, bound = normalised(x, gamma, beta)
    y, stats = capi.layer_norm(x, gamma, beta, EPS, return_stats=True)
    assert ((y.double() - want).abs() <= bound + ROUND[dtype] * 1.001 * want.abs() + LEAST[dtype]).all()
    assert ((stats[0].double() - mean[:, 0]).abs() <= off[:, 0] + 1e-30).all()
    assert ((stats[1].double() / rstd[:, 0] - 1).abs() <= summing(c) + 4 * E32 + (off * rstd)[:, 0] ** 2).all()
    del y
    q, scale = capi.layer_norm_quantize(x, gamma, beta, EPS)
    scale, most = scale.double()[:, None], want.abs().amax(1, keepdim=True)
    assert ((scale * 127 - most).abs() <= bound.amax(1, keepdim=True) + 4 * E32 * most).all()
    # half a step, the value's own error and the scale's at up to 127 steps
    tol = scale * (0.5 + 127 * 8 * E32) + bound + bound.amax(1, keepdim=True)
    assert ((q.double() * scale - want).abs() <= tol).all()
    del want, bound, tol
    # The quantisation alone, in its definition's own fp32 arithmetic.
    q, scale = capi.quantize_rows(x)
    v = x.float()
    most, of_127 = v.abs().amax(1, keepdim=True), torch.full((rows, 1), 127.0, device="cuda")
    assert torch.equal(scale[:, None], most / of_127)
    assert torch.equal(q, torch.round(v * (of_127 / most)).to(torch.int8))


# The same for the gradient, which holds 16 elements a thread and has at least eight threads a row.
GRAD_FORMS = {"bf16": ("bf16", 0, 3), "f32": ("f32", 0, 3), "f32 anywhere": ("f32", 1, 3), "f16 anywhere": ("f16", 1, 4)}


@pytest.mark.parametrize("form", list(GRAD_FORMS))
@pytest.mark.parametrize("threads", [8, 16, 32, 64, 128, 256, 512])
def test_gradient(capi, threads, form):
    dtype, pad, slots = GRAD_FORMS[form]
    c, rows = 12 * threads + pad, rows_for(threads, 2 * slots + 1)
    x, dy, gamma = rows_of(threads, rows, c, dtype, pad, shift=0.5), rows_of(7, rows, c, dtype, 0), vector(1, c, 0.5)
    _, stats = capi.layer_norm(x, None, None, EPS, return_stats=True)
    dx, dgamma, dbeta = capi.layer_norm_backward(dy, x, gamma, stats)
    # The formula in 64 bits, from the statistics the call was given.
    x, dy, g = x.double(), dy.double(), dy.double() * gamma.double()
    mean, rstd = stats[0].double()[:, None], stats[1].double()[:, None]
    h = (x - mean) * rstd
    want = rstd * (g - g.mean(1, keepdim=True) - h * (g * h).mean(1, keepdim=True))
    eh = 4 * E32 * (x.abs() + mean.abs()) * rstd  # of h
    s, ag, ah = summing(c), g.abs(), h.abs()
    s1, s2 = ag.mean(1, keepdim=True), (ag * ah).mean(1, keepdim=True)
    es2 = (s + 8 * E32) * s2 + (ag * eh).mean(1, keepdim=True)
    bound = rstd * (8 * E32 * (ag + s1 + ah * s2) + s * s1 + ah * es2 + eh * s2)
    assert ((dx.double() - want).abs() <= bound + ROUND[dtype] * 1.001 * want.abs() + LEAST[dtype]).all()
    # down a column: a thread's rounds, the rows of a block side by side, and the blocks' partial sums
    deep = (2 * slots + 2 + 32 + 32 + 16 + 8) * E32
    assert ((dgamma.double() - (dy * h).sum(0)).abs() <= (deep * dy.abs() * ah + dy.abs() * eh).sum(0) + 1e-37).all()
    assert ((dbeta.double() - dy.sum(0)).abs() <= deep * dy.abs().sum(0) + 1e-37).all()


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_long_rows_off_alignment(capi, dtype):
    # 8193 to 9500 channels off alignment: 512 threads a row up to 1000 rows, and beyond them one row a block at a time
    for rows in (1000, 1001):
        c = 9001
        x, gamma, beta = rows_of(rows, rows, c, dtype, 1, shift=0.5), vector(1, c, 0.5), vector(2, c)
        want, mean, rstd, off, bound = normalised(x, gamma, beta)
        y = capi.layer_norm(x, gamma, beta, EPS)
        assert ((y.double() - want).abs() <= bound + ROUND[dtype] * 1.001 * want.abs() + LEAST[dtype]).all()
