"""Root-mean-square norm, its int8 output and its gradient on the GPU against the 64-bit oracle.
Every tolerance is a bound from the arithmetic: unit roundoffs of the output's type and of fp32,
and the number of additions a thread makes in a row."""
import numpy as np
import pytest
import torch

from oracle import token_ops as ref

pytestmark = pytest.mark.gpu

TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
ROUND = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8, "f16": 2.0 ** -11}
LEAST = {"f32": 2.0 ** -149, "bf16": 2.0 ** -133, "f16": 2.0 ** -24}
E32 = 2.0 ** -24
EPS = 1e-6


@pytest.fixture(scope="module")
def capi():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from conv2d_batchnorm_silu_gb300 import capi
    return capi


def host(t):
    return t.detach().double().cpu().numpy()


def rows_of(seed, rows, c, dtype, pad=0, offset=0, size=1.0):
    """[rows][c] on the GPU, a slice of a buffer `pad` elements wider that starts at `offset`."""
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(rows, c + pad + offset, generator=g) * (0.25 + 2 * torch.rand(rows, 1, generator=g)) * size
    return x.to(TYPES[dtype]).cuda()[:, offset:offset + c]


def vector(seed, c):
    return (0.5 + torch.rand(c, generator=torch.Generator().manual_seed(seed))).cuda()


def summing(c):
    """Relative error of a row sum of like signs: at most c/32 + 32 additions after one another."""
    return (c / 32 + 32) * E32


def check_norm(x, gamma, y, dtype, rstd=None, total=None):
    at = host(x if total is None else total)
    want, want_rstd = ref.rms_norm(at, None if gamma is None else host(gamma), EPS)
    off = summing(at.shape[1]) / 2 + 4 * E32  # of rstd: half the mean square's, the root's and a product's
    if rstd is not None:
        assert (np.abs(host(rstd) / want_rstd - 1) <= off).all()
    if y is not None:
        assert (np.abs(host(y) - want) <= np.abs(want) * (off + 4 * E32 + ROUND[dtype] * 1.001) + LEAST[dtype]).all()
    return want, off


WIDTHS = [1, 2, 7, 8, 16, 33, 64, 127, 128, 136, 256, 257, 512, 520, 777, 1000, 1024, 1025, 2048, 2049, 4096, 4099, 4104,
          8192, 8193, 8200, 16384, 16392, 16385, 20001]


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("c", WIDTHS)
def test_norm_and_residual(capi, c, dtype):
    for rows in (1, 5, 37):
        x, residual, gamma = rows_of(c, rows, c, dtype), rows_of(c + 1, rows, c, dtype, size=3.0), vector(1, c)
        y, rstd = capi.rms_norm(x, gamma, EPS, return_rstd=True)
        assert y.dtype == x.dtype and y.shape == x.shape and rstd.shape == (rows,)
        check_norm(x, gamma, y, dtype, rstd)
        y, total, rstd = capi.rms_norm(x, gamma, EPS, residual=residual, return_rstd=True)
        assert torch.equal(total, (x.float() + residual.float()).to(x.dtype))
        check_norm(x, gamma, y, dtype, rstd, total)


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("c", [1, 8, 24, 130, 256, 1023, 1536, 4096, 4097, 8192, 9001, 16384, 20000])
def test_quantised(capi, c, dtype):
    for rows in (1, 9, 41):
        x, residual, gamma = rows_of(c, rows, c, dtype), rows_of(c + 1, rows, c, dtype), vector(2, c)
        q, scale, total, y, rstd = capi.rms_norm_quantize(x, gamma, EPS, residual=residual, return_y=True, return_rstd=True)
        want, off = check_norm(x, gamma, y, dtype, rstd, total)
        assert q.dtype == torch.int8 and scale.shape == (rows,)
        assert torch.equal(total, (x.float() + residual.float()).to(x.dtype))
        scales = ref.row_scales(want)
        assert (np.abs(host(scale) / scales - 1) <= off + 6 * E32).all()
        # half a step, and the value's and scale's own errors, of up to 127 steps
        assert (np.abs(host(q) * scales[:, None] - want) <= scales[:, None] * (0.5 + 127 * (2 * off + 12 * E32))).all()
        q2, scale2 = capi.rms_norm_quantize(total, gamma, EPS)
        assert torch.equal(q, q2) and torch.equal(scale, scale2)


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("adds", [False, True])
@pytest.mark.parametrize("c", [1, 2, 8, 15, 16, 64, 129, 256, 257, 520, 777, 1024, 1025, 2048, 3001, 4096, 4104, 4099, 8192,
                               8193, 8200, 12001])
def test_gradient(capi, c, dtype, adds):
    for rows in (1, 6, 700):
        x, dy, gamma = rows_of(c, rows, c, dtype), rows_of(c + 1, rows, c, dtype, size=0.1), vector(3, c)
        residual = rows_of(c + 2, rows, c, dtype, size=0.1) if adds else None
        _, rstd = capi.rms_norm(x, gamma, EPS, return_rstd=True)
        dx, dgamma = capi.rms_norm_backward(dy, x, gamma, rstd, residual=residual)
        check_gradient(dy, x, gamma, rstd, residual, dx, dgamma, dtype)


def check_gradient(dy, x, gamma, rstd, residual, dx, dgamma, dtype):
    rows, c = x.shape
    want, want_g = ref.rms_norm_backward(host(dy), host(x), host(gamma), host(rstd), None if residual is None else host(residual))
    r, gm = host(rstd)[:, None], host(gamma)
    h, g = np.abs(host(x)) * r, np.abs(host(dy)) * gm
    mean = (g * h).mean(axis=1, keepdims=True)
    bound = r * (h * mean * (summing(c) + 6 * E32) + 4 * E32 * (g + h * mean)) + (ROUND[dtype] * 1.001 + 2 * E32) * np.abs(want)
    if residual is not None:
        bound = bound + 2 * E32 * np.abs(host(residual))
    assert dx.dtype == x.dtype and (np.abs(host(dx) - want) <= bound + LEAST[dtype]).all()
    # a column's sum: rows of a block one after another, then the blocks' (10 loads and a tree)
    adds = min(rows, rows / 100 + 400) + 2
    assert (np.abs(host(dgamma) - want_g) <= adds * E32 * (np.abs(host(dy)) * h).sum(0) + 1e-30).all()


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("c,pad,offset", [(96, 5, 0), (256, 8, 8), (777, 23, 0), (1024, 3, 1), (4096, 1, 3), (9000, 7, 5)])
def test_slices_at_any_alignment(capi, c, pad, offset, dtype):
    x, residual = rows_of(1, 45, c, dtype, pad, offset), rows_of(2, 45, c, dtype, pad, offset + 1)
    gamma = vector(4, c + 1)[1:]
    out = [torch.full((45, c + 9), 7.0, dtype=TYPES[dtype], device="cuda") for _ in range(3)]
    y, total, dx = (t[:, 3:3 + c] for t in out)
    _, _, rstd = capi.rms_norm(x, gamma, EPS, residual=residual, return_rstd=True, y=y, total=total)
    check_norm(x, gamma, y, dtype, rstd, total)
    dy = rows_of(5, 45, c, dtype, pad, offset)
    dx, dgamma = capi.rms_norm_backward(dy, total, gamma, rstd, residual=residual, dx=dx)
    check_gradient(dy, total, gamma, rstd, residual, dx, dgamma, dtype)
    for t in out:  # nothing beside the outputs is written
        assert (t[:, :3] == 7).all() and (t[:, 3 + c:] == 7).all()
    qs = torch.full((45, c + 9), 7, dtype=torch.int8, device="cuda")
    q, scale, total2 = capi.rms_norm_quantize(x, gamma, EPS, residual=residual, q=qs[:, 5:5 + c])
    dense, dense_scale = capi.rms_norm_quantize(total2.contiguous(), gamma.clone(), EPS)
    assert torch.equal(total2, total) and (qs[:, :5] == 7).all() and (qs[:, 5 + c:] == 7).all()
    # another kernel may order a row's sum otherwise: the scales agree to its error, values to a step
    assert (host(scale) / host(dense_scale) - 1).__abs__().max() <= 2 * summing(c) + 16 * E32
    assert (q.int() - dense.int()).abs().max() <= 1


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("c", [96, 1001, 4096, 20001])
def test_in_place(capi, c, dtype):
    x, residual, gamma = rows_of(1, 333, c, dtype), rows_of(2, 333, c, dtype), vector(5, c)
    y, total = capi.rms_norm(x, gamma, EPS, residual=residual)
    stream = residual.clone()
    y2, total2 = capi.rms_norm(x, gamma, EPS, residual=stream, total=stream)
    assert total2.data_ptr() == stream.data_ptr() and torch.equal(stream, total) and torch.equal(y, y2)
    dy = rows_of(3, 333, c, dtype)
    _, rstd = capi.rms_norm(total, gamma, EPS, return_rstd=True)
    dx, dgamma = capi.rms_norm_backward(dy, total, gamma, rstd, residual=residual)
    into = residual.clone()
    dx2, dgamma2 = capi.rms_norm_backward(dy, total, gamma, rstd, residual=into, dx=into)
    assert torch.equal(dx, into) and torch.equal(dx, dx2) and torch.equal(dgamma, dgamma2)


def test_gradient_by_differences(capi):
    """Central differences of the forward call itself, in fp32: values of order 1 with errors of some 2^-22 over a
    step of 2^-6 leave 2^-15 and the step's square."""
    x, dy, gamma = rows_of(1, 3, 40, "f32"), rows_of(2, 3, 40, "f32"), vector(6, 40)
    _, rstd = capi.rms_norm(x, gamma, EPS, return_rstd=True)
    dx, dgamma = capi.rms_norm_backward(dy, x, gamma, rstd)
    step = 2.0 ** -6

    def loss(x, gamma):
        return float((capi.rms_norm(x, gamma, EPS).double() * dy.double()).sum())

    for r, c in ((0, 0), (1, 17), (2, 39)):
        e = torch.zeros_like(x)
        e[r, c] = step
        assert abs((loss(x + e, gamma) - loss(x - e, gamma)) / (2 * step) - float(dx[r, c])) < 4e-3
    for c in (0, 21, 39):
        e = torch.zeros_like(gamma)
        e[c] = step
        assert abs((loss(x, gamma + e) - loss(x, gamma - e)) / (2 * step) - float(dgamma[c])) < 4e-3


def test_empty_constant_and_special_rows(capi):
    gamma = vector(7, 64)
    x = torch.zeros(5, 64, device="cuda")
    x[1], x[2, 3], x[3, 5] = 2.0, float("nan"), float("inf")
    x[4] = 1e30  # whose squares leave fp32
    y, rstd = capi.rms_norm(x, gamma, EPS, return_rstd=True)
    assert (y[0] == 0).all() and (y[1] / gamma - 1).abs().max() < 1e-6
    assert y[2].isnan().all() and y[3, 5].isnan() and (y[4] == 0).all() and rstd[4] == 0
    q, scale = capi.rms_norm_quantize(x, gamma, EPS)
    assert (q[0] == 0).all() and (q[2:4] == 0).all() and not scale[2:4].isfinite().any() and scale[:2].isfinite().all()
    none = torch.empty(0, 64, device="cuda")
    y, total, rstd = capi.rms_norm(none, gamma, EPS, residual=none, return_rstd=True)
    assert y.shape == total.shape == (0, 64) and rstd.shape == (0,)
    dx, dgamma = capi.rms_norm_backward(none, none, gamma, rstd)
    assert dx.shape == (0, 64) and (dgamma == 0).all()


def test_shapes_streams_and_graphs(capi):
    x, residual, gamma = rows_of(1, 24, 256, "bf16").view(2, 3, 4, 256), rows_of(2, 24, 256, "bf16").view(2, 3, 4, 256), vector(8, 256)
    q, scale, total, rstd = capi.rms_norm_quantize(x, gamma, EPS, residual=residual, return_rstd=True)
    assert q.shape == x.shape and scale.shape == rstd.shape == (2, 3, 4)
    # one row for all, as residual
    one = residual[0, 0, :1].expand(24, 256)
    y, total1 = capi.rms_norm(x.view(24, 256), gamma, EPS, residual=one)
    assert torch.equal(total1, (x.view(24, 256).float() + one.float()).bfloat16())
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    other = capi.rms_norm_quantize(x, gamma, EPS, residual=residual, stream=side)
    side.synchronize()
    assert torch.equal(other[0], q) and torch.equal(other[1], scale)
    graph, dy = torch.cuda.CUDAGraph(), residual
    with torch.cuda.graph(graph):
        y, total2, rstd2 = capi.rms_norm(x, gamma, EPS, residual=residual, return_rstd=True)
        dx, dgamma = capi.rms_norm_backward(dy, total2, gamma, rstd2)
    x.copy_(x.flip(0))
    graph.replay()
    want, _, want_rstd = capi.rms_norm(x, gamma, EPS, residual=residual, return_rstd=True)
    want_dx, want_dg = capi.rms_norm_backward(dy, total2, gamma, want_rstd)
    assert torch.equal(y, want) and torch.equal(dx, want_dx) and torch.equal(dgamma, want_dg)


def test_refusals(capi):
    x, gamma = torch.zeros(4, 32, device="cuda"), torch.ones(32, device="cuda")
    for call in (lambda: capi.rms_norm(x, gamma, residual=x.half()), lambda: capi.rms_norm(x, gamma.half()),
                 lambda: capi.rms_norm(x.double(), gamma), lambda: capi.rms_norm_backward(x, x, gamma, None)):
        with pytest.raises(TypeError):
            call()
    for call in (lambda: capi.rms_norm(x, gamma, residual=x[:3]), lambda: capi.rms_norm(x, gamma, total=x.clone()),
                 lambda: capi.rms_norm(x.cpu(), gamma), lambda: capi.rms_norm(x, gamma[:31]),
                 lambda: capi.rms_norm(x.t(), gamma[:4]), lambda: capi.rms_norm_backward(x[:2], x, gamma, gamma[:4]),
                 lambda: capi.rms_norm(x, gamma, -1.0), lambda: capi.rms_norm_backward(x, x, gamma, gamma[:3])):
        with pytest.raises((ValueError, RuntimeError)):
            call()
