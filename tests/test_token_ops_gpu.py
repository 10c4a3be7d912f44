"""Layer norm, its gradient, quantised rows and the int8 linear layer on the GPU against the 64-bit
oracle.  Every tolerance is a bound derived from the arithmetic: unit roundoffs of the output type
and of fp32, and the number of additions a thread makes in a row."""
import numpy as np
import pytest
import torch

from oracle import token_ops as ref

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


def host(t):
    return t.detach().double().cpu().numpy()


def rows_of(seed, rows, c, dtype, pad=0, offset=0, shift=0.0):
    """[rows][c] on the GPU, a slice of a buffer `pad` elements wider that starts at `offset`."""
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(rows, c + pad + offset, generator=g) * (0.25 + 2 * torch.rand(rows, 1, generator=g)) + shift
    return x.to(TYPES[dtype]).cuda()[:, offset:offset + c]


def vector(seed, c, low=None):
    g = torch.Generator().manual_seed(seed)
    v = torch.randn(c, generator=g) if low is None else low + torch.rand(c, generator=g)
    return v.cuda()


def summing(c):
    """Relative error of a row sum: at most c/32 + 32 additions after one another."""
    return (c / 32 + 32) * E32


def norm_bound(x, gamma, y, mean, rstd, dtype):
    x, c = host(x), x.shape[1]
    s = summing(c)
    h = np.abs(x - mean[:, None]) * rstd[:, None]
    off = s * np.abs(x).mean(1)  # of the mean
    g = 1.0 if gamma is None else np.abs(host(gamma))
    return (g * (rstd * off)[:, None] + g * h * (2 * s + 8 * E32) + g * rstd[:, None] * np.abs(x) * 2 * E32
            + 4 * E32 * (np.abs(y) + g * h) + ROUND[dtype] * np.abs(y) * 1.001 + LEAST[dtype])


WIDTHS = [1, 2, 7, 8, 15, 16, 24, 32, 33, 40, 64, 96, 127, 128, 200, 256, 257, 512, 520, 777, 1000, 1024, 1025, 1032,
          1536, 2048, 2049, 4096, 4099, 4104, 8192, 8193, 8200, 12296, 16384, 16392, 16385, 20001]


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("c", WIDTHS)
def test_layer_norm(capi, c, dtype):
    for rows in (1, 5, 37):
        x = rows_of(c, rows, c, dtype, shift=1.5)
        gamma, beta = vector(1, c, 0.5), vector(2, c)
        y, stats = capi.layer_norm(x, gamma, beta, EPS, return_stats=True)
        want, mean, rstd = ref.layer_norm(host(x), host(gamma), host(beta), EPS)
        assert y.dtype == x.dtype and y.shape == x.shape and stats.shape == (2, rows)
        assert (np.abs(host(y) - want) <= norm_bound(x, gamma, want, mean, rstd, dtype)).all()
        s = summing(c)
        assert (np.abs(host(stats[0]) - mean) <= s * np.abs(host(x)).mean(1) + 1e-30).all()
        # relative error of rstd: half the variance's, which is 2s, and the mean's error squared
        off = s * np.abs(host(x)).mean(1) * rstd
        assert (np.abs(host(stats[1]) / rstd - 1) <= s + 4 * E32 + off * off).all()


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("pad,offset", [(3, 0), (8, 0), (8, 8), (5, 1), (16, 2)])
@pytest.mark.parametrize("c", [40, 777, 1024, 4096, 16400])
def test_layer_norm_of_slices_leaves_the_rest_alone(capi, c, pad, offset, dtype):
    rows = 19
    x = rows_of(3, rows, c, dtype, pad, offset)
    store = torch.full((rows, c + pad + offset), 7.0, dtype=TYPES[dtype], device="cuda")
    y = capi.layer_norm(x, None, None, EPS, y=store[:, offset:offset + c])
    want, mean, rstd = ref.layer_norm(host(x), None, None, EPS)
    assert (np.abs(host(y) - want) <= norm_bound(x, None, want, mean, rstd, dtype)).all()
    assert (store[:, :offset] == 7).all() and (store[:, offset + c:] == 7).all()


def test_layer_norm_far_from_zero(capi):
    # a spread of 1 around 4096: fp32 keeps 2^-12 of it, and the two-pass variance loses no more
    x = rows_of(5, 8, 1000, "f32", shift=4096.0)
    y, stats = capi.layer_norm(x, None, None, EPS, return_stats=True)
    want, mean, rstd = ref.layer_norm(host(x), None, None, EPS)
    assert (np.abs(host(y) - want) <= norm_bound(x, None, want, mean, rstd, "f32")).all()


def test_layer_norm_of_constant_rows_and_special_values(capi):
    x = torch.full((4, 300), 3.0, device="cuda")
    x[1, 7] = float("nan")
    x[2, 9] = float("inf")
    y = capi.layer_norm(x, None, vector(1, 300), EPS)
    assert torch.equal(y[0], vector(1, 300)) and torch.equal(y[3], y[0])
    assert y[1].isnan().all() and y[2].isnan().all()


def test_layer_norm_many_dimensions_empty_and_broadcast(capi):
    x = rows_of(1, 24, 64, "bf16").view(2, 3, 4, 64)
    y, stats = capi.layer_norm(x, return_stats=True)
    assert y.shape == x.shape and torch.equal(y.view(24, 64), capi.layer_norm(x.view(24, 64)))
    none, stats = capi.layer_norm(x[:0], return_stats=True)
    assert none.shape == (0, 3, 4, 64) and stats.shape == (2, 0)
    one = rows_of(2, 1, 64, "bf16")
    assert torch.equal(capi.layer_norm(one.expand(9, 64)), capi.layer_norm(one).expand(9, 64))
    vec = capi.layer_norm(one[0])
    assert vec.shape == (64,) and torch.equal(vec, capi.layer_norm(one)[0])


def grad_bounds(dy, x, gamma, mean, rstd, dtype):
    dy, x = np.abs(host(dy)), host(x)
    rows, c = x.shape
    h = np.abs(x - mean[:, None]) * rstd[:, None]
    eh = 4 * E32 * (np.abs(x) + np.abs(mean)[:, None]) * rstd[:, None]  # of h
    g = dy if gamma is None else dy * np.abs(host(gamma))
    s = summing(c)
    s1, s2 = g.mean(1)[:, None], (g * h).mean(1)[:, None]
    es2 = (s + 8 * E32) * s2 + (g * eh).mean(1)[:, None]
    dx = rstd[:, None] * (8 * E32 * (g + s1 + h * s2) + s * s1 + h * es2 + eh * s2)
    # down a column, whatever the split: fewer additions after one another than rows
    deep = (min(rows, rows / 64 + 700) + 8) * E32
    return dx, (deep * (dy * h) + dy * eh).sum(0) + 1e-37, deep * dy.sum(0) + 1e-37


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("c", WIDTHS)
def test_layer_norm_backward(capi, c, dtype):
    for rows in (1, 6, 61 if c > 3000 else 1500):
        x, dy = rows_of(c, rows, c, dtype, shift=0.5), rows_of(c + 1, rows, c, dtype)
        gamma = vector(1, c, 0.5) if c % 3 else None
        _, stats = capi.layer_norm(x, None, None, EPS, return_stats=True)
        dx, dgamma, dbeta = capi.layer_norm_backward(dy, x, gamma, stats)
        mean, rstd = host(stats)
        want = ref.layer_norm_backward(host(dy), host(x), None if gamma is None else host(gamma), mean, rstd)
        bx, bg, bb = grad_bounds(dy, x, gamma, mean, rstd, dtype)
        assert (np.abs(host(dx) - want[0]) <= bx + ROUND[dtype] * 1.001 * np.abs(want[0]) + LEAST[dtype]).all()
        assert (np.abs(host(dgamma) - want[1]) <= bg).all()
        assert (np.abs(host(dbeta) - want[2]) <= bb).all()


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("pad,offset", [(3, 0), (8, 8), (5, 1)])
@pytest.mark.parametrize("c", [40, 777, 1024, 4096])
def test_layer_norm_backward_of_slices(capi, c, pad, offset, dtype):
    rows = 203
    x, dy = rows_of(3, rows, c, dtype, pad, offset), rows_of(4, rows, c, dtype, 2 * pad, 0)
    gamma = vector(1, c, 0.5)
    _, stats = capi.layer_norm(x, None, None, EPS, return_stats=True)
    store = torch.full((rows, c + pad + offset), 7.0, dtype=TYPES[dtype], device="cuda")
    dx, dgamma, dbeta = capi.layer_norm_backward(dy, x, gamma, stats, dx=store[:, offset:offset + c])
    mean, rstd = host(stats)
    want = ref.layer_norm_backward(host(dy), host(x), host(gamma), mean, rstd)
    bx, bg, bb = grad_bounds(dy, x, gamma, mean, rstd, dtype)
    assert (np.abs(host(dx) - want[0]) <= bx + ROUND[dtype] * 1.001 * np.abs(want[0]) + LEAST[dtype]).all()
    assert (np.abs(host(dgamma) - want[1]) <= bg).all() and (np.abs(host(dbeta) - want[2]) <= bb).all()
    assert (store[:, :offset] == 7).all() and (store[:, offset + c:] == 7).all()


def test_layer_norm_backward_repeats_and_takes_no_rows(capi):
    x, dy = rows_of(1, 3001, 264, "bf16"), rows_of(2, 3001, 264, "bf16")
    _, stats = capi.layer_norm(x, None, None, EPS, return_stats=True)
    first = capi.layer_norm_backward(dy, x, None, stats)
    for _ in range(3):
        again = capi.layer_norm_backward(dy, x, None, stats)
        assert all(torch.equal(a, b) for a, b in zip(first, again))
    dx, dgamma, dbeta = capi.layer_norm_backward(dy[:0], x[:0], None, stats[:, :0].contiguous())
    assert dx.shape == (0, 264) and not dgamma.any() and not dbeta.any()


def test_layer_norm_gradient_by_differences(capi):
    # the GPU's own forward pass in fp32 against its gradient: <dy, (y(x + d) - y(x - d)) / 2> = <dx, d>
    x, dy, d = (rows_of(s, 16, 200, "f32") for s in (1, 2, 3))
    gamma, beta = vector(1, 200, 0.5), vector(2, 200)
    _, stats = capi.layer_norm(x, gamma, beta, EPS, return_stats=True)
    dx, dgamma, _ = capi.layer_norm_backward(dy, x, gamma, stats)
    step = 2.0 ** -8
    up, down = (capi.layer_norm(x + k * step * d, gamma, beta, EPS) for k in (1, -1))
    quotient = ((up.double() - down.double()) / (2 * step) * dy.double()).sum(1)
    slope = (dx.double() * d.double()).sum(1)
    # truncation: step^2 / 6 times a third derivative of order 10 per element; rounding: 2^-24 / step per element
    size = dy.double().abs().sum(1) * 4
    assert ((quotient - slope).abs() <= size * (2 * step ** 2 + 4 * E32 / step)).all()


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("c", WIDTHS)
def test_quantize_rows(capi, c, dtype):
    for rows, pad, offset in ((1, 0, 0), (37, 0, 0), (5, 8, 8), (5, 3, 1)):
        x = rows_of(c, rows, c, dtype, pad, offset)
        q, scale = capi.quantize_rows(x)
        wq, ws = ref.quantize_rows_f32(x.float().cpu().numpy())
        assert np.array_equal(q.cpu().numpy(), wq) and np.array_equal(scale.cpu().numpy(), ws)
        # half a step, and the fp32 product's rounding at up to 127 steps
        assert (np.abs(host(q) * host(scale)[:, None] - host(x)) <= host(scale)[:, None] * (0.5 + 127 * 4 * E32)).all()


def test_quantize_special_rows(capi):
    x = torch.zeros(6, 100, device="cuda")
    x[1, 3], x[2, 5], x[3, 5], x[4] = float("nan"), float("inf"), float("-inf"), 1e-40
    x[5] = torch.linspace(-1, 1, 100)
    q, scale = capi.quantize_rows(x)
    assert not q[:5].any() and scale[1].isnan() and scale[2].isinf() and scale[3].isinf()
    assert scale[0] > 0 and scale[4] == scale[0] and q[5, 0] == -127 and q[5, -1] == 127
    y = capi.linear_int8(q, torch.ones(8, 100, dtype=torch.int8, device="cuda"), scale, torch.ones(8, device="cuda"))
    assert y[1].isnan().all() and y[2].isnan().all() and y[3].isnan().all() and not y[0].any()


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("c", WIDTHS)
def test_layer_norm_quantize(capi, c, dtype):
    for rows, pad, offset in ((1, 0, 0), (37, 0, 0), (5, 3, 1)):
        x = rows_of(c, rows, c, dtype, pad, offset, shift=0.5)
        gamma, beta = vector(1, c, 0.5), vector(2, c)
        q, scale = capi.layer_norm_quantize(x, gamma, beta, EPS)
        v, mean, rstd = ref.layer_norm(host(x), host(gamma), host(beta), EPS)
        off = norm_bound(x, gamma, v, mean, rstd, "f32")
        want = ref.row_scales(v)
        assert (np.abs(host(scale) - want) <= off.max(1) / 127 + 4 * E32 * want).all()
        # half a step, the value's own error and the scale's at up to 127 steps
        assert (np.abs(host(q) * host(scale)[:, None] - v)
                <= host(scale)[:, None] * (0.5 + 127 * 8 * E32) + off + off.max(1)[:, None]).all()


# ---------------------------------------------------------------- linear
def ints(seed, rows, k, pad=0, offset=0):
    g = torch.Generator().manual_seed(seed)
    return torch.randint(-128, 128, (rows, k + pad + offset), generator=g, dtype=torch.int8).cuda()[:, offset:offset + k]


def check_linear(capi, m, n, k, out="bf16", activation="identity", bias=True, residual=False, pad=0, offset=0, a=None,
                 w=None, seed=0):
    a = ints(seed + 1, m, k, pad, offset) if a is None else a
    w = ints(seed + 2, n, k, pad, offset) if w is None else w
    a_scale, w_scale = vector(3, m, 0.5) / 64, vector(4, n, 0.5) / (64 * max(1, k) ** 0.5)
    b = vector(5, n) if bias else None
    res = rows_of(6, m, n, out, pad) if residual else None
    store = torch.full((m, n + pad + offset), 7.0, dtype=TYPES[out], device="cuda")
    y = capi.linear_int8(a, w, a_scale, w_scale, b, activation, res, TYPES[out], y=store[:, offset:offset + n])
    want, z, total = ref.linear_int8(host(a), host(w), host(a_scale), host(w_scale), None if b is None else host(b),
                                     activation, None if res is None else host(res))
    scales = host(a_scale)[:, None] * host(w_scale)[None, :]
    # sums below 2^24 are exact; beyond, each of the k/16 additions of a tensor-core sum (or the one
    # rounding of an integer sum) errs by up to 2^-23 of the largest partial sum
    summed = np.where(total < 2.0 ** 24, 0.0, (k / 16 + 1) * 2.0 ** -23 * total)
    zerr = scales * summed + 4 * E32 * (np.abs(z) + scales * total)
    act = zerr * 1.1
    if activation == "silu":  # the exponential errs by 2 + 1.2|z| ulp, the quotient by 2
        act = act + np.abs(ref.activate(z, "silu")) * (6 + 1.2 * np.abs(z)) * 2 * E32 + 1e-37
    tol = act + 2 * E32 * np.abs(want) + ROUND[out] * 1.001 * np.abs(want) + LEAST[out]
    off = np.abs(host(y) - want)
    assert (off <= tol).all(), (m, n, k, float((off - tol).max()))
    assert (store[:, :offset] == 7).all() and (store[:, offset + n:] == 7).all()
    capi.check()


SIZES = [(1, 1, 1), (1, 8, 16), (1, 64, 64), (1, 128, 4096), (1, 300, 1000), (2, 7, 33), (3, 129, 65), (4, 256, 2048),
         (5, 1000, 17), (7, 65, 127), (8, 128, 128), (8, 512, 4096), (9, 257, 1008), (12, 96, 8192), (15, 64, 32),
         (16, 16, 16), (17, 255, 129), (24, 384, 640), (31, 63, 15), (32, 256, 4096), (33, 128, 1024), (48, 777, 96),
         (63, 200, 208), (64, 1024, 2048), (65, 136, 80), (100, 1, 512), (127, 127, 127), (128, 128, 64),
         (129, 264, 192), (200, 640, 1001), (255, 129, 255), (256, 256, 256), (257, 520, 384), (300, 33, 4096),
         (333, 777, 1001), (512, 512, 512), (513, 257, 65), (640, 128, 3), (1000, 1000, 1000), (1025, 300, 528),
         (2048, 64, 128), (3000, 520, 272), (1, 5, 0), (70, 9, 0)]


@pytest.mark.parametrize("m,n,k", SIZES)
def test_linear(capi, m, n, k):
    which = (m * 7 + n * 3 + k) % 9
    check_linear(capi, m, n, k, list(TYPES)[which % 3], ("identity", "silu", "relu")[which // 3], residual=bool(m & 1))


@pytest.mark.parametrize("out", list(TYPES))
@pytest.mark.parametrize("activation", ["identity", "silu", "relu"])
@pytest.mark.parametrize("m", [1, 6, 40, 100, 300])
def test_linear_epilogues(capi, m, activation, out):
    check_linear(capi, m, 264, 320, out, activation, bias=False, residual=False)
    check_linear(capi, m, 264, 320, out, activation, bias=True, residual=True)


@pytest.mark.parametrize("out", list(TYPES))
@pytest.mark.parametrize("pad,offset", [(16, 0), (16, 16), (7, 0), (3, 1), (8, 8)])
@pytest.mark.parametrize("m,n,k", [(1, 136, 256), (6, 136, 250), (40, 129, 512), (200, 200, 333), (600, 264, 128)])
def test_linear_of_slices(capi, m, n, k, pad, offset, out):
    check_linear(capi, m, n, k, out, "relu", residual=True, pad=pad, offset=offset)


@pytest.mark.parametrize("m", [1, 8, 16, 64, 130, 512])
@pytest.mark.parametrize("k", [1024, 16384, 131071])
def test_linear_of_extreme_integers(capi, m, k):
    if m * k > 1 << 25:
        pytest.skip("same arithmetic at smaller m")
    low = torch.full((m, k), -128, dtype=torch.int8, device="cuda")
    check_linear(capi, m, 40, k, "f32", a=low, w=torch.full((40, k), -128, dtype=torch.int8, device="cuda"))
    mixed = torch.where(torch.arange(k, device="cuda") % 2 == 0, 127, -128).to(torch.int8).expand(40, k)
    check_linear(capi, m, 40, k, "f32", a=low, w=mixed)


def test_linear_exact_below_two_to_the_24(capi):
    # k = 1024 of the largest products: every partial sum is an integer up to 2^24
    for m in (1, 8, 50, 200, 700):
        a, w = ints(1, m, 1024), ints(2, 192, 1024)
        one_m, one_n = torch.ones(m, device="cuda"), torch.ones(192, device="cuda")
        y = capi.linear_int8(a, w, one_m, one_n, out_dtype=torch.float32)
        assert torch.equal(y.double(), a.double() @ w.double().t())


def test_linear_in_place_residual_dimensions_and_empty(capi):
    a, w = ints(1, 60, 128), ints(2, 72, 128)
    sa, sw = vector(3, 60, 0.5), vector(4, 72, 0.5)
    res = rows_of(5, 60, 72, "bf16")
    want = capi.linear_int8(a, w, sa, sw, residual=res)
    y = res.clone()
    assert torch.equal(capi.linear_int8(a, w, sa, sw, residual=y, y=y), want)
    cube = capi.linear_int8(a.reshape(3, 4, 5, 128), w, sa.view(3, 4, 5), sw, residual=res.view(3, 4, 5, 72))
    assert cube.shape == (3, 4, 5, 72) and torch.equal(cube.view(60, 72), want)
    assert capi.linear_int8(a[:0], w, sa[:0], sw).shape == (0, 72)
    assert capi.linear_int8(a, w[:0], sa, sw[:0]).shape == (60, 0)
    same = capi.linear_int8(a[:1].expand(60, 128), w, sa[:1].expand(60).contiguous(), sw)
    assert torch.equal(same, same[:1].expand(60, 72))


def test_operators_on_another_stream_and_in_a_graph(capi):
    x = rows_of(1, 500, 512, "bf16")
    w, sw = ints(2, 640, 512), vector(3, 640, 0.5) / 1000
    gamma, beta = vector(4, 512, 0.5), vector(5, 512)

    def block(stream=None):
        y, stats = capi.layer_norm(x, gamma, beta, EPS, return_stats=True, stream=stream)
        grads = capi.layer_norm_backward(y, x, gamma, stats, stream=stream)
        q, scale = capi.layer_norm_quantize(x, gamma, beta, EPS, stream=stream)
        return (*grads, capi.linear_int8(q, w, scale, sw, activation="silu", stream=stream),
                capi.linear_int8(q[:3], w, scale[:3], sw, stream=stream))

    want = [t.clone() for t in block()]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for stream in (side, side.cuda_stream):
        got = block(stream)
        side.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(want, got))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = block()
    x0 = x.clone()
    x.copy_(rows_of(9, 500, 512, "bf16"))
    fresh = [t.clone() for t in block()]
    graph.replay()
    assert all(torch.equal(a, b) for a, b in zip(fresh, got))
    x.copy_(x0)
    graph.replay()
    assert all(torch.equal(a, b) for a, b in zip(want, got))


def test_binding_refusals(capi):
    x, w = rows_of(1, 4, 64, "bf16"), ints(1, 32, 64)
    a, sa, sw = ints(2, 4, 64), vector(1, 4), vector(1, 32)
    with pytest.raises(TypeError):
        capi.layer_norm(x.double())
    with pytest.raises(TypeError):
        capi.layer_norm(x, gamma=vector(1, 64).half())
    with pytest.raises(ValueError):
        capi.layer_norm(x, gamma=vector(1, 63))
    with pytest.raises(ValueError):
        capi.layer_norm(x.cpu())
    with pytest.raises(ValueError):
        capi.layer_norm(x.t())
    with pytest.raises(ValueError):
        capi.layer_norm(x, y=torch.empty(4, 63, dtype=x.dtype, device="cuda"))
    with pytest.raises(ValueError):
        capi.layer_norm(rows_of(1, 24, 64, "bf16").view(2, 12, 64)[:, ::5])
    with pytest.raises(capi.CbsError):
        capi.layer_norm(x, eps=-1.0)
    with pytest.raises(capi.CbsError):
        capi.layer_norm(x[:, :0])
    _, stats = capi.layer_norm(x, return_stats=True)
    with pytest.raises(TypeError):
        capi.layer_norm_backward(x.float(), x, None, stats)
    with pytest.raises(ValueError):
        capi.layer_norm_backward(x[:2], x, None, stats)
    with pytest.raises(ValueError):
        capi.layer_norm_backward(x, x, None, stats[:, :3].contiguous())
    with pytest.raises(TypeError):
        capi.linear_int8(x, w, sa, sw)
    with pytest.raises(ValueError):
        capi.linear_int8(a[:, :60], w, sa, sw)
    with pytest.raises(ValueError):
        capi.linear_int8(a, w, sa[:3], sw)
    with pytest.raises(ValueError):
        capi.linear_int8(a, w, sa, sw, activation="gelu")
    with pytest.raises(TypeError):
        capi.linear_int8(a, w, sa, sw, out_dtype=torch.float64)
    with pytest.raises(TypeError):
        capi.linear_int8(a, w, sa, sw, residual=torch.zeros(4, 32, device="cuda"))
    with pytest.raises(ValueError):
        capi.linear_int8(a, w, sa, sw, residual=torch.zeros(4, 31, dtype=torch.bfloat16, device="cuda"))


# Sizes at which each of the layer's kernels is the one that runs (152 SMs): weights widened on their way with
# row tiles of 32, 64, 128 and 256, then both widened before, in tiles of 128 x 64, 256 x 128 and 256 x 256.
LARGER = [(20, 300, 4096), (40, 712, 2048), (100, 712, 2048), (300, 300, 4096), (700, 1300, 400), (1500, 1300, 400),
          (2300, 2000, 1040)]


@pytest.mark.parametrize("out", list(TYPES))
@pytest.mark.parametrize("activation", ["identity", "silu", "relu"])
@pytest.mark.parametrize("m,n,k", LARGER)
def test_larger_linear_epilogues(capi, m, n, k, activation, out):
    check_linear(capi, m, n, k, out, activation, bias=False, residual=False)
    check_linear(capi, m, n, k, out, activation, bias=True, residual=True)
    check_linear(capi, m, n - 3, k, out, activation, bias=True, residual=True)  # columns and rows of y at any alignment


@pytest.mark.parametrize("out", list(TYPES))
@pytest.mark.parametrize("pad,offset", [(16, 0), (16, 16), (7, 0), (3, 1), (8, 8)])
@pytest.mark.parametrize("m,n,k", [(20, 300, 4096), (40, 707, 2001), (130, 712, 2048), (300, 296, 4095), (710, 1296, 403),
                                   (1501, 1300, 400)])
def test_larger_linear_of_slices(capi, m, n, k, pad, offset, out):
    check_linear(capi, m, n, k, out, "silu", residual=True, pad=pad, offset=offset)


@pytest.mark.parametrize("m,n,k", [(3, 264, 320), (40, 264, 320)] + LARGER)
def test_linear_silu_far_from_zero_and_special_scales(capi, m, n, k):
    a, w = ints(1, m, k), ints(2, n, k)
    # z has a deviation of some 50, so that many are where e^-z leaves the range of fp32
    a_scale, w_scale = vector(3, m, 0.5), vector(4, n, 0.5) * 0.6 / (64 * k ** 0.5)
    y = capi.linear_int8(a, w, a_scale, w_scale, activation="silu", out_dtype=torch.float32)
    want, z, total = ref.linear_int8(host(a), host(w), host(a_scale), host(w_scale), None, "silu", None)
    assert (z < -88).any() and (z > 88).any()
    scales = host(a_scale)[:, None] * host(w_scale)[None, :]
    summed = np.where(total < 2.0 ** 24, 0.0, (k / 16 + 1) * 2.0 ** -23 * total)
    zerr = scales * summed + 4 * E32 * (np.abs(z) + scales * total)
    tol = zerr * 1.1 + np.abs(want) * (6 + 1.2 * np.abs(z)) * 2 * E32 + 1e-37 + 3 * E32 * np.abs(want)
    assert (np.abs(host(y) - want) <= tol).all()
    # a NaN or an infinity among the scales is its own row's and column's alone
    a_scale[m // 2], w_scale[5], w_scale[n - 1] = float("inf"), float("nan"), float("inf")
    y = host(capi.linear_int8(a, w, a_scale, w_scale, activation="silu", out_dtype=torch.float32))
    assert np.isnan(y[:, 5]).all() and not np.isfinite(y[m // 2][z[m // 2] > 0]).any()
    rows, cols = np.arange(m) != m // 2, np.ones(n, bool)
    cols[[5, n - 1]] = False
    assert (np.abs(y - want) <= tol)[np.ix_(rows, cols)].all()
    capi.check()


@pytest.mark.parametrize("m,n,k", [(8, 300, 4096)] + LARGER)
def test_linear_repeats_to_the_bit(capi, m, n, k):
    a, w, sa, sw = ints(1, m, k), ints(2, n, k), vector(3, m, 0.5), vector(4, n, 0.5)
    first = capi.linear_int8(a, w, sa, sw, activation="silu")
    assert all(torch.equal(first, capi.linear_int8(a, w, sa, sw, activation="silu")) for _ in range(5))


# Few channels for many rows: the rows are widened on their way.
# (Of these, 6000x300x8192 is modelled faster with both widened before, and runs so; tests/linear_cases.py has sizes
# whose kernel is asserted.)
TURNED = [(700, 40, 4096), (1500, 9, 4096), (5000, 33, 1040), (9000, 100, 2048), (9000, 200, 4096), (6000, 300, 8192)]


@pytest.mark.parametrize("out", list(TYPES))
@pytest.mark.parametrize("activation", ["identity", "silu", "relu"])
@pytest.mark.parametrize("m,n,k", TURNED)
def test_linear_of_few_channels(capi, m, n, k, activation, out):
    check_linear(capi, m, n, k, out, activation, bias=False, residual=False)
    check_linear(capi, m - 1, n, k, out, activation, bias=True, residual=True)
    check_linear(capi, m, n, k, out, activation, bias=True, residual=True, pad=16, offset=16)


@pytest.mark.parametrize("m,n,k", TURNED)
def test_linear_of_few_channels_repeats_to_the_bit(capi, m, n, k):
    a, w, sa, sw = ints(1, m, k), ints(2, n, k), vector(3, m, 0.5), vector(4, n, 0.5)
    first = capi.linear_int8(a, w, sa, sw, activation="silu")
    assert all(torch.equal(first, capi.linear_int8(a, w, sa, sw, activation="silu")) for _ in range(5))
    sa[m // 2] = float("nan")
    y = capi.linear_int8(a, w, sa, sw, activation="silu")
    assert y[m // 2].isnan().all()
    rest = torch.arange(m, device="cuda") != m // 2
    assert torch.equal(y[rest], first[rest])


# Rows that start at multiples of 4 bytes, and one size of more channels than a tile of the turned product.
@pytest.mark.parametrize("out", list(TYPES))
@pytest.mark.parametrize("m,n,k,pad", [(904, 64, 12644, 0), (64, 3265, 2004, 0), (2368, 40, 4996, 0), (300, 296, 4092, 0),
                                       (100, 712, 2052, 4), (20, 300, 4100, 8), (700, 40, 4096, 4), (64, 300, 4096, 12),
                                       (5467, 386, 9264, 0)])
def test_linear_of_rows_at_words(capi, m, n, k, pad, out):
    check_linear(capi, m, n, k, out, "silu", residual=True, pad=pad, offset=pad)


# Rows that start anywhere, at sizes for which they are widened on their way.
# (Of these, 6000x250x4101 runs with both widened before, and 64x1000x129 in the one-launch tile kernel.)
@pytest.mark.parametrize("out", list(TYPES))
@pytest.mark.parametrize("m,n,k,pad", [(13, 4000, 6005, 0), (20, 300, 4097, 0), (40, 712, 2050, 0), (100, 712, 2051, 0),
                                       (300, 300, 4095, 0), (200, 1000, 2048, 7), (1024, 38, 4967, 0), (3823, 21, 2853, 0),
                                       (5000, 100, 4018, 1), (5000, 33, 2048, 3), (6000, 250, 4101, 0), (64, 1000, 129, 2)])
def test_linear_of_rows_anywhere(capi, m, n, k, pad, out):
    check_linear(capi, m, n, k, out, "silu", residual=True, pad=pad, offset=pad)


@pytest.mark.parametrize("out", list(TYPES))
@pytest.mark.parametrize("m,n,k", LARGER + TURNED[:5])
def test_larger_linear_adds_to_its_residual_in_place(capi, m, n, k, out):
    a, w, sa, sw = ints(1, m, k), ints(2, n, k), vector(3, m, 0.5) / 64, vector(4, n, 0.5) / (64 * k ** 0.5)
    res = rows_of(5, m, n, out)
    want = capi.linear_int8(a, w, sa, sw, None, "silu", res, TYPES[out])
    y = res.clone()
    assert capi.linear_int8(a, w, sa, sw, None, "silu", y, TYPES[out], y=y) is not None
    assert torch.equal(y, want)


@pytest.mark.parametrize("m,n,k", [(5, 300, 4096), (20, 300, 4096), (64, 712, 2048), (300, 300, 4096), (1500, 9, 4096), (1500, 1300, 400)])
def test_linear_of_one_row_broadcast(capi, m, n, k):
    a = ints(1, 1, k).expand(m, k)
    check_linear(capi, m, n, k, "f32", "silu", residual=True, a=a)
    check_linear(capi, m, n, k, "bf16", a=a, w=ints(2, 1, k).expand(n, k))


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("rows,c", [(3, 9501), (40, 12345), (700, 16383), (1001, 9001)])
def test_layer_norm_of_long_rows_off_alignment(capi, rows, c, dtype):
    x, gamma, beta = rows_of(c, rows, c, dtype, pad=1), vector(1, c, 0.5), vector(2, c)
    y, stats = capi.layer_norm(x, gamma, beta, EPS, return_stats=True)
    want, mean, rstd = ref.layer_norm(host(x), host(gamma), host(beta), EPS)
    assert (np.abs(host(y) - want) <= norm_bound(x, gamma, want, mean, rstd, dtype)).all()
    q, scale = capi.quantize_rows(x)
    most = np.abs(host(x)).max(1)
    assert (np.abs(host(scale) * 127 - most) <= 4 * E32 * most).all()
    assert (np.abs(host(q) * host(scale)[:, None] - host(x)) <= host(scale)[:, None] * (0.5 + 127 * 8 * E32)).all()
