"""Low-rank adapters and their gradients on the GPU against the 64-bit oracle.  Bounds come from the
arithmetic: a matrix instruction's additions may cut instead of round (two unit roundoffs each, 16
products an addition), 16-bit hidden rows are rounded once to the activations' type, the weights'
gradients take the hidden rows in two parts (bf16: 2^-18 of them)."""
import numpy as np
import pytest
import torch

from oracle import token_ops as ref

pytestmark = pytest.mark.gpu

TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
ROUND = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8, "f16": 2.0 ** -11}
LEAST = {"f32": 2.0 ** -149, "bf16": 2.0 ** -133, "f16": 2.0 ** -24}
E32 = 2.0 ** -24


@pytest.fixture(scope="module")
def capi():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from conv2d_batchnorm_silu_gb300 import capi
    return capi


def host(t):
    return t.detach().double().cpu().numpy()


def made(seed, *shape, dtype="f32", size=1.0, pad=0, offset=0):
    """On the GPU, the last dimension a slice of one `pad` wider from `offset` on."""
    g = torch.Generator().manual_seed(seed)
    full = torch.randn(*shape[:-1], shape[-1] + pad + offset, generator=g) * size
    return full.to(TYPES[dtype]).cuda()[..., offset:offset + shape[-1]]


def index_of(seed, m, adapters, kind):
    rng = np.random.default_rng(seed)
    if kind == "mixed":
        v = rng.integers(-1, adapters + 1, m)
    elif kind == "runs":
        v = np.repeat(rng.integers(-1, adapters, 5), m // 5 + 1)[:m]
    elif kind == "one":
        v = np.full(m, adapters - 1)
    else:  # none has one
        v = np.where(rng.random(m) < 0.5, -2 ** 31, 2 ** 31 - 1)
    return torch.from_numpy(v.astype(np.int32)).cuda()


def sums(length):
    """Relative error, of the sum of the terms' magnitudes, of a sum of `length` products."""
    return (length / 16 + 64) * 2 * E32


PARTS = {"f32": 2.0 ** -20, "bf16": 0.0, "f16": 0.0}       # of products of two-part floats
SMALL = {"f32": 2.0 ** -20, "bf16": 2.0 ** -17, "f16": 2.0 ** -21}  # of hidden rows in two parts


def product_bound(total, first, rank, want, hidden, w2, s, dtype):
    """Of s * w2 @ hidden + base: total, the sum of all terms' magnitudes; first, the first product's length."""
    bound = total * (sums(first) + sums(rank) + 2 * PARTS[dtype] + 4 * E32) + (ROUND[dtype] * 1.001 + 2 * E32) * np.abs(want) + LEAST[dtype]
    if dtype != "f32":
        bound = bound + s[:, None] * np.einsum("inr,ir->in", w2, np.abs(hidden)) * ROUND[dtype] * 1.01
        if dtype == "f16":  # values far below a row's largest keep 2^-24 of that
            bound = bound + s[:, None] * w2.sum(2) * np.abs(hidden).max(1, keepdims=True) * 2.0 ** -24
    return bound


def check(capi, m, k, n, rank, adapters, dtype, kind, pad=0, offset=0, with_base=True, with_scale=True):
    x, base = made(1, m, k, dtype=dtype, pad=pad, offset=offset), made(2, m, n, dtype=dtype, pad=pad, offset=offset)
    a, b = made(3, adapters, rank, k, dtype=dtype, size=k ** -0.5), made(4, adapters, n, rank, dtype=dtype)
    scale = (0.5 + torch.rand(adapters, generator=torch.Generator().manual_seed(5))).cuda() if with_scale else None
    index = index_of(m + k, m, adapters, kind)
    y, hidden = capi.linear_adapters(x, index, a, b, scale, base=base if with_base else None, return_hidden=True)
    at = index.cpu().numpy()
    own = np.where((at >= 0) & (at < adapters), at, -1)
    s_host = np.ones(adapters) if scale is None else host(scale)
    want, want_h, total = ref.linear_adapters(host(x), at, host(a), host(b), s_host, host(base) if with_base else None)
    s = np.where(own >= 0, s_host[own], 0.0)
    off_h = sums(k) + PARTS[dtype] + 2 * E32
    terms_h = np.stack([np.abs(host(a)[g]) @ np.abs(host(x)[i]) if g >= 0 else np.zeros(rank) for i, g in enumerate(own)])
    assert y.dtype == x.dtype and y.shape == (m, n) and hidden.shape == (m, rank)
    assert (np.abs(host(hidden) - want_h) <= off_h * terms_h).all()
    w2 = np.abs(host(b))[own]
    assert (np.abs(host(y) - want) <= product_bound(total, k, rank, want, want_h, w2, s, dtype)).all()
    again = capi.linear_adapters(x, index, a, b, scale, base=base if with_base else None)
    assert torch.equal(again, y)  # the same bits, with hidden rows kept or not

    dy = made(6, m, n, dtype=dtype, pad=pad, offset=offset, size=0.1)
    gbase = made(7, m, k, dtype=dtype, pad=pad, offset=offset, size=0.1) if with_base else None
    dx, da, db = capi.linear_adapters_backward(dy, x, index, a, b, scale, hidden, base=gbase)
    (wx, wa, wb), (tx, ta, tb) = ref.linear_adapters_backward(host(dy), host(x), at, host(a), host(b), s_host, host(hidden),
                                                              None if gbase is None else host(gbase))
    dh = np.stack([host(b)[g].T @ host(dy)[i] if g >= 0 else np.zeros(rank) for i, g in enumerate(own)])
    assert (np.abs(host(dx) - wx) <= product_bound(tx, n, rank, wx, dh, np.abs(host(a))[own].transpose(0, 2, 1), s, dtype)).all()
    assert da.shape == a.shape and db.shape == b.shape and da.dtype == db.dtype == torch.float32
    off = sums(m) + SMALL[dtype] + PARTS[dtype] + 8 * E32
    assert (np.abs(host(da) - wa) <= ta * (off + sums(n) + PARTS[dtype])).all()
    assert (np.abs(host(db) - wb) <= tb * off).all()
    for g in range(adapters):
        if not (own == g).any():
            assert (da[g] == 0).all() and (db[g] == 0).all()
    for got, first in zip(capi.linear_adapters_backward(dy, x, index, a, b, scale, hidden, base=gbase), (dx, da, db)):
        assert torch.equal(got, first)


SIZES = [(1, 32, 16, 1, 1), (1, 2048, 1024, 16, 8), (3, 40, 24, 4, 2), (17, 8, 8, 8, 3), (33, 100, 77, 12, 5), (64, 256, 512, 16, 70),
         (255, 64, 96, 16, 1), (256, 96, 128, 32, 3), (257, 128, 64, 16, 2), (300, 136, 264, 64, 4), (400, 128, 128, 128, 3),
         (500, 33, 31, 100, 2), (1500, 72, 40, 16, 2), (2100, 64, 64, 24, 40), (5000, 40, 48, 8, 1), (130, 1, 1, 3, 4),
         (1024, 16, 32, 48, 300), (1025, 520, 16, 16, 1), (1300, 200, 136, 64, 3), (2500, 264, 128, 32, 2), (1100, 152, 56, 40, 8),
         (600, 128, 64, 128, 2), (3000, 32, 32, 8, 120), (65, 40, 48, 16, 95), (1000, 64, 64, 16, 94), (640, 48, 40, 4, 30)]


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("kind", ["mixed", "runs", "one", "none"])
@pytest.mark.parametrize("m,k,n,rank,adapters", SIZES)
def test_sizes(capi, m, k, n, rank, adapters, kind, dtype):
    check(capi, m, k, n, rank, adapters, dtype, kind)


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("pad,offset", [(8, 0), (8, 8), (3, 1), (23, 4)])
@pytest.mark.parametrize("m,k,n,rank,adapters", [(9, 64, 96, 8, 2), (300, 72, 80, 16, 3), (260, 33, 65, 20, 2)])
def test_slices(capi, m, k, n, rank, adapters, pad, offset, dtype):
    check(capi, m, k, n, rank, adapters, dtype, "mixed", pad, offset, with_base=offset != 8, with_scale=pad != 3)


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("m,n", [(5, 24), (200, 77), (900, 64)])
def test_in_place_and_rows_without_an_adapter(capi, m, n, dtype):
    x, a, b = made(1, m, 48, dtype=dtype), made(2, 3, 16, 48, dtype=dtype), made(3, 3, n, 16, dtype=dtype)
    wide = made(4, m + 3, n + 8, dtype=dtype)
    wide[-3:] = float("nan")  # rows of a padded batch behind the last sequence
    x = torch.cat((x, torch.full((3, 48), float("nan"), device="cuda", dtype=x.dtype)))
    index = index_of(1, m + 3, 3, "mixed")
    index[-3:] = -1
    before = wide.clone()
    want, hidden = capi.linear_adapters(x, index, a, b, base=wide[:, :n], return_hidden=True)
    got = capi.linear_adapters(x, index, a, b, base=wide[:, :n], y=wide[:, :n])
    assert got.data_ptr() == wide.data_ptr()
    bits = torch.int32 if dtype == "f32" else torch.int16
    without = (index < 0) | (index >= 3)
    assert torch.equal(wide[without].view(bits), before[without].view(bits)) and torch.equal(wide[:, n:].view(bits), before[:, n:].view(bits))
    assert torch.equal(wide[:m, :n], want[:m]) and want[-3:].isnan().all() and (hidden[without] == 0).all()
    dy, into = made(5, m + 3, n, dtype=dtype), made(6, m + 3, 48, dtype=dtype)
    dy[-3:] = float("nan")
    keep = into.clone()
    want = capi.linear_adapters_backward(dy, x, index, a, b, None, hidden, base=keep)
    dx, da, db = capi.linear_adapters_backward(dy, x, index, a, b, None, hidden, base=into, dx=into)
    assert torch.equal(dx, want[0]) and torch.equal(da, want[1]) and torch.equal(db, want[2])
    assert torch.equal(into[without], keep[without]) and da.isfinite().all() and db.isfinite().all()


@pytest.mark.parametrize("dtype", list(TYPES))
def test_values_that_are_not_finite_stay_in_their_rows(capi, dtype):
    for m in (40, 600):
        x, a, b = made(1, m, 64, dtype=dtype), made(2, 4, 16, 64, dtype=dtype), made(3, 4, 40, 16, dtype=dtype)
        index = torch.arange(m, device="cuda").remainder(4).int()
        want = capi.linear_adapters(x, index, a, b)
        x2, a2 = x.clone(), a.clone()
        x2[4, 3], x2[9, 63], a2[3, 2, 5] = float("nan"), float("inf"), float("nan")
        got = capi.linear_adapters(x2, index, a2, b)
        spoiled = index == 3
        spoiled[4] = spoiled[9] = True
        assert torch.equal(got[~spoiled], want[~spoiled]) and not got[spoiled].isfinite().any()


def test_hidden_rows_beyond_the_range_of_f16(capi):
    """Rows whose hidden values leave f16 (65504), or lie below its smallest, as long as y does not."""
    for m in (6, 300):
        x, a = torch.ones(m, 512, device="cuda", dtype=torch.float16), torch.ones(1, 8, 512, device="cuda", dtype=torch.float16)
        x[0] *= 1000
        x[1] *= 2.0 ** -20
        b, scale = made(1, 1, 32, 8, dtype="f16", size=0.5), torch.full((1,), 0.001, device="cuda")
        y, hidden = capi.linear_adapters(x, torch.zeros(m, dtype=torch.int32, device="cuda"), a, b, scale, return_hidden=True)
        assert (hidden[0] == 512000).all() and y.isfinite().all()
        want = 0.001 * host(hidden) @ host(b)[0].T
        assert (np.abs(host(y) - want) <= 2.0 ** -10 * 0.001 * np.abs(host(hidden)) @ np.abs(host(b)[0].T) + 2.0 ** -24).all()


def test_gradient_by_differences(capi):
    """Central differences of the forward call in fp32, which is of the third order in a, b and x: a step of 2^-5 and
    errors of some 2^-18 of values of order 10 leave 2^-9 of them."""
    m, k, n, rank, adapters = 7, 24, 20, 5, 2
    x, a, b, dy = made(1, m, k), made(2, adapters, rank, k, size=0.3), made(3, adapters, n, rank, size=0.3), made(4, m, n)
    scale, index = torch.tensor([0.5, 2.0], device="cuda"), torch.tensor([0, 1, 1, -1, 0, 5, 1], dtype=torch.int32, device="cuda")
    _, hidden = capi.linear_adapters(x, index, a, b, scale, return_hidden=True)
    grads = capi.linear_adapters_backward(dy, x, index, a, b, scale, hidden)
    step = 2.0 ** -5

    def loss(x, a, b):
        return float((capi.linear_adapters(x, index, a, b, scale).double() * dy.double()).sum())

    for which, grad in enumerate(grads):
        args = [x, a, b]
        for flat in (0, 11, grad.numel() // 2 + 3, grad.numel() - 1):
            e = torch.zeros_like(args[which]).view(-1)
            e[flat] = step
            up, down = list(args), list(args)
            up[which], down[which] = args[which] + e.view_as(args[which]), args[which] - e.view_as(args[which])
            assert abs((loss(*up) - loss(*down)) / (2 * step) - float(grad.view(-1)[flat])) < 2e-2


def test_leading_dimensions_streams_and_graphs(capi):
    for m in (24, 600):
        x = made(1, 2, m // 2, 64, dtype="bf16")
        a, b = made(2, 3, 16, 64, dtype="bf16"), made(3, 3, 32, 16, dtype="bf16")
        index = index_of(2, m, 3, "mixed")
        y, hidden = capi.linear_adapters(x, index.view(2, m // 2), a, b, return_hidden=True)
        assert y.shape == (2, m // 2, 32) and hidden.shape == (2, m // 2, 16)
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        other = capi.linear_adapters(x, index, a, b, stream=side)
        side.synchronize()
        assert torch.equal(other, y)
        dy = made(4, 2, m // 2, 32, dtype="bf16")
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            y2, hidden2 = capi.linear_adapters(x, index, a, b, return_hidden=True)
            grads = capi.linear_adapters_backward(dy, x, index, a, b, None, hidden2)
        index.copy_(index_of(9, m, 3, "mixed"))  # the next step's requests
        x.copy_(x.flip(1))
        graph.replay()
        want, want_h = capi.linear_adapters(x, index, a, b, return_hidden=True)
        assert torch.equal(y2, want) and torch.equal(hidden2, want_h)
        for got, w in zip(grads, capi.linear_adapters_backward(dy, x, index, a, b, None, want_h)):
            assert torch.equal(got, w)


def test_rows_do_not_depend_on_their_neighbours(capi):
    """A row gives the same bits in whatever batch of the same kernels it comes, and one row for all costs no more."""
    x, a, b = made(1, 900, 96, dtype="bf16"), made(2, 5, 16, 96, dtype="bf16"), made(3, 5, 64, 16, dtype="bf16")
    index = index_of(3, 900, 5, "mixed")
    y = capi.linear_adapters(x, index, a, b)
    order = torch.randperm(900, generator=torch.Generator().manual_seed(1)).cuda()
    assert torch.equal(capi.linear_adapters(x[order].contiguous(), index[order].contiguous(), a, b), y[order])
    one = capi.linear_adapters(x[:1].expand(900, 96), index, a, b)
    for g in range(5):
        rows = (index == g).nonzero()[:, 0]
        assert (one[rows] == one[rows[0]]).all()


def test_many_adapters(capi):
    """As many as a call takes, few of them used, in batches on both sides of the kernels' sizes."""
    a, b = made(1, 4096, 4, 16, dtype="bf16"), made(2, 4096, 8, 4, dtype="bf16")
    for m in (1, 200, 2000, 5000):
        x, dy = made(3, m, 16, dtype="bf16"), made(4, m, 8, dtype="bf16")
        index = torch.randint(0, 4096, (m,), generator=torch.Generator().manual_seed(m)).int().cuda()
        index[: m // 2] = 4095
        y, hidden = capi.linear_adapters(x, index, a, b, return_hidden=True)
        want_h = torch.einsum("mrk,mk->mr", a[index.long()].double(), x.double())
        assert (hidden.double() - want_h).abs().max() <= 1e-4
        want = torch.einsum("mnr,mr->mn", b[index.long()].double(), want_h)
        assert (y.double() - want).abs().max() <= 2.0 ** -6 * want.abs().max()
        dx, da, db = capi.linear_adapters_backward(dy, x, index, a, b, None, hidden)
        wb = torch.zeros(4096, 8, 4, dtype=torch.float64, device="cuda").index_add_(
            0, index.long(), torch.einsum("mn,mr->mnr", dy.double(), hidden.double()))
        assert (db.double() - wb).abs().max() <= 1e-4 * wb.abs().max()


def test_refusals(capi):
    x, a, b = made(1, 4, 16, dtype="bf16"), made(2, 2, 8, 16, dtype="bf16"), made(3, 2, 24, 8, dtype="bf16")
    index, hidden = torch.zeros(4, dtype=torch.int32, device="cuda"), torch.zeros(4, 8, device="cuda")
    y, dy = torch.zeros(4, 24, dtype=torch.bfloat16, device="cuda"), torch.zeros(4, 24, dtype=torch.bfloat16, device="cuda")

    def f(x=x, index=index, a=a, b=b, **more):
        return lambda: capi.linear_adapters(x, index, a, b, **more)

    def g(dy=dy, hidden=hidden, **more):
        return lambda: capi.linear_adapters_backward(dy, x, index, a, b, None, hidden, **more)

    for call in (f(index=index.long()), f(a=a.float()), f(b=b.half()), f(scale=torch.ones(2, dtype=torch.bfloat16, device="cuda")),
                 f(base=y.float()), f(x=x.double()), f(index=None), g(hidden=None), g(dy=dy.float()), g(dx=x.float())):
        with pytest.raises(TypeError):
            call()
    big = torch.zeros(2, 129, 16, dtype=torch.bfloat16, device="cuda"), torch.zeros(2, 24, 129, dtype=torch.bfloat16, device="cuda")
    for call in (f(index=index[:3]), f(index=index.cpu()), f(a=a[:1]), f(a=a[..., :8]), f(b=b[..., :4]), f(b=b.transpose(1, 2)),
                 f(scale=torch.ones(3, device="cuda")), f(base=y[:, :23]), f(y=y[:3]), f(x=x.cpu()), f(a=big[0], b=big[1]),
                 f(a=a[:0], b=b[:0]), f(y=y[:1].expand(4, 24)), g(hidden=hidden[:3]), g(dy=dy[:, :8]), g(base=x[:3])):
        with pytest.raises((ValueError, RuntimeError)):
            call()
    assert capi.linear_adapters(x[:0], index[:0], a, b).shape == (0, 24)
    dx, da, db = capi.linear_adapters_backward(dy[:0], x[:0], index[:0], a, b, None, hidden[:0])
    assert dx.shape == (0, 16) and (da == 0).all() and (db == 0).all()
