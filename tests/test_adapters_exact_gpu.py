"""Low-rank adapters on whole numbers, whose sums every part of the arithmetic holds exactly: outputs are the exact
result rounded once, bit by bit, in every kernel, so that no part of a row may be left out.

Magnitudes stay below 2^24 wherever fp32 adds; hidden rows take up to 15 bits, which two parts of bf16 (8 bits each) or
f16 (11) hold and one does not, and the rows of the weights' gradients 22 bits (bf16: three parts) or 20 (f16 and f32:
two 19-bit floats of 11 bits).  Random values then stay within what those parts keep."""
import numpy as np
import pytest
import torch

from oracle import token_ops as ref

pytestmark = pytest.mark.gpu

TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


@pytest.fixture(scope="module")
def capi():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from conv2d_batchnorm_silu_gb300 import capi
    return capi


def host(t):
    return t.detach().double().cpu().numpy()


def whole(rng, most, *shape):
    return rng.integers(-most, most + 1, shape).astype(np.float64)


def gpu(v, dtype):
    t = torch.from_numpy(np.asarray(v, np.float64)).to(TYPES[dtype]).cuda()
    assert (host(t) == v).all()  # what the type holds
    return t


def rounded(v, dtype):
    return host(torch.from_numpy(v).float().to(TYPES[dtype]))


# The kernels of up to 256 rows, of rows counted, of 16 ordered rows and of 128, for each number of ranks held; and rows,
# weights and ranks off their boundaries.
SIZES = [(1, 64, 48, 16, 2), (40, 64, 48, 8, 3), (200, 40, 64, 64, 2), (600, 64, 40, 16, 5), (700, 48, 33, 12, 90),
         (300, 32, 48, 16, 200), (900, 64, 40, 64, 2), (600, 33, 33, 100, 2), (2100, 64, 48, 16, 3), (1400, 48, 64, 32, 3),
         (1300, 64, 40, 64, 2), (1250, 40, 64, 128, 2), (2100, 33, 31, 13, 3), (1250, 31, 65, 50, 2), (1200, 33, 33, 100, 2)]


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("m,k,n,rank,adapters", SIZES)
def test_products_keep_hidden_rows_whole(capi, m, k, n, rank, adapters, dtype):
    """y = base + s B (A x) and dx likewise, base the nearest to minus the adapters' part: what is left of it shows a
    hidden row's low bits."""
    rng = np.random.default_rng(m + n)
    x, a, b = whole(rng, 16, m, k), whole(rng, 16, adapters, rank, k), whole(rng, 2, adapters, n, rank)
    index = rng.integers(-1, adapters, m)
    index[0] = 0
    scale = 2.0 ** rng.integers(-7, -5, adapters)
    part, hidden, total = ref.linear_adapters(x, index, a, b, scale)
    assert np.abs(hidden).max() < 2 ** 15 and (total / scale.min()).max() < 2 ** 24
    base = -rounded(part, dtype)
    at, s = torch.from_numpy(index.astype(np.int32)).cuda(), gpu(scale, "f32")
    args = at, gpu(a, dtype), gpu(b, dtype), s
    y, kept = capi.linear_adapters(gpu(x, dtype), *args, base=gpu(base, dtype), return_hidden=True)
    assert (host(kept) == hidden).all()
    assert (host(y) == rounded(part + base, dtype)).all()
    if dtype != "f32" and k > 40:  # one rounding of the hidden rows would show
        once, s_row = rounded(hidden, dtype), np.where(index >= 0, scale[index], 0.0)
        assert (s_row[:, None] * np.einsum("mnr,mr->mn", b[index], once - hidden) != 0).any() or dtype == "f16"

    dy, b = whole(rng, 16, m, n), whole(rng, 16, adapters, n, rank)
    a = whole(rng, 2, adapters, rank, k)
    (part, _, _), (total, _, _) = ref.linear_adapters_backward(dy, x, index, a, b, scale, hidden)
    assert (total / scale.min()).max() < 2 ** 24
    base = -rounded(part, dtype)
    dx, _, _ = capi.linear_adapters_backward(gpu(dy, dtype), gpu(x, dtype), at, gpu(a, dtype), gpu(b, dtype), s, kept,
                                             base=gpu(base, dtype))
    assert (host(dx) == rounded(part + base, dtype)).all()


GRADS = [(1, 64, 48, 16, 2), (20, 40, 64, 8, 8), (300, 64, 48, 64, 4), (500, 33, 31, 100, 3), (1100, 64, 72, 16, 3),
         (1300, 72, 40, 32, 2), (1500, 136, 64, 64, 2), (1200, 64, 64, 100, 2), (1100, 33, 72, 16, 40)]


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("m,k,n,rank,adapters", GRADS)
def test_weight_gradients_keep_hidden_rows_whole(capi, m, k, n, rank, adapters, dtype):
    """Two rows of each adapter carry the gradient, so that sums of rows that need all their bits stay exact."""
    rng = np.random.default_rng(m + n)
    bits = 22 if dtype == "bf16" else 20
    index = rng.integers(-1, adapters, m)
    carries = np.zeros(m, bool)
    for g in range(adapters):
        carries[np.flatnonzero(index == g)[-2:]] = True
    x, dy = whole(rng, 1, m, k) * carries[:, None], whole(rng, 1, m, n) * carries[:, None]
    hidden = whole(rng, 2 ** bits, m, rank)
    scale = 2.0 ** rng.integers(-1, 2, adapters)
    # dh = B^T dy of many bits too: two of B's columns far above the others.
    a, b = whole(rng, 2, adapters, rank, k), whole(rng, 1, adapters, n, rank)
    b[:, 1], b[:, 2] = 2.0 ** 8, 2.0 ** (bits - 6)
    (_, wa, wb), (_, ta, tb) = ref.linear_adapters_backward(dy, x, index, a, b, scale, hidden)
    assert max((ta / scale[:, None, None]).max(), (tb / scale[:, None, None]).max()) < 2 ** 24
    _, da, db = capi.linear_adapters_backward(gpu(dy, dtype), gpu(x, dtype), torch.from_numpy(index.astype(np.int32)).cuda(),
                                              gpu(a, dtype), gpu(b, dtype), gpu(scale, "f32"), gpu(hidden, "f32"))
    assert (host(da) == wa).all() and (host(db) == wb).all()


def sums(length):
    """Relative error, of the sum of the terms' magnitudes, of a sum of `length` products: a matrix instruction's
    additions may cut instead of round (two unit roundoffs each, 16 products an addition)."""
    return (length / 16 + 64) * 2.0 ** -23


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("m,k,n,rank,adapters", [(40, 96, 64, 16, 3), (600, 64, 96, 16, 5), (2100, 72, 64, 16, 3), (1300, 64, 56, 64, 2),
                                                 (1250, 33, 65, 100, 2)])
def test_random_values_stay_within_the_parts(capi, m, k, n, rank, adapters, dtype):
    """Two parts of bf16 keep 2^-16 of a hidden value, of f16 2^-22 and 2^-25 of the row's largest, two 19-bit floats of
    either operand 2^-21; three parts of bf16 2^-24.  Every output is rounded once beside."""
    rng = np.random.default_rng(m)
    draw = lambda *shape: torch.from_numpy(rng.normal(size=shape)).to(TYPES[dtype]).cuda()
    x, a, b, dy, base = draw(m, k), draw(adapters, rank, k) / 8, draw(adapters, n, rank), draw(m, n), draw(m, n)
    index = rng.integers(-1, adapters, m)
    scale = 0.5 + rng.random(adapters).astype(np.float32)
    at, s = torch.from_numpy(index.astype(np.int32)).cuda(), torch.from_numpy(scale).cuda()
    y, hidden = capi.linear_adapters(x, at, a, b, s, base=base, return_hidden=True)
    want, wh, total = ref.linear_adapters(host(x), index, host(a), host(b), scale, host(base))
    one = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8, "f16": 2.0 ** -11}[dtype] * 1.001 + 2.0 ** -23
    part = {"f32": 2.0 ** -21, "bf16": 2.0 ** -16, "f16": 2.0 ** -22}[dtype] * 1.01
    first = 2.0 ** -21 if dtype == "f32" else 0.0
    row_scale = np.where(index >= 0, scale[index], 0.0)[:, None]

    def bound(want, total, h, w2, length):
        off = total * (sums(length) + sums(rank) + first + 2.0 ** -22) + one * np.abs(want) + part * row_scale * np.einsum("mnr,mr->mn", np.abs(w2)[index], np.abs(h))
        if dtype == "f16":
            off = off + row_scale * np.abs(w2)[index].sum(2) * np.abs(h).max(1, keepdims=True) * 2.0 ** -25 + 2.0 ** -25
        return off

    assert (np.abs(host(y) - want) <= bound(want, total, wh, host(b), k)).all()
    dx, da, db = capi.linear_adapters_backward(dy, x, at, a, b, s, hidden)
    (wx, wa, wb), (tx, ta, tb) = ref.linear_adapters_backward(host(dy), host(x), index, host(a), host(b), scale, host(hidden))
    dh = np.stack([host(b)[g].T @ host(dy)[i] if g >= 0 else np.zeros(rank) for i, g in enumerate(index)])
    assert (np.abs(host(dx) - wx) <= bound(wx, tx, dh, host(a).transpose(0, 2, 1), n)).all()
    kept = {"f32": 2.0 ** -21, "bf16": 2.0 ** -24, "f16": 2.0 ** -22}[dtype] + sums(m) + 2.0 ** -22
    assert (np.abs(host(da) - wa) <= ta * (kept + sums(n) + first)).all()
    assert (np.abs(host(db) - wb) <= tb * kept).all()
