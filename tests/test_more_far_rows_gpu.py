"""The RMS norm, its gradient, the adapters and the AdamW step on rows and elements whose offsets leave 32 bits: the same
bits as on rows that lie together."""
import pytest
import torch

pytestmark = pytest.mark.gpu
FAR = (1 << 31) + 64  # elements between two rows


@pytest.fixture(scope="module")
def capi():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from conv2d_batchnorm_silu_gb300 import capi
    yield capi
    torch.cuda.empty_cache()


@pytest.fixture(scope="module")
def memory(capi):
    return torch.empty(2 * FAR + (1 << 20), dtype=torch.bfloat16, device="cuda")


def far(memory, rows, at=0):
    """A copy of rows [3][c] in memory, FAR elements apart, from `at` on."""
    view = memory.as_strided((3, rows.shape[1]), (FAR, 1), at)
    view.copy_(rows)
    return view


def rand(seed, *shape):
    return torch.randn(*shape, generator=torch.Generator().manual_seed(seed)).cuda()


@pytest.mark.parametrize("c", [96, 1001, 4096, 20000])
def test_norm(capi, memory, c):
    x, residual, gamma = rand(1, 3, c).bfloat16(), rand(2, 3, c).bfloat16(), 0.5 + rand(3, c).abs()
    y, total, rstd = capi.rms_norm(x, gamma, residual=residual, return_rstd=True)
    dx, dgamma = capi.rms_norm_backward(residual, total, gamma, rstd, residual=x)
    places = [far(memory, t, 32768 * i) for i, t in enumerate((x, residual, x, x, x))]
    y2, total2, rstd2 = capi.rms_norm(places[0], gamma, residual=places[1], return_rstd=True, y=places[2], total=places[3])
    assert torch.equal(y2, y) and torch.equal(total2, total) and torch.equal(rstd2, rstd)
    dx2, dgamma2 = capi.rms_norm_backward(places[1], total2, gamma, rstd2, residual=places[0], dx=places[4])
    assert torch.equal(dx2, dx) and torch.equal(dgamma2, dgamma)


@pytest.mark.parametrize("c,n", [(96, 64), (101, 77)])
def test_adapters(capi, memory, c, n):
    x, base, a, b = rand(1, 3, c).bfloat16(), rand(2, 3, n).bfloat16(), rand(3, 2, 16, c).bfloat16(), rand(4, 2, n, 16).bfloat16()
    index = torch.tensor([1, -1, 0], dtype=torch.int32, device="cuda")
    y, hidden = capi.linear_adapters(x, index, a, b, base=base, return_hidden=True)
    grads = capi.linear_adapters_backward(y, x, index, a, b, None, hidden, base=x)
    at = [far(memory, t, 32768 * i) for i, t in enumerate((x, base, base, x))]
    y2, hidden2 = capi.linear_adapters(at[0], index, a, b, base=at[1], return_hidden=True, y=at[2])
    assert torch.equal(y2, y) and torch.equal(hidden2, hidden)
    for got, want in zip(capi.linear_adapters_backward(at[2], at[0], index, a, b, None, hidden, base=at[0], dx=at[3]), grads):
        assert torch.equal(got, want)


@pytest.mark.parametrize("c,n", [(64, 4096), (4096, 64)])
def test_adapters_of_many_rows(capi, memory, c, n):
    """A million rows: y of 2^32 elements (or x), through the kernels of many rows and the weights' gradients; a part of
    them on its own gives the same rows."""
    rows = 1 << 20
    wide = memory.as_strided((rows, 4096), (4096, 1), 0)
    narrow = rand(1, 4096, 64).bfloat16().repeat(rows // 4096, 1)
    wide.view(rows // 4096, 4096, 4096).copy_((rand(2, 4096, 4096) * 0.05).bfloat16())
    a, b = (rand(3, 2, 16, c) * c ** -0.5).bfloat16(), rand(4, 2, n, 16).bfloat16()
    index = torch.arange(rows, device="cuda").div(rows // 4, rounding_mode="floor").remainder(2).int()
    if n == 4096:
        y = capi.linear_adapters(narrow, index, a, b, base=wide, y=wide)
        first = capi.linear_adapters(narrow[:8192], index[:8192], a, b, base=(rand(2, 4096, 4096) * 0.05).bfloat16().repeat(2, 1))
        assert torch.equal(y[:8192], first) and torch.equal(y[rows // 2: rows // 2 + 8192], first)
        assert torch.equal(y[rows // 4: rows // 4 + 4096], y[-4096:])
    else:
        y, hidden = capi.linear_adapters(wide, index, a, b, return_hidden=True)
        assert torch.equal(y[:4096], y[rows // 2: rows // 2 + 4096]) and torch.equal(y[-4096:], y[rows // 4: rows // 4 + 4096])
        dy = rand(5, 4096, 64).bfloat16().repeat(rows // 4096, 1)
        _, da, db = capi.linear_adapters_backward(dy, wide, index, a, b, None, hidden)
        # rows repeat 4096 by 4096: the sums over them, 128 times for each adapter
        part = torch.einsum("mn,mr->nr", dy[:4096].double(), hidden[:4096].double()) * (rows // 8192)
        assert (db[0].double() - part).abs().max() <= 2e-5 * part.abs().max()


def test_adamw_of_a_tensor_beyond_32_bits(capi, memory):
    n = (1 << 32) + 1000
    p = memory[:n]
    p.fill_(1.0)
    g, state = torch.zeros(n, dtype=torch.bfloat16, device="cuda"), capi.adamw_state([p], 8)
    g[-5:], g[:3] = 1.0, -1.0
    capi.adamw_step([p], [g], step=1, lr=0.25, weight_decay=0.0, **state)
    # the first step is lr times the sign of the gradient
    assert (p[-5:] == 0.75).all() and (p[:3] == 1.25).all() and (p[3:-5] == 1.0).all()
