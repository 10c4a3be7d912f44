"""The workspaces of the low-rank adapters: what their sizes need and no more, and nothing written beyond."""
import pytest
import torch

pytestmark = pytest.mark.gpu

TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


@pytest.fixture(scope="module")
def capi():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from conv2d_batchnorm_silu_gb300 import capi
    return capi


@pytest.mark.parametrize("m,k,n,rank,adapters", [(1000, 64, 64, 64, 4096), (1 << 20, 64, 72, 100, 4096), (1 << 20, 63, 72, 64, 4000),
                                                 (100000, 64, 64, 64, 2000)])
def test_gradients_that_no_tensor_map_serves_reserve_no_operands(capi, m, k, n, rank, adapters):
    """Rows by adapter, their tiles, the hidden gradient and two partial sums a chunk: at most 456 chunks of CTAs, or one for
    1024 rows.  The operands of 64-row steps, 24 KB each at rank 64, are for sizes that such a kernel takes."""
    need = capi.raw_status("conv_bn_silu_linear_adapters_backward_workspace", m, k, n, rank, adapters)
    rows = 4 * m + m + 40 * (adapters + 2) + 4 * m * rank + 4096
    assert 0 < need <= rows + 8 * max(456, m // 1024 + 1) * rank * (k + n)


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("m,k,n,rank,adapters", [(3, 16, 24, 8, 2), (18, 40, 32, 16, 8), (300, 33, 40, 12, 70), (1000, 32, 32, 64, 300),
                                                 (1100, 64, 72, 16, 3), (1500, 33, 40, 64, 2), (1300, 64, 64, 128, 2), (2100, 48, 56, 16, 700)])
def test_nothing_is_written_beyond(capi, m, k, n, rank, adapters, dtype):
    gen = torch.Generator("cuda").manual_seed(m)
    draw = lambda *shape: torch.randn(*shape, generator=gen, device="cuda").to(TYPES[dtype])
    x, dy, a, b = draw(m, k), draw(m, n), draw(adapters, rank, k), draw(adapters, n, rank)
    index = torch.randint(-1, adapters, (m,), generator=gen, device="cuda", dtype=torch.int32)
    y, hidden = capi.linear_adapters(x, index, a, b, return_hidden=True)
    want = capi.linear_adapters_backward(dy, x, index, a, b, None, hidden)
    number = list(TYPES).index(dtype)
    sizes = m, k, n, rank, adapters
    stream = torch.cuda.current_stream().cuda_stream

    def work(need):
        t = torch.full((need + 4096,), 77, dtype=torch.uint8, device="cuda")
        return t, t.data_ptr() if need else None, need

    t, at, need = work(capi.raw_status("conv_bn_silu_linear_adapters_workspace", *sizes))
    y2 = torch.empty_like(y)
    assert capi.raw_status("conv_bn_silu_linear_adapters", x.data_ptr(), k, index.data_ptr(), a.data_ptr(), b.data_ptr(), None, None, 0,
                           y2.data_ptr(), n, None, *sizes, number, at, need, stream) == capi.CBS_OK
    assert torch.equal(y2, y) and (t[need:] == 77).all()
    t, at, need = work(capi.raw_status("conv_bn_silu_linear_adapters_backward_workspace", *sizes))
    dx, da, db = (torch.empty_like(w) for w in want)

    def call(bytes_):
        return capi.raw_status("conv_bn_silu_linear_adapters_backward", dy.data_ptr(), n, x.data_ptr(), k, index.data_ptr(), a.data_ptr(),
                               b.data_ptr(), None, hidden.data_ptr(), None, 0, dx.data_ptr(), k, da.data_ptr(), db.data_ptr(), *sizes,
                               number, at, bytes_, stream)

    assert call(need - 1) == capi.CBS_ERR_INVALID_ARG and call(need) == capi.CBS_OK
    assert torch.equal(dx, want[0]) and torch.equal(da, want[1]) and torch.equal(db, want[2]) and (t[need:] == 77).all()
