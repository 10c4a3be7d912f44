"""Rows so far apart that their offsets leave 32 bits: the same results as for the same rows side by side."""
import pytest
import torch

pytestmark = pytest.mark.gpu

FAR = 1 << 24  # elements from row to row: 300 rows reach 5e9


@pytest.fixture(scope="module")
def capi():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from conv2d_batchnorm_silu_gb300 import capi
    yield capi
    torch.cuda.empty_cache()  # some 60 GB


def far(like):
    store = torch.empty(like.shape[0] * FAR, dtype=like.dtype, device="cuda")
    return store.as_strided(like.shape, (FAR, 1)).copy_(like)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("c", [256, 777])
def test_norm(capi, c, dtype):
    x, dy = torch.randn(300, c, device="cuda").to(dtype), torch.randn(300, c, device="cuda").to(dtype)
    gamma, beta = torch.rand(c, device="cuda"), torch.rand(c, device="cuda")
    y, stats = capi.layer_norm(x, gamma, beta, return_stats=True)
    grads = capi.layer_norm_backward(dy, x, gamma, stats)
    q, scale = capi.layer_norm_quantize(x, gamma, beta)
    x, dy, out = far(x), far(dy), far(torch.zeros_like(x))
    assert torch.equal(capi.layer_norm(x, gamma, beta, y=out), y)
    assert all(torch.equal(a, b) for a, b in zip(capi.layer_norm_backward(dy, x, gamma, stats, dx=out), grads))
    del dy, out
    got = capi.layer_norm_quantize(x, gamma, beta, q=far(torch.zeros_like(q)))
    assert torch.equal(got[0], q) and torch.equal(got[1], scale)


# A size for each kernel; weights, rows, residual and output all far apart.
@pytest.mark.parametrize("m,n,k", [(8, 300, 512), (24, 300, 64), (40, 300, 2048), (300, 300, 4096), (300, 9, 4096), (300, 280, 3333),
                                   (300, 300, 512)])
def test_linear(capi, m, n, k):
    a = torch.randint(-128, 128, (m, k), dtype=torch.int8, device="cuda")
    w = torch.randint(-128, 128, (n, k), dtype=torch.int8, device="cuda")
    sa, sw, res = torch.rand(m, device="cuda"), torch.rand(n, device="cuda"), torch.randn(m, n, device="cuda").bfloat16()
    # The kernel goes by alignment, which FAR keeps.
    want = capi.linear_int8(a, w, sa, sw, residual=res) if k % 16 == 0 else None
    fa, fw, fres, y = far(a), far(w), far(res), far(torch.zeros_like(res))
    got = capi.linear_int8(fa, fw, sa, sw, residual=fres, y=y)
    if want is None:
        pad = torch.zeros(m, (k + 15) // 16 * 16, dtype=torch.int8, device="cuda")
        want = capi.linear_int8(pad[:, :k].copy_(a), pad.new_zeros(n, pad.shape[1])[:, :k].copy_(w), sa, sw, residual=res)
    assert torch.equal(got, want)
    capi.check()
