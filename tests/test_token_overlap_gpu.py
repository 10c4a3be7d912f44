"""Calls back to back, each of whose kernels may start while the one before still runs: scales and parameters that are
written right before the layer that reads them, at the same addresses every time."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def capi():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from conv2d_batchnorm_silu_gb300 import capi
    return capi


@pytest.mark.parametrize("m,n,k", [(6, 300, 512), (24, 300, 64), (20, 300, 4096), (64, 1024, 1024), (300, 300, 4096),
                                   (1500, 9, 4096), (700, 1300, 400), (100, 712, 2051)])
def test_scales_written_right_before(capi, m, n, k):
    g = torch.Generator(device="cuda").manual_seed(1)
    xs = [torch.randn(m, k, generator=g, device="cuda") * 4.0 ** (i % 5) for i in range(8)]
    ws = [torch.randn(n, k, generator=g, device="cuda") * 4.0 ** (i % 3) for i in range(8)]
    biases = [torch.randn(n, generator=g, device="cuda") for _ in range(8)]

    def layer(i, bias):
        q, scale = capi.quantize_rows(xs[i])
        w, w_scale = capi.quantize_rows(ws[(3 * i) % 8])
        bias.copy_(biases[i])
        return capi.linear_int8(q, w, scale, w_scale, bias, "silu", out_dtype=torch.float32)

    bias = torch.empty(n, device="cuda")
    want = []
    for i in range(8):
        want.append(layer(i, bias))
        torch.cuda.synchronize()
    for _ in range(20):
        got = [layer(i, bias) for i in range(8)]
        assert all(torch.equal(a, b) for a, b in zip(want, got))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = [layer(i, bias) for i in range(8)]
    for _ in range(20):
        graph.replay()
        assert all(torch.equal(a, b) for a, b in zip(want, got))
    capi.check()
