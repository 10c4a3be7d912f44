"""What the compiled calls of the token-wise operators raise, and the streams that they take."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def capi():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from conv2d_batchnorm_silu_gb300 import capi
    return capi


def test_out_of_memory_is_pytorchs_own_error(capi):
    # One row broadcast to 2^18: an output of a terabyte, which the process's share refuses without asking the driver.
    x = torch.zeros(1, 1 << 20, device="cuda").expand(1 << 18, 1 << 20)
    a, w = torch.zeros(1, 16, dtype=torch.int8, device="cuda"), torch.zeros(1 << 18, 16, dtype=torch.int8, device="cuda")
    ones = torch.ones(1, device="cuda").expand(1 << 20).contiguous()
    _, stats = capi.layer_norm(x[:1], return_stats=True)
    stats = stats[:, :1].expand(2, 1 << 18).contiguous()
    torch.cuda.set_per_process_memory_fraction(0.5)
    try:
        for call in (lambda: capi.layer_norm(x), lambda: capi.layer_norm_backward(x, x, None, stats),
                     lambda: capi.quantize_rows(x.expand(1 << 18, 1 << 20)), lambda: capi.layer_norm_quantize(x),
                     lambda: capi.linear_int8(a.expand(1 << 20, 16), w, ones, ones[: 1 << 18].contiguous())):
            with pytest.raises(torch.OutOfMemoryError, match="out of memory"):
                call()
    finally:
        torch.cuda.set_per_process_memory_fraction(1.0)
    assert not capi.layer_norm(x[:3]).any()  # and the calls go on


def test_an_argument_without_a_truth_value(capi):
    class Neither:
        def __bool__(self):
            raise KeyError("neither")

    with pytest.raises(KeyError, match="neither"):
        capi.layer_norm(torch.zeros(2, 8, device="cuda"), return_stats=Neither())


def test_streams_by_handle(capi):
    # The default stream, the runtime's two names for it, and a stream of one's own, each alone and in PyTorch's class.
    x = torch.randn(300, 64, device="cuda").bfloat16()
    w, scale = torch.randint(-9, 9, (32, 64), dtype=torch.int8, device="cuda"), torch.rand(32, device="cuda")

    def block(stream):
        y, stats = capi.layer_norm(x, return_stats=True, stream=stream)
        q, rows = capi.layer_norm_quantize(x, stream=stream)
        return (y, *capi.layer_norm_backward(y, x, None, stats, stream=stream), *capi.quantize_rows(x, stream=stream),
                capi.linear_int8(q, w, rows, scale, stream=stream))

    want = block(None)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for stream in (0, 1, 2, side, side.cuda_stream, torch.cuda.ExternalStream(side.cuda_stream)):
        got = block(stream)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(want, got)), stream
        assert torch.cuda.current_stream() == torch.cuda.default_stream()
    with pytest.raises(TypeError):
        capi.layer_norm(x, stream=object())
