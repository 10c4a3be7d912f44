"""The projection with adapters on a stream that the caller gives, while PyTorch's current stream has work of its own."""
import pytest
import torch

pytestmark = pytest.mark.gpu


def rand(seed, *shape):
    return torch.randn(*shape, generator=torch.Generator().manual_seed(seed)).cuda()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("rows", [5, 2000])
def test_a_given_stream_gives_the_same_bits(rows, dtype):
    from conv2d_batchnorm_silu_gb300.token_block import AdaptedProjection
    c, n, rank, adapters = 256, 512, 16, 24
    block = AdaptedProjection(1 + 0.1 * rand(1, c), rand(2, n, c) / c ** 0.5, 0.1 * rand(3, n), rand(4, adapters, rank, c) / c ** 0.5,
                              0.3 * rand(5, adapters, n, rank))
    h, residual = rand(7, rows, c).to(dtype), rand(8, rows, c).to(dtype)
    index = torch.randint(-1, adapters, (rows,), generator=torch.Generator().manual_seed(9)).int().cuda()
    want, want_total = block(h, residual, index)
    busy = rand(10, 4096, 4096)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for given in (side, side.cuda_stream):
        out = []
        for _ in range(3):
            for _ in range(8):
                busy = busy @ busy / 64  # the current stream is some milliseconds behind
            out.append(block(h, residual, index, stream=given))
            torch.empty(adapters, n, rank, dtype=dtype, device="cuda").fill_(float("nan"))  # memory that the call gave back, if it was this stream's
        side.synchronize()
        for z, total in out:
            assert torch.equal(z, want) and torch.equal(total, want_total)
        torch.cuda.synchronize()
    for default in (0, 1):
        z, total = block(h, residual, index, stream=default)
        torch.cuda.synchronize()
        assert torch.equal(z, want) and torch.equal(total, want_total)
