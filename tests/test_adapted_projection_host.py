"""Which stream the parts of a projection with adapters run on, without a GPU: every call and every cast of PyTorch's
between them is made where the caller's stream is the current one, or given."""
import contextlib

import pytest
import torch


class Stream:
    """Of another library: a handle alone."""
    cuda_stream = 1234


class Weights:
    def __init__(self, seen):
        self.seen = seen

    def to(self, dtype):
        self.seen("cast")
        return self


@pytest.mark.parametrize("stream,want", [(None, None), (Stream(), 1234), (5678, 5678), (0, "default"), (1, "default")])
def test_every_part_runs_on_the_calls_stream(monkeypatch, stream, want):
    from conv2d_batchnorm_silu_gb300 import _build
    _build.build()
    from conv2d_batchnorm_silu_gb300 import capi, token_block
    current, log = [None], []

    @contextlib.contextmanager
    def as_current(s):
        before = current[0]
        current[0] = before if s is None else s
        yield
        current[0] = before

    def seen(what, stream=None):
        log.append((what, current[0] if stream is None else capi._stream_handle(stream)))

    monkeypatch.setattr(torch.cuda, "stream", as_current)
    monkeypatch.setattr(torch.cuda, "ExternalStream", lambda handle: handle)
    monkeypatch.setattr(torch.cuda, "default_stream", lambda device=None: "default")
    monkeypatch.setattr(capi, "rms_norm_quantize", lambda *a, stream=None, **k: (seen("norm", stream), (None,) * 4)[1])
    monkeypatch.setattr(capi, "linear_int8", lambda *a, stream=None, **k: seen("projection", stream))
    monkeypatch.setattr(capi, "linear_adapters", lambda *a, stream=None, **k: seen("adapters", stream))
    block = object.__new__(token_block.AdaptedProjection)
    block.gamma = block.bias = block.scale = block.w = block.w_scale = None
    block.eps, block.a, block.b = 1e-6, Weights(seen), Weights(seen)
    block(torch.zeros(2, 4, dtype=torch.bfloat16), None, None, stream=stream)
    assert [what for what, _ in log] == ["norm", "projection", "cast", "cast", "adapters"]
    assert {at for _, at in log} == {want}, log
