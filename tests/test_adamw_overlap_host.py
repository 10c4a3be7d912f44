"""Tensors of an AdamW step that share memory, without a GPU: the C entry refuses what two blocks would write, or one
write and another read, before any CUDA call, and nothing else for its place in memory."""
import ctypes
import random

import pytest

KINDS = ("param", "exp_avg", "exp_avg_sq", "exp_avg_scale", "exp_avg_sq_scale")
N = 600  # elements a tensor


@pytest.fixture(scope="module")
def capi():
    from conv2d_batchnorm_silu_gb300 import _build
    _build.build()
    from conv2d_batchnorm_silu_gb300 import capi
    return capi


def step(capi, tensors, bits=8, **options):
    """The status of a call on stand-ins for device pointers: one that is not refused fails at its first CUDA call, as
    there is no device."""
    table = (capi.AdamWTensor * len(tensors))(*(capi.AdamWTensor(n=N, param_dtype=0, grad_dtype=0, **t) for t in tensors))
    o = capi.AdamWOptions(lr=1e-3, beta1=0.9, beta2=0.999, eps=1e-8, grad_scale=1.0, step=1, state_bits=bits)
    for name, value in options.items():
        setattr(o, name, value)
    return capi.raw_status("conv_bn_silu_adamw_step", table, len(tensors), ctypes.byref(o), None)


def laid_out(count, order=None):
    """`count` tensors, each part 4096 bytes from the next; order: the parts' places in memory."""
    places = list(range(count * 6))
    if order:
        order.shuffle(places)
    at = iter(places)
    return [{name: (1 << 20) + 4096 * next(at) for name in KINDS + ("grad",)} for _ in range(count)]


@pytest.fixture(autouse=True)
def no_device():
    import torch
    if torch.cuda.is_available():
        pytest.skip("stand-in pointers: only where no device would follow them")


@pytest.mark.parametrize("shuffled", [False, True])
def test_what_is_apart_is_not_refused(capi, shuffled):
    for count in (1, 3, 40):
        tensors = laid_out(count, random.Random(count) if shuffled else None)
        assert step(capi, tensors) == capi.CBS_ERR_CUDA
        for t in tensors:  # float32 scales of 600 elements: 12 bytes; the moments' end touches the next
            t["exp_avg_sq"] = t["exp_avg"] + N
        assert step(capi, tensors) == capi.CBS_ERR_CUDA
        for t in tensors[1:]:
            t["grad"] = tensors[0]["grad"] + 400  # gradients may share memory
        assert step(capi, tensors) == capi.CBS_ERR_CUDA


@pytest.mark.parametrize("shuffled", [False, True])
@pytest.mark.parametrize("first", KINDS)
def test_what_is_written_twice_is_refused(capi, first, shuffled):
    size = {"param": 4 * N, "exp_avg": N, "exp_avg_sq": N, "exp_avg_scale": 12, "exp_avg_sq_scale": 12}
    for second in KINDS + ("grad",):
        for i, j in ((0, 1), (7, 3), (9, 9), (0, 9)):
            if i == j and first == second:
                continue
            for back in (0, size[first] - 4):
                tensors = laid_out(10, random.Random(i) if shuffled else None)
                tensors[j][second] = tensors[i][first] + back
                assert step(capi, tensors) == capi.CBS_ERR_INVALID_ARG, (second, i, j, back)


def test_numbers_among_what_is_written_are_refused(capi):
    tensors = laid_out(3)
    for name, bytes_ in (("lr_device", 4), ("grad_scale_device", 4), ("step_device", 8)):
        assert step(capi, tensors, **{name: tensors[2]["exp_avg"] + 8}) == capi.CBS_ERR_INVALID_ARG
        assert step(capi, tensors, **{name: tensors[2]["param"] + 4 * N - bytes_}) == capi.CBS_ERR_INVALID_ARG
        assert step(capi, tensors, **{name: 1 << 30}) == capi.CBS_ERR_CUDA


def test_moments_of_32_bits(capi):
    tensors = laid_out(4)
    for t in tensors:
        t["exp_avg_scale"] = t["exp_avg_sq_scale"] = None
    assert step(capi, tensors, 32) == capi.CBS_ERR_CUDA
    tensors[1]["exp_avg"] = tensors[0]["exp_avg"] + 4 * N - 4
    assert step(capi, tensors, 32) == capi.CBS_ERR_INVALID_ARG
