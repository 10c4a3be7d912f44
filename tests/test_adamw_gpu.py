"""The AdamW step on the GPU against the 64-bit oracle, with moments in 32 and in 8 bits.  Bounds count
the fp32 roundings of each formula."""
import numpy as np
import pytest
import torch

from oracle import token_ops as ref

pytestmark = pytest.mark.gpu

TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
ROUND = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8, "f16": 2.0 ** -11}
LEAST = {"f32": 2.0 ** -149, "bf16": 2.0 ** -133, "f16": 2.0 ** -24}
E32 = 2.0 ** -24
RATES = dict(lr=3e-3, betas=(0.9, 0.999), eps=1e-8, weight_decay=0.02)


@pytest.fixture(scope="module")
def capi():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from conv2d_batchnorm_silu_gb300 import capi
    return capi


def host(t):
    return t.detach().double().cpu().numpy().reshape(-1)


def made(seed, n, dtype, size=1.0, offset=0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(n + offset, generator=g) * size).to(TYPES[dtype]).cuda()[offset:]


def check_step(before, g, m, v, after, step, dtype, grad_scale=1.0, rates=RATES):
    """p against the oracle's, from the moments in 64 bits (before the step); returns the new moments and bounds."""
    lr, (b1, b2), eps, decay = rates["lr"], rates["betas"], rates["eps"], rates["weight_decay"]
    p, m1, v1 = ref.adamw(before, g, m, v, step, lr, b1, b2, eps, decay, grad_scale)
    off_m = 6 * E32 * (b1 * np.abs(m) + (1 - b1) * np.abs(g * grad_scale)) + 2.0 ** -149
    c1, c2 = 1 - b1 ** step, 1 - b2 ** step
    denominator = np.sqrt(v1 / c2) + eps
    u = np.abs(m1) / c1 / denominator
    bound = lr * (off_m / c1 / denominator + u * 24 * E32) + 4 * E32 * np.abs(before) + (ROUND[dtype] * 1.001 + E32) * np.abs(p)
    assert (np.abs(host(after) - p) <= bound + LEAST[dtype]).all()
    return m1, v1, off_m


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("grad", list(TYPES))
def test_32_bit(capi, dtype, grad):
    sizes = [1, 7, 255, 256, 257, 4096, 4097, 10000, 0, 65536]
    p = [made(i, n, dtype) for i, n in enumerate(sizes)]
    g = [made(100 + i, n, grad, 0.1) for i, n in enumerate(sizes)]
    m, v = [made(200 + i, n, "f32", 0.05) for i, n in enumerate(sizes)], [made(300 + i, n, "f32", 0.1).square() for i, n in enumerate(sizes)]
    old = [[host(t) for t in ts] for ts in (p, g, m, v)]
    capi.adamw_step(p, g, m, v, step=7, grad_scale=0.25, **RATES)
    for i in range(len(sizes)):
        m1, v1, off = check_step(old[0][i], old[1][i], old[2][i], old[3][i], p[i], 7, dtype, 0.25)
        assert (np.abs(host(m[i]) - m1) <= off).all()
        assert (np.abs(host(v[i]) - v1) <= 8 * E32 * v1 + 2.0 ** -149).all()


def test_first_step_from_zero_and_odd_addresses(capi):
    for offset in (0, 1, 4, 8):
        p, g = [made(1, 3001, "bf16", offset=offset)], [made(2, 3001, "f32", 1e-3, offset=offset)]
        state = capi.adamw_state(p)
        before = host(p[0])
        capi.adamw_step(p, g, step=1, **RATES, **state)
        zero = np.zeros(3001)
        check_step(before, host(g[0]), zero, zero, p[0], 1, "bf16")


def values(state, i, block=256):
    """The moments that an 8-bit state holds, m and v's root, with their blocks' scales an element, in 64 bits."""
    out = []
    for name in ("exp_avg", "exp_avg_sq"):
        held, scale = host(state[name][i].float()), np.repeat(host(state[name + "_scale"][i]), block)
        out += [held * scale[:len(held)], scale[:len(held)]]
    return out


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("offset", [0, 3])
def test_8_bit(capi, dtype, offset):
    sizes = [1, 100, 256, 300, 4096, 5000, 70001]
    p = [made(i, n, dtype, offset=offset) for i, n in enumerate(sizes)]
    state = capi.adamw_state(p, bits=8)
    for step in range(1, 5):
        g = [made(10 * step + i, n, "f32", 0.1, offset) * torch.exp(2 * made(50 + i, n, "f32")) for i, n in enumerate(sizes)]
        before, held = [host(t) for t in p], [values(state, i) for i in range(len(sizes))]
        capi.adamw_step(p, g, step=step, **RATES, **state)
        for i, n in enumerate(sizes):
            m1, v1, off = check_step(before[i], host(g[i]), held[i][0], held[i][2] ** 2, p[i], step, dtype)
            um, uv = ref.dither(n, step)
            new = values(state, i)
            for got, scale, want, u, slack in ((new[0], new[1], m1, um, off), (new[2], new[3], np.sqrt(v1), uv, 8 * E32 * np.sqrt(v1))):
                pad = -n % 256
                most = np.abs(np.pad(want, (0, pad))).reshape(-1, 256).max(1)
                # a block's largest: within the error of its elements
                most_off = np.pad(slack, (0, pad)).reshape(-1, 256).max(1)
                scales = np.repeat(np.maximum(most, 2.0 ** -100) / 448, 256)[:n]
                assert (np.abs(scale - scales) <= np.repeat(most_off, 256)[:n] / 448 + 4 * E32 * scales).all()
                x = np.abs(want) / scales
                distance = ref.e4m3_distance(x)
                at = x / distance + u
                expected = np.minimum(np.floor(at) * distance, 448.0)
                if want is not m1:
                    expected = np.where((expected == 0) & (want > 0), 2.0 ** -9, expected)
                # The same value, but where the fp32 error of x, its own and its scale's, reaches the border between two.
                off_x = slack / scales + x * (np.repeat(most_off, 256)[:n] / 448 / scales + 8 * E32)
                near = np.abs(at - np.round(at)) <= off_x / distance + 2.0 ** -19
                near |= np.abs(np.log2(np.maximum(x, 2.0 ** -60)) - np.round(np.log2(np.maximum(x, 2.0 ** -60)))) < 1e-4
                same = np.abs(np.abs(got) / scale - expected) <= 1e-6 * expected
                assert (same | near).all() and near.mean() < 0.2
                assert (np.sign(got) == np.sign(want))[np.abs(got) > 0].all()


def test_8_bit_moments_follow_small_changes(capi):
    """A thousand steps without a gradient: v's root shrinks by 0.9995 each, far below half a step of the 8 bits.  Each
    step moves a value by its sixteenth to eighth with the odds of about 0.0005 * 16: some 2.7 moves, a spread of
    about 0.18 in the end, 0.003 for the mean of 4096 values."""
    p, g = [torch.zeros(4096, device="cuda")], [made(1, 4096, "f32")]
    state = capi.adamw_state(p, bits=8)
    capi.adamw_step(p, g, step=1, **RATES, **state)
    start = values(state, 0)
    zero = [torch.zeros(4096, device="cuda")]
    for step in range(2, 1002):
        capi.adamw_step(p, zero, step=step, **RATES, **state)
    end = values(state, 0)
    assert abs(end[2].mean() / start[2].mean() / 0.999 ** 500 - 1) < 0.02
    assert np.abs(end[0]).max() < 1e-6 * np.abs(start[0]).max() and p[0].isfinite().all()


def test_many_tensors(capi):
    """More than one launch holds, of mixed types and sizes; the same bits as each on its own."""
    for bits in (8, 32):
        kinds = list(TYPES)
        p = [made(i, 1 + 97 * i % 4500, kinds[i % 3]) for i in range(1000)]
        g = [made(2000 + i, 1 + 97 * i % 4500, kinds[i // 3 % 3], 0.1) for i in range(1000)]
        alone, state = [t.clone() for t in p], capi.adamw_state(p, bits)
        other = capi.adamw_state(p, bits)
        capi.adamw_step(p, g, step=3, **RATES, **state)
        for i in range(1000):
            capi.adamw_step([alone[i]], [g[i]], step=3, **RATES, **{name: [ts[i]] for name, ts in other.items()})
            assert torch.equal(alone[i], p[i])
            for name in state:
                assert torch.equal(state[name][i].view(torch.uint8), other[name][i].view(torch.uint8))


def test_numbers_on_the_device_and_graphs(capi):
    p, g = [made(1, 5000, "f32"), made(2, 300, "bf16")], [made(3, 5000, "f32", 0.1), made(4, 300, "bf16", 0.1)]
    for bits in (8, 32):
        start = [t.clone() for t in p]
        mine, theirs = [t.clone() for t in p], [t.clone() for t in p]
        state, state2 = capi.adamw_state(p, bits), capi.adamw_state(p, bits)
        step, lr = torch.ones(1, dtype=torch.int64, device="cuda"), torch.full((1,), 3e-3, device="cuda")
        scale = torch.full((), 0.5, device="cuda")
        graph = torch.cuda.CUDAGraph()
        rest = dict(betas=(0.9, 0.999), eps=1e-8, weight_decay=0.02)
        with torch.cuda.graph(graph):
            capi.adamw_step(mine, g, step=step, lr=lr, grad_scale=scale, **rest, **state)
            step.add_(1)
        for t in range(1, 40):
            lr.fill_(3e-3 / t)
            graph.replay()
            capi.adamw_step(theirs, g, step=t, lr=3e-3 / t, grad_scale=0.5, **rest, **state2)
        assert int(step) == 40
        # 39 steps of at most lr / t each, equal but for the roundings of 1 - beta^t and of p
        for a, b, s in zip(mine, theirs, start):
            moved = (b.double() - s.double()).abs().max()
            assert moved > 1e-3
            off = (a.double() - b.double()).abs().max()
            assert off <= (1e-4 if a.dtype == torch.float32 else 2.0 ** -6) * max(1.0, float(s.abs().max()))


def test_streams_and_poisoned_blocks(capi):
    p, g = [torch.zeros(1000, device="cuda")], [torch.ones(1000, device="cuda")]
    g[0][300], g[0][800] = float("nan"), float("inf")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    state = capi.adamw_state(p, bits=8)
    side.wait_stream(torch.cuda.current_stream())
    capi.adamw_step(p, g, step=1, stream=side, **RATES, **state)
    side.synchronize()
    bad = p[0].isnan()
    assert bad[300] and bad[800] and int(bad.sum()) == 2
    m = state["exp_avg"][0].float() * state["exp_avg_scale"][0].repeat_interleave(256)[:1000]
    assert m[256:512].isnan().all() and m[768:].isnan().all() and m[:256].isfinite().all() and m[512:768].isfinite().all()


def test_refusals(capi):
    p, g = [torch.zeros(64, device="cuda") for _ in range(2)], [torch.zeros(64, device="cuda") for _ in range(2)]
    state, state8 = capi.adamw_state(p), capi.adamw_state(p, 8)

    def step(p=p, g=g, state=state, step=1, lr=1e-3, **more):
        return lambda: capi.adamw_step(p, g, step=step, lr=lr, **{**state, **more})

    for call in (step(p=p[0]), step(g=[t.double() for t in g]), step(p=[p[0], None]), step(lr="fast"), step(step=1.5),
                 step(state={**state8, "exp_avg": state["exp_avg"]}), step(lr=torch.ones(1, dtype=torch.float64, device="cuda"))):
        with pytest.raises(TypeError):
            call()
    whole = torch.zeros(96, device="cuda")
    for call in (step(g=g[:1]), step(g=[g[0], g[1][:63]]), step(p=[p[0].cpu(), p[1]]), step(p=[torch.zeros(8, 16, device="cuda")[:, :8], p[1]]),
                 step(step=torch.ones(2, dtype=torch.int64, device="cuda")), step(step=torch.ones(1, dtype=torch.int64)),
                 step(state={**state8, "exp_avg_scale": [t[:0] for t in state8["exp_avg_scale"]]}), step(step=0),
                 step(betas=(1.0, 0.9)), step(eps=-1.0), step(lr=float("nan")), step(p=[p[0], p[0]]),
                 step(p=[whole[:64], whole[32:]])):
        with pytest.raises((ValueError, RuntimeError)):
            call()
    with pytest.raises(ValueError):
        capi.adamw_state(p, bits=16)
    capi.adamw_step([], [], [], [], step=1, lr=1e-3)
    for t in p:
        assert (t == 0).all()
