"""AdamW in 8 bits with its step on the device: the bits of calls whose step counts on the host, eager and replayed from a graph."""
import warnings

import pytest

from test_gpu_block import state_values
from test_gpu_layer import gen_for, normal, ops, torch  # noqa: F401 (fixtures)

pytestmark = pytest.mark.gpu

SIZES = [1, 31, 33, 4096, 4097, 20_000] + [5, 300, 64] * 20    # two launches


def tensors(torch, ops, dt):
    gen = gen_for(torch, 51)
    ps = [normal(torch, gen, n).to(dt) for n in SIZES]
    gs = [(1e-2 * normal(torch, gen, n)).to(dt) for n in SIZES]
    return ps, gs, [ops.adamw8_state(p) for p in ps]


def same(torch, a, b):
    return all(torch.equal(p, q) for p, q in zip(a[0], b[0])) and all(
        torch.equal(x.view(torch.uint8), y.view(torch.uint8)) for s, t in zip(a[2], b[2]) for x, y in zip(s, t))


@pytest.mark.parametrize("dtype", ["bfloat16", "float16", "float32"])
@pytest.mark.parametrize("correct", [False, True])
def test_a_step_on_the_device_is_the_step_on_the_host(torch, ops, dtype, correct):
    one, two = (tensors(torch, ops, getattr(torch, dtype)) for _ in range(2))
    at = torch.zeros(3, dtype=torch.int64, device="cuda")
    hp = dict(lr=1e-2, beta1=0.9, beta2=0.999, bias_correction=correct, seed=2 ** 63 + 12345)
    for step in (1, 2, 3, 100, 12_345, 10 ** 6, 2 ** 31 - 1):
        at[1] = step
        ops.adamw8_step(*one, step=step, **hp)
        ops.adamw8_step(*two, step=at[1:2], **hp)
        assert same(torch, one, two), step
    assert at.tolist() == [0, 2 ** 31 - 1, 0]                 # read, not written
    # out of range: the nearest step
    for given, meant in ((0, 1), (-5, 1), (-2 ** 63, 1), (2 ** 31, 2 ** 31 - 1), (2 ** 62, 2 ** 31 - 1)):
        at[1] = given
        ops.adamw8_step(*one, step=meant, **hp)
        ops.adamw8_step(*two, step=at[1], **hp)
        assert same(torch, one, two), given


@pytest.mark.parametrize("dtype", ["bfloat16", "float32"])
def test_replays_count_on(torch, ops, dtype):
    """A graph that advances the step: six replays leave the bits of eager calls with steps 1 to 6, bias corrections among them."""
    one, two = (tensors(torch, ops, getattr(torch, dtype)) for _ in range(2))
    hp = dict(lr=1e-2, bias_correction=True, seed=7)
    step = torch.zeros((), dtype=torch.int64, device="cuda")
    ops.adamw8_step(*tensors(torch, ops, getattr(torch, dtype)), step=1, **hp)
    graph = torch.cuda.CUDAGraph()
    with warnings.catch_warnings():
        warnings.simplefilter("error")
        with torch.cuda.graph(graph):
            step.add_(1)
            ops.hybrid_step([], [(p, g, s) for p, g, s in zip(*two)], muon={}, adamw=dict(lr=1e-2, step=step, bias_correction=True), seed=7)
    for i in range(1, 7):
        graph.replay()
        torch.cuda.synchronize()
        ops.adamw8_step(*one, step=i, **hp)
        assert same(torch, one, two), i
    assert int(step) == 6


def test_roots_decay_in_replays(torch, ops):
    """Without gradients the mean root falls by sqrt(beta2) a replay, also where a step's change is 1/250 of a code's: with the same random
    numbers in every replay 99 % of the elements would never move."""
    n = 1 << 18
    p, g = torch.zeros(n, device="cuda"), torch.full((n,), 0.37, device="cuda")
    state = ops.adamw8_state(p)
    step = torch.ones(1, dtype=torch.int64, device="cuda")
    ops.adamw8_step([p], [g], [state], lr=1e-3, beta2=0.999, step=step, seed=5)
    g.zero_()
    root = lambda: float(state_values(torch, state[2], state[3]).mean())
    first = root()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step.add_(1)
        ops.adamw8_step([p], [g], [state], lr=1e-3, beta2=0.999, step=step, seed=5)
    for _ in range(3000):
        graph.replay()
    torch.cuda.synchronize()
    # each of 3000 roundings moves a root by at most 1/8 of itself with a chance of 1/250 and the mean of 2^18 by a 512th of such a step:
    # sqrt(3000 / 250) / 8 / 512 = 1e-3 of it
    assert abs(root() / first / 0.999 ** 1500 - 1) < 6e-3


def test_a_captured_step_of_the_host_warns(torch, ops):
    ps, gs, ss = tensors(torch, ops, torch.bfloat16)
    graph = torch.cuda.CUDAGraph()
    with pytest.warns(UserWarning, match="every replay uses again"):
        with torch.cuda.graph(graph):
            ops.adamw8_step(ps, gs, ss, lr=1e-3, step=3)


def test_steps_of_several_streams(torch, ops):
    """Two streams, a step of their own each, more than once."""
    sets = [tensors(torch, ops, torch.bfloat16) for _ in range(4)]
    hp = dict(lr=1e-2, bias_correction=True, seed=1)
    streams = [torch.cuda.Stream() for _ in range(2)]
    steps = [torch.zeros(1, dtype=torch.int64, device="cuda") for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(4):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                steps[i].add_(1 + i)
                ops.adamw8_step(*sets[i], step=steps[i], **hp)
    torch.cuda.synchronize()
    for k in range(4):
        for i in range(2):
            ops.adamw8_step(*sets[2 + i], step=(k + 1) * (1 + i), **hp)
    assert same(torch, sets[0], sets[2]) and same(torch, sets[1], sets[3])
