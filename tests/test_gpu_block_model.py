"""The operators together as a model's training step uses them: embedding, norms on a residual stream, gated experts, every
gradient, and the optimizer on all of them; against autograd in 64 bits, and replayed from a graph."""
import math

import pytest

from helpers import say
from test_gpu_layer import gen_for, normal, ops, torch  # noqa: F401 (fixtures)

pytestmark = pytest.mark.gpu


def inputs(torch, dt, tokens=200, vocab=97, k=4, experts=10, dim=256, inner=192):
    gen = gen_for(torch, 2)
    s = {"k": k, "experts": experts, "scale": math.sqrt(dim)}
    s["tokens"] = torch.randint(0, vocab, (tokens,), generator=gen, device="cuda")
    s["tokens"][-9:] = -1                                     # padding
    s["table"] = (normal(torch, gen, vocab, dim) * dim ** -0.5).to(dt)
    s["n1"], s["n2"] = ((1 + 0.1 * normal(torch, gen, dim)).to(dt) for _ in range(2))
    s["gate"], s["up"] = ((normal(torch, gen, experts, inner, dim) * dim ** -0.5).to(dt) for _ in range(2))
    s["down"] = (normal(torch, gen, experts, dim, inner) * inner ** -0.5).to(dt)
    s["c"] = normal(torch, gen, tokens, dim).to(dt)
    picks = torch.topk(normal(torch, gen, tokens, experts), k, dim=1)
    s["ids"], s["weights"] = picks.indices, torch.softmax(picks.values, dim=1)
    s["ids"][-9:] = -1
    return s


def step(ops, s):
    """The loss is sum(c y2); returns y2 and the gradients of every parameter and of the router's weights."""
    h0 = ops.embed(s["tokens"], s["table"], scale=s["scale"])
    y1, _, r1 = ops.rms_norm(h0, s["n1"], eps=1e-5)
    offsets, rank = ops.expert_sort(s["ids"], s["experts"])
    xs = ops.expert_dispatch(y1, rank, offsets)
    act, gate, up = ops.expert_gated(xs, s["gate"], s["up"], offsets, keep=True)
    ys = ops.expert_matmul(act, s["down"], offsets)
    out = ops.expert_combine(ys, s["weights"], rank)
    y2, h1, r2 = ops.rms_norm(out, s["n2"], residual=h0, eps=1e-5)
    dh1, dn2 = ops.rms_norm_backward(s["c"], h1, r2, s["n2"])
    dys, dweights = ops.expert_combine_backward(dh1, ys, s["weights"], rank, offsets)
    dact, ddown = ops.expert_matmul_backward(dys, act, s["down"], offsets)
    dxs, dgate, dup = ops.expert_gated_backward(dact, xs, s["gate"], s["up"], gate, up, offsets)
    dy1 = ops.expert_dispatch_backward(dxs, rank)
    dh0, dn1 = ops.rms_norm_backward(dy1, h0, r1, s["n1"], dh=dh1)
    dtable = ops.embed_backward(dh0, s["tokens"], s["table"].shape[0], scale=s["scale"])
    return {"y": y2, "weights": dweights, "down": ddown, "gate": dgate, "up": dup, "n1": dn1, "n2": dn2, "table": dtable}


def test_the_step_against_autograd_in_64_bits(torch, ops):
    s = inputs(torch, torch.float32)
    got = step(ops, s)
    leaf = {n: s[n].double().cpu().requires_grad_() for n in ("table", "n1", "n2", "gate", "up", "down", "weights")}
    norm = lambda h, w: h * (h.square().mean(dim=1, keepdim=True) + 1e-5).rsqrt() * w
    tokens = s["tokens"].cpu()
    h0 = torch.where((tokens >= 0)[:, None], leaf["table"][tokens.clamp(min=0)] * float(torch.tensor(s["scale"])), torch.zeros((), dtype=torch.float64))
    y1 = norm(h0, leaf["n1"])
    rows = []
    for t, ids in enumerate(s["ids"].cpu().tolist()):
        acc = torch.zeros(y1.shape[1], dtype=torch.float64)
        for j, e in enumerate(ids):
            if e >= 0:
                acc = acc + leaf["weights"][t, j] * (leaf["down"][e] @ (torch.nn.functional.silu(leaf["gate"][e] @ y1[t]) * (leaf["up"][e] @ y1[t])))
        rows.append(acc)
    y2 = norm(h0 + torch.stack(rows), leaf["n2"])
    (y2 * s["c"].double().cpu()).sum().backward()
    for name, a in got.items():
        r = y2.detach() if name == "y" else leaf[name].grad
        e = float((a.double().cpu() - r).norm() / r.norm())
        say(f"step {name}: rel {e:.2e}")
        # a chain of ten fp32 sums of at most 800 terms of random sign: 10 sqrt(800) 2^-24, and twice as much for the slopes of the
        # norms and of the activation, which the errors of their arguments move
        assert e < 30 * 800 ** 0.5 * 2.0 ** -24, name


@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
def test_the_step_and_its_optimizer_in_a_graph(torch, ops, dtype):
    """Three steps eager and three replayed leave the same parameters and states, bit for bit."""
    dt = getattr(torch, dtype)

    def fresh():
        s = inputs(torch, dt)
        mats = {n: torch.zeros(s[n].shape, device="cuda") for n in ("gate", "up", "down")}
        vecs = {n: [torch.zeros_like(s[n], dtype=torch.float32) for _ in range(2)] for n in ("n1", "n2")}
        return s, mats, vecs, ops.adamw8_state(s["table"])

    def train(s, mats, vecs, state, ws):
        g = step(ops, s)
        ops.muon_step_grouped([s["gate"], s["up"], s["down"]], [g["gate"], g["up"], g["down"]], list(mats.values()), lr=0.02, momentum=0.95,
                              weight_decay=0.1, workspace=ws)
        ops.hybrid_step([], [(s[n], g[n], *vecs[n]) for n in vecs] + [(s["table"], g["table"], state)], muon={}, adamw=dict(lr=1e-3, step=3), seed=9)
        return g

    ws_of = lambda s: torch.empty(ops.workspace_bytes_grouped(ops.GRAM, [s["gate"], s["up"], s["down"]], ops.ns_params(io_dtype=ops.dtype_code(s["gate"]))),
                                  dtype=torch.uint8, device="cuda")
    one = fresh()
    ws = ws_of(one[0])
    for _ in range(3):
        train(*one, ws)
    torch.cuda.synchronize()
    assert torch.isfinite(one[0]["table"].float()).all() and not torch.equal(one[0]["table"], inputs(torch, dt)["table"])
    two = fresh()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        train(*fresh(), ws_of(two[0]))                        # libraries are loaded, nothing of `two` is touched
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    ws = ws_of(two[0])
    with torch.cuda.graph(graph):
        train(*two, ws)
    for _ in range(3):
        graph.replay()
        torch.cuda.synchronize()
        step(ops, one[0])                                     # eager work in between
    for n in ("table", "n1", "n2", "gate", "up", "down"):
        assert torch.equal(one[0][n], two[0][n]), n
    for a, b in zip(one[3], two[3]):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
    for n in one[2]:
        assert all(torch.equal(a, b) for a, b in zip(one[2][n], two[2][n]))
