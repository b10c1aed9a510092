"""The gated block's values away from ordinary ones: gates that are infinite or no numbers."""
import pytest

from test_gpu_gated import ACTS, activate, make
from test_gpu_layer import gen_for, normal, ops, torch, uneven  # noqa: F401 (fixtures)

pytestmark = pytest.mark.gpu

# the kernel for few rows, 64 x 64 tiles split over waves, 128 x 64 tiles, 256 x 256 tiles, a dense layer's cut last round
PATHS = [([2, 0, 1], 136, 264, False), ([40, 0, 70], 72, 328, False), ([300, 0, 200], 130, 136, False), (uneven(60, 300, 9), 264, 328, False),
         ([600], 2064, 2568, True)]
name = lambda p: f"{len(p[0])}x{sum(p[0])}_{p[1]}x{p[2]}"  # noqa: E731


def same_kind(torch, got, want, what):
    """NaN where the definition has one, and its infinities; the rest within 1/16 (its accuracy is measured elsewhere)."""
    got = got.double()
    assert torch.equal(torch.isnan(got), torch.isnan(want)), (what, int((torch.isnan(got) != torch.isnan(want)).sum()))
    assert torch.equal(got.isinf() * got.sign().nan_to_num(), want.isinf() * want.sign().nan_to_num()), what
    fine = want.isfinite()
    a, b = got[fine], want[fine]
    assert float((a - b).norm()) <= float(b.norm()) / 16, what


@pytest.mark.parametrize("dtype", ["bfloat16", "float16", "float32"])
@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("path", PATHS, ids=name)
def test_gates_that_are_no_numbers_or_infinite(torch, ops, path, act, dtype):
    counts, n, k, dense = path
    dt = getattr(torch, dtype)
    gen = gen_for(torch, n + 1)
    x, dh, wg, wu, offsets = make(torch, gen, dt, counts, 0, n, k)
    rows = sum(counts)
    expert = torch.repeat_interleave(torch.arange(len(counts), device="cuda"), torch.tensor(counts, device="cuda"))
    args = (wg[0], wu[0], None) if dense else (wg, wu, offsets)
    # forward: a column of gates that are NaN, one of infinities of both signs
    x[:, 0] = 1 - 2.0 * (torch.arange(rows, device="cuda") % 2)
    good = wg.clone()
    wg[:, 1, 3] = float("nan")
    wg[:, n - 1] = 0
    wg[:, n - 1, 0] = float("inf")
    h, gate, up = ops.expert_gated(x, *args, act=act, keep=True)
    assert torch.equal(h.isnan(), ops.expert_gated(x, *args, act=act).isnan())
    assert gate[:, 1].isnan().all() and (gate[:, n - 1] == x[:, 0] * float("inf")).all()
    g, u = gate.double(), up.double()
    same_kind(torch, h, activate(torch, g, act)[0] * u, "h")
    # backward: such gates in some rows, every matrix finite
    wg.copy_(good)
    _, gate, up = ops.expert_gated(x, *args, act=act, keep=True)
    gate[0::7, 1] = float("nan")
    gate[1::7, n - 1] = float("inf")
    gate[2::7, 5] = float("-inf")
    v, s = activate(torch, gate.double(), act)
    dg, du = dh.double() * up.double() * s, dh.double() * v
    dx, dwg, dwu = ops.expert_gated_backward(dh, x, *args[:2], gate, up, args[2], act=act)
    dwg, dwu = dwg.view(wg.shape), dwu.view(wu.shape)
    assert dwu[:, 1].isnan().any() and dx[0::7].isnan().all()
    for e in range(len(counts)):
        r = expert == e
        a, b = dg[r], du[r]
        same_kind(torch, dx[r], a @ wg[e].double() + b @ wu[e].double(), f"dx of expert {e}")
        same_kind(torch, dwg[e], a.T @ x[r].double(), f"dw_gate of expert {e}")
        same_kind(torch, dwu[e], b.T @ x[r].double(), f"dw_up of expert {e}")


def test_offsets_whose_last_is_not_their_largest_read_no_stale_workspace(torch, ops):
    """[0, rows, 3]: every row is the first expert's, whose weights' gradients are those of [0, rows, rows], whatever the workspace held."""
    gen = gen_for(torch, 15)
    for rows, n, k, dt in ((10, 64, 64, torch.float32), (300, 264, 328, torch.bfloat16), (2000, 520, 136, torch.float16)):
        x, dh, wg, wu, ordered = make(torch, gen, dt, [rows, 0], 0, n, k)
        _, gate, up = ops.expert_gated(x, wg, wu, ordered, keep=True)
        want = ops.expert_gated_backward(dh, x, wg, wu, gate, up, ordered)
        falls = torch.tensor([0, rows, 3], dtype=torch.int32, device="cuda")
        for byte in (0, 255):
            ws = torch.full((ops.expert_gated_workspace_bytes(rows, n, x)[1],), byte, dtype=torch.uint8, device="cuda")
            got = ops.expert_gated_backward(dh, x, wg, wu, gate, up, falls, workspace=ws)
            assert all(torch.equal(a, b) for a, b in zip(got[1:], want[1:])), (rows, byte)
            assert torch.equal(got[0][:3], want[0][:3]) and not got[0].isnan().any()


U = 2.0 ** -24


@pytest.mark.parametrize("act", ["silu", "gelu"])
def test_activation_of_fp32_rows_over_its_range(torch, ops, act):
    """The activation and its slope as fp32 functions evaluated to a few roundings, wherever the gate lies: up = 1 and one column of
    x, so that gate, h and both gradients are exact but for them."""
    n = 4096
    gates = torch.linspace(-80.0, 80.0, n, device="cuda") + 0.013
    if act == "gelu":
        gates /= 8                            # its tail ends at -13 in fp32
    x = torch.ones(1, 1, device="cuda")
    wg, wu = gates[:, None].clone(), torch.ones(n, 1, device="cuda")
    h, gate, up = ops.expert_gated(x, wg, wu, act=act, keep=True)
    assert torch.equal(gate[0], gates) and (up == 1).all()
    g = gates.double()
    v, s = activate(torch, g, act)
    if act == "silu":
        # exp to an ulp (2 U), 1 + exp, the quotient and the product a rounding each; the slope a few more of terms up to |g| s
        ev, es = 6 * U * v.abs(), 12 * U * (torch.sigmoid(g) * (1 + g.abs() * torch.sigmoid(-g)))
    else:
        # erfc's argument is rounded: 2 t^2 = g^2 of it in the tail, to 8 ulp; exp(-g^2 / 2) likewise
        f = 0.5 * torch.erfc(-g / 2 ** 0.5)
        tail = torch.where(g < 0, g * g, torch.zeros_like(g))
        ev = (20 + 2 * tail) * U * v.abs()
        es = (20 + 2 * tail) * U * f + (6 + 2 * g * g) * U * g.abs() * torch.exp(-g * g / 2) * 0.4
    assert ((h[0].double() - v).abs() <= ev + 1e-37).all(), ((h[0].double() - v).abs() / (v.abs() * U)).max()
    _, dwg, dwu = ops.expert_gated_backward(torch.ones(1, n, device="cuda"), x, wg, wu, gate, up, act=act)
    assert ((dwu[:, 0].double() - v).abs() <= ev + 1e-37).all(), ((dwu[:, 0].double() - v).abs() / (v.abs() * U)).max()
    assert ((dwg[:, 0].double() - s).abs() <= es + 1e-37).all(), ((dwg[:, 0].double() - s).abs() / (s.abs() * U)).max()


@pytest.mark.parametrize("dtype", ["bfloat16", "float16"])
def test_gelu_of_16_bit_rows_in_its_lower_tail(torch, ops, dtype):
    """dup = dh gelu(gate) is the forward's gelu of the kept gate, rounded once: right to its last bit or next to it down to where it
    underflows, as the forward result is."""
    dt = getattr(torch, dtype)
    n = 2048
    gates = torch.linspace(-4.6 if dtype == "float16" else -12.0, 4.0, n, device="cuda").to(dt)
    x, wg, wu = torch.ones(1, 1, dtype=dt, device="cuda"), gates[:, None].clone(), torch.ones(n, 1, dtype=dt, device="cuda")
    h, gate, up = ops.expert_gated(x, wg, wu, act="gelu", keep=True)
    _, _, dwu = ops.expert_gated_backward(torch.ones(1, n, dtype=dt, device="cuda"), x, wg, wu, gate, up, act="gelu")
    assert torch.equal(gate[0], gates)
    v = activate(torch, gates.double(), "gelu")[0]
    info = torch.finfo(dt)
    # half a step of the type (of its smallest numbers below its normal range), and 4e-6 + g^2 2^-24 of the value in fp32 before it
    bound = info.eps / 2 * v.abs().clamp(min=info.tiny) + (4e-6 + gates.double() ** 2 * 4 * U) * v.abs()
    for got in (h[0], dwu[:, 0]):
        assert ((got.double() - v).abs() <= bound).all(), ((got.double() - v).abs() / bound).max()


@pytest.mark.parametrize("dtype", ["bfloat16", "float16"])
def test_the_workspace_asked_for_is_all_that_a_dense_call_takes(torch, ops, dtype):
    """A call with far more room gives the bits of one with as much as it asks for, over the rules that choose its kernel."""
    dt = getattr(torch, dtype)
    gen = gen_for(torch, 60)
    room = torch.empty(256 << 20, dtype=torch.uint8, device="cuda")
    for n, k in ((72, 2560), (1024, 2568), (2064, 2560), (4104, 4096), (1216, 20000), (9000, 2504)):
        wg, wu = (normal(torch, gen, n, k).mul(k ** -0.5).to(dt) for _ in range(2))
        for rows in (1, 4, 5, 17, 64, 100, 300, 512, 600, 1100, 2500):
            x, dh = normal(torch, gen, rows, k).to(dt), normal(torch, gen, rows, n).to(dt)
            h, gate, up = ops.expert_gated(x, wg, wu, keep=True)
            assert torch.equal(h, ops.expert_gated(x, wg, wu, workspace=room)), (rows, n, k)
            own = ops.expert_gated_backward(dh, x, wg, wu, gate, up)
            wide = ops.expert_gated_backward(dh, x, wg, wu, gate, up, workspace=room)
            assert all(torch.equal(a, b) for a, b in zip(own, wide)), (rows, n, k)


@pytest.mark.parametrize("act", ACTS)
def test_each_gradient_against_differences_in_64_bits(torch, ops, act):
    """The directional derivative of sum(c h), taken from the definition in 64 bits, along each of x, w_gate and w_up alone."""
    gen = gen_for(torch, 19)
    counts, n, k = [7, 0, 20, 5], 40, 72
    x, c, wg, wu, offsets = make(torch, gen, torch.float32, counts, 2, n, k)
    _, gate, up = ops.expert_gated(x, wg, wu, offsets, act=act, keep=True)
    if act == "relu":
        c = c * (gate.abs() > 1e-3)           # no gate changes its side within a step
    dirs = [normal(torch, gen, *t.shape).double() for t in (x, wg, wu)]
    bounds = offsets.tolist()

    def loss(x, wg, wu):
        total = 0.0
        for e, (lo, hi) in enumerate(zip(bounds, bounds[1:])):
            total += (c[lo:hi].double() * activate(torch, x[lo:hi] @ wg[e].T, act)[0] * (x[lo:hi] @ wu[e].T)).sum()
        return total

    grads = ops.expert_gated_backward(c, x, wg, wu, gate, up, offsets, act=act)
    at = [t.double() for t in (x, wg, wu)]
    step = 2.0 ** -18
    for i, what in enumerate(("dx", "dw_gate", "dw_up")):
        ends = [loss(*(t + s * step * dirs[i] if j == i else t for j, t in enumerate(at))) for s in (1, -1)]
        want = (ends[0] - ends[1]) / (2 * step)
        got = (grads[i].double() * dirs[i]).sum()
        # three chained sums of at most 80 terms of random sign at 2^-24 each, with slopes and factors of order 1, are off by less than
        # 20 sqrt(80) 2^-24 = 1.1e-5 of the gradient's norm, and a normal direction picks up its error's norm, four times that at most; the
        # difference's own error, step^2 of third derivatives, is 1e-11. A gradient left out would be off by its norm.
        bound = 5e-5 * grads[i].double().norm()
        assert abs(got - want) <= bound and abs(want) > 20 * bound, (what, got, want, bound)
