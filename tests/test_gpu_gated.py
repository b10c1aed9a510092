"""The gated block and its gradients against their definitions in 64 bits.

Tolerances: a result is rounded once to its type, at most half a step; an MFMA sum of k terms is off by at most
(k + 2) 2^-23 times the sum of their magnitudes. The activation of g is off by the error of g times its slope (below 1.2)
and by (8 + 2 |g|) 2^-24 |g| (the exponential's argument is rounded, then a few operations); its slope by as much of 1 + |g|.
dgate and dup are rounded to the type once more before they are summed, half a step each.
"""
import math

import pytest

from test_gpu_layer import DTYPES, MANY, PRODUCTS, buffer, close, gen_for, normal, ops, torch, uneven  # noqa: F401 (fixtures)
from test_gpu_layer_loops import ALIGNED, LOOPS

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
ACTS = ["silu", "gelu", "relu"]


def activate(torch, g, act):
    if act == "relu":
        return g.clamp(min=0), (g > 0).double()
    if act == "silu":
        s = torch.sigmoid(g)
        return g * s, s * (1 + g * (1 - s))
    f = 0.5 * torch.erfc(-g / math.sqrt(2))
    return g * f, f + g * torch.exp(-g * g / 2) / math.sqrt(2 * math.pi)


def make(torch, gen, dt, counts, rest, n, k, pad=0, shift=0):
    rows = sum(counts) + rest
    x, dh = buffer(torch, gen, dt, rows, k, pad, shift), buffer(torch, gen, dt, rows, n, pad, shift)
    ws = []
    for _ in range(2):
        w = buffer(torch, gen, dt, len(counts) * n, k, pad, shift)
        ws.append(w.as_strided((len(counts), n, k), (n * w.stride(0), w.stride(0), 1), w.storage_offset()))
        ws[-1].mul_(2 * k ** -0.5)
    offsets = torch.tensor([0] + counts, device="cuda").cumsum(0).to(torch.int32)
    return x, dh, ws[0], ws[1], offsets


def check(torch, ops, x, dh, wg, wu, counts, offsets, act):
    h, gate, up = ops.expert_gated(x, wg, wu, offsets, act=act, keep=True)
    assert torch.equal(ops.expert_gated(x, wg, wu, offsets, act=act), h)
    dx, dwg, dwu = ops.expert_gated_backward(dh, x, wg, wu, gate, up, offsets, act=act)
    assert dx.shape == x.shape and dwg.shape == wg.shape and dwu.shape == wu.shape
    wg3, wu3 = wg.reshape(-1, *wg.shape[-2:]), wu.reshape(-1, *wu.shape[-2:])
    dwg, dwu = dwg.view(wg3.shape), dwu.view(wu3.shape)
    n, k = wg.shape[-2:]
    info = torch.finfo(x.dtype)
    half = info.eps / 2
    least = info.tiny * half
    at = 0
    for e, c in enumerate(counts):
        if c == 0:
            assert not dwg[e].any() and not dwu[e].any()
            continue
        r = slice(at, at + c)
        a, mg, mu = x[r].double(), wg3[e].double(), wu3[e].double()
        g, u = a @ mg.T, a @ mu.T
        eg, eu = ((k + 2) * 2 * U * (a.abs() @ m.abs().T) for m in (mg, mu))
        close(gate[r], g, eg, f"gate of expert {e}")
        close(up[r], u, eu, f"up of expert {e}")
        v, _ = activate(torch, g, act)
        ev = 1.2 * eg + (8 + 2 * g.abs()) * U * g.abs()
        close(h[r], v * u, ev * (u.abs() + eu) + v.abs() * eu + U * (v * u).abs(), f"h of expert {e}")
        # the gradients from gate and up as kept
        g, u, d = gate[r].double(), up[r].double(), dh[r].double()
        v, s = activate(torch, g, act)
        dg, du = d * u * s, d * v
        eg = half * dg.abs() + (16 + 4 * g.abs()) * U * (1 + g.abs()) * (d * u).abs() + least
        eu = half * du.abs() + (10 + 2 * g.abs()) * U * g.abs() * d.abs() + least
        close(dx[r], dg @ mg + du @ mu, eg @ mg.abs() + eu @ mu.abs() + (2 * n + 2) * 2 * U * (dg.abs() @ mg.abs() + du.abs() @ mu.abs()), f"dx of expert {e}")
        close(dwg[e], dg.T @ a, eg.T @ a.abs() + (c + 2) * 2 * U * (dg.abs().T @ a.abs()), f"dw_gate of expert {e}")
        close(dwu[e], du.T @ a, eu.T @ a.abs() + (c + 2) * 2 * U * (du.abs().T @ a.abs()), f"dw_up of expert {e}")
        at += c
    for t in (h, gate, up, dx):
        assert not t[at:].any()


def run_case(torch, ops, case, dtype, act, pad=0, shift=0):
    counts, rest, n, k = case
    gen = gen_for(torch, n + k)
    x, dh, wg, wu, offsets = make(torch, gen, getattr(torch, dtype), counts, rest, n, k, pad, shift)
    x[sum(counts):] = float("nan")           # rows of nobody are not read into anything
    dh[sum(counts):] = float("nan")
    check(torch, ops, x, dh, wg, wu, counts, offsets, act)


name = lambda c: f"{len(c[0])}x{sum(c[0])}+{c[1]}_{c[2]}x{c[3]}"  # noqa: E731


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("case", list(enumerate(PRODUCTS)), ids=lambda c: name(c[1]))
def test_gated(torch, ops, case, dtype):
    run_case(torch, ops, case[1], dtype, ACTS[case[0] % 3])


# the 256 x 256 tiles, many experts; widths N of no whole chunk, whose gradients take them as well
WIDE = MANY + [(uneven(70, 600, 21), 3, 265, 264), (uneven(33, 300, 22), 0, 1407, 1024), ([300] * 60, 0, 131, 1032), (uneven(40, 500, 23), 5, 2047, 136)]


@pytest.mark.parametrize("dtype", ["bfloat16", "float16"])
@pytest.mark.parametrize("case", list(enumerate(WIDE)), ids=lambda c: name(c[1]))
def test_gated_of_many_experts(torch, ops, case, dtype):
    run_case(torch, ops, case[1], dtype, ACTS[case[0] % 3], pad=8)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("case", LOOPS + [(*c, 0, 0) for c in ALIGNED], ids=name)
def test_gated_of_several_tiles_a_workgroup(torch, ops, case, dtype):
    run_case(torch, ops, case[:4], dtype, "silu", *case[4:])


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("pad,shift", [(8, 0), (3, 0), (8, 1), (0, 8), (1, 3)])
def test_gated_strided_and_unaligned(torch, ops, dtype, pad, shift):
    run_case(torch, ops, ([70, 0, 200, 1], 4, 264, 328), dtype, "gelu", pad, shift)
    run_case(torch, ops, ([3, 0, 2], 1, 72, 137), dtype, "silu", pad, shift)


NARROW = [(1, 9), (3, 8), (4, 4), (5, 7), (7, 5), (8, 3), (9, 1), (9, 17), (12, 31), (130, 15), (15, 130), (257, 33), (33, 2067), (300, 5), (301, 261)]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("counts,rest", [([2, 0, 1], 1), ([17, 0, 3, 40], 0), ([400, 0, 390], 1)], ids=str)
@pytest.mark.parametrize("n,k", NARROW)
def test_gated_of_rows_shorter_than_a_load(torch, ops, n, k, counts, rest, dtype):
    run_case(torch, ops, (counts, rest, n, k), dtype, ACTS[(n + k) % 3], 1, 1)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("shape", [(1, 264, 520), (5, 1000, 776), (40, 2048, 512), (300, 520, 264), (2048, 1032, 264), (1500, 1031, 265), (600, 7, 3), (0, 64, 72)], ids=str)
def test_gated_dense(torch, ops, shape, dtype):
    """One pair of matrices, no offsets: the one expert's calls, bit for bit."""
    rows, n, k = shape
    gen = gen_for(torch, n)
    x, dh, wg, wu, offsets = make(torch, gen, getattr(torch, dtype), [rows], 0, n, k)
    check(torch, ops, x, dh, wg[0], wu[0], [rows], None, "silu")
    h, gate, up = ops.expert_gated(x, wg, wu, offsets, keep=True)
    assert torch.equal(h, ops.expert_gated(x, wg[0], wu[0])) and torch.equal(h, ops.expert_gated(x, wg, wu))
    one = ops.expert_gated_backward(dh, x, wg, wu, gate, up, offsets)
    two = ops.expert_gated_backward(dh, x, wg[0], wu[0], gate, up)
    assert torch.equal(one[0], two[0]) and torch.equal(one[1][0], two[1]) and torch.equal(one[2][0], two[2])
    # either half of the gradients on its own
    assert torch.equal(ops.expert_gated_backward(dh, x, wg, wu, gate, up, need_weights=False)[0], one[0])
    half = ops.expert_gated_backward(dh, x, wg, wu, gate, up, need_input=False)
    assert half[0] is None and torch.equal(half[1], one[1]) and torch.equal(half[2], one[2])


# whole rounds and a cut one, a cut one alone in two to sixteen parts, N of no whole chunk (the input gradient's contraction),
# contractions that end inside a stage, parts that begin in the second of the input gradient's
CUT = [(600, 2064, 2056, 0), (1030, 2064, 2056, 8), (300, 4104, 2120, 0), (2500, 4160, 2048, 0), (1290, 2047, 2056, 8), (520, 1099, 4104, 0), (770, 18440, 2056, 0),
       (600, 2064, 2568, 0), (1030, 2064, 2632, 8), (2500, 4160, 2616, 0), (300, 4104, 4104, 8)]


@pytest.mark.parametrize("dtype", ["bfloat16", "float16"])
@pytest.mark.parametrize("shape", CUT, ids=str)
def test_gated_dense_with_a_cut_last_round(torch, ops, shape, dtype):
    rows, n, k, pad = shape
    gen = gen_for(torch, n)
    dt = getattr(torch, dtype)
    x, dh, wg, wu, _ = make(torch, gen, dt, [rows], 0, n, k, pad)
    check(torch, ops, x, dh, wg[0], wu[0], [rows], None, "silu")
    # a workspace of its own, and one of the size of an uncut call: the same gradients up to the sums' order
    fwd, bwd = ops.expert_gated_workspace_bytes(rows, n, x, dense=True)
    least = ops.expert_gated_workspace_bytes(rows, n, x)[1]
    ws = torch.full((bwd + 256,), 255, dtype=torch.uint8, device="cuda")
    h, gate, up = ops.expert_gated(x, wg[0], wu[0], keep=True, workspace=ws[128:128 + fwd])
    again = ops.expert_gated(x, wg[0], wu[0], keep=True)
    assert all(torch.equal(a, b) for a, b in zip((h, gate, up), again))
    dx = ops.expert_gated_backward(dh, x, wg[0], wu[0], gate, up, need_weights=False, workspace=ws[128:128 + bwd])[0]
    assert torch.equal(dx, ops.expert_gated_backward(dh, x, wg[0], wu[0], gate, up, need_weights=False)[0])
    assert (ws[:128] == 255).all() and (ws[128 + bwd:] == 255).all()
    flat = ops.expert_gated_backward(dh, x, wg[0], wu[0], gate, up, need_weights=False, workspace=ws[128:128 + least])[0]
    u = (2 * n + 40) * 2 * U
    d = dh.double()
    v, s = activate(torch, gate.double(), "silu")
    mag = (d * up.double() * s).abs() @ wg[0].double().abs() + (d * v).abs() @ wu[0].double().abs()
    assert ((dx.double() - flat.double()).abs() <= torch.finfo(dt).eps * flat.double().abs() + u * mag + torch.finfo(dt).tiny).all()
    # the matrices' own rows of different length, in both halves of the contraction
    wide = torch.cat([wu[0], wu[0]], dim=1)[:, :k]
    assert torch.equal(ops.expert_gated(x, wg[0], wide), h)
    assert torch.equal(ops.expert_gated_backward(dh, x, wg[0], wide, gate, up, need_weights=False)[0], dx)


@pytest.mark.parametrize("dtype", ["bfloat16", "float32"])
def test_gated_matrices_of_one_buffer_and_of_different_strides(torch, ops, dtype):
    """Gate and up matrices side by side in one batch [experts, 2, N, K], and two with rows of different length."""
    dt = getattr(torch, dtype)
    for counts, n, k in (([40, 0, 70, 9], 72, 136), (uneven(60, 300, 9), 264, 328), ([2, 1], 1000, 776)):
        gen = gen_for(torch, n)
        x, dh, wg, wu, offsets = make(torch, gen, dt, counts, 0, n, k)
        h, gate, up = ops.expert_gated(x, wg, wu, offsets, keep=True)
        want = ops.expert_gated_backward(dh, x, wg, wu, gate, up, offsets)
        both = torch.stack([wg, wu], dim=1)
        wide = torch.cat([wu, wu], dim=2)[:, :, :k]
        for a, b in ((both[:, 0], both[:, 1]), (wg, wide), (wide, wg)):
            swap = a is wide
            got = ops.expert_gated(x, b if swap else a, a if swap else b, offsets, keep=True)
            assert all(torch.equal(p, q) for p, q in zip(got, (h, gate, up)))
            got = ops.expert_gated_backward(dh, x, b if swap else a, a if swap else b, gate, up, offsets)
            assert all(torch.equal(p, q) for p, q in zip(got, want))


def test_gated_writes_nothing_outside(torch, ops):
    gen = gen_for(torch, 12)
    for counts, n, k in (([40, 0, 70], 72, 136), (uneven(60, 300, 9), 264, 328), ([3, 1], 72, 136)):
        rows = sum(counts)
        x, dh, wg, wu, offsets = make(torch, gen, torch.bfloat16, counts, 0, n, k)
        full = torch.full((rows + 4, n + 16), 7.0, dtype=torch.bfloat16, device="cuda")
        got = ops.expert_gated(x, wg, wu, offsets, out=full[2:-2, 8:-8]).clone()
        full[2:-2, 8:-8] = 7.0
        assert (full == 7.0).all() and torch.equal(got, ops.expert_gated(x, wg, wu, offsets))
        h, gate, up = ops.expert_gated(x, wg, wu, offsets, keep=True)
        need = ops.expert_gated_workspace_bytes(rows, n, x)[1]
        ws = torch.full((need + 256,), 255, dtype=torch.uint8, device="cuda")
        got = ops.expert_gated_backward(dh, x, wg, wu, gate, up, offsets, workspace=ws[128:128 + need])
        assert (ws[:128] == 255).all() and (ws[128 + need:] == 255).all()
        assert all(torch.equal(p, q) for p, q in zip(got, ops.expert_gated_backward(dh, x, wg, wu, gate, up, offsets)))


def test_gated_extremes(torch, ops):
    """Gates far out on both sides: the activation goes to 0 and to g, its slope to 0 and 1, without a NaN."""
    x = torch.ones(1, 8, device="cuda")
    wg = torch.tensor([-3e38, -1e4, -90.0, -1e-30, 0.0, 1e-30, 90.0, 1e4, 3e38], device="cuda")[:, None] * torch.eye(8, device="cuda")[0]
    wu = torch.ones(9, 1, device="cuda") * torch.eye(8, device="cuda")[0]
    for act in ACTS:
        h, gate, up = ops.expert_gated(x, wg, wu, act=act, keep=True)
        assert torch.equal(gate[0], wg[:, 0]) and (up == 1).all()
        assert torch.equal(h[0, 6:], gate[0, 6:]) and not h[0, :2].any() and h[0, 2].abs() < 1e-36 and h[0, 4] == 0
        dx, dwg, dwu = ops.expert_gated_backward(torch.ones(1, 9, device="cuda"), x, wg, wu, gate, up, act=act)
        assert torch.isfinite(dwg).all() and torch.isfinite(dwu).all()
        assert ((dwu[:, 0] - h[0]).abs() <= 4 * U * h[0].abs()).all() and (dwg[6:, 0] == 1).all() and (dwg[:2, 0] == 0).all()
        assert dwg[4, 0] == (0.0 if act == "relu" else 0.5)


@pytest.mark.parametrize("act", ACTS)
def test_gated_gradient_against_differences(torch, ops, act):
    gen = gen_for(torch, 9)
    counts = [7, 0, 20, 5]
    x, c, wg, wu, offsets = make(torch, gen, torch.float32, counts, 2, 40, 72)
    vx, vg, vu = (normal(torch, gen, *t.shape) for t in (x, wg, wu))
    step = 2.0 ** -8 if act != "relu" else 2.0 ** -12   # relu: few gates change their side within a step
    _, g0, _ = ops.expert_gated(x, wg, wu, offsets, act=act, keep=True)
    _, g1, _ = ops.expert_gated(x + step * vx, wg + step * vg, wu, offsets, act=act, keep=True)
    _, g2, _ = ops.expert_gated(x - step * vx, wg - step * vg, wu, offsets, act=act, keep=True)
    same = ((g0 > 0) == (g1 > 0)) & ((g0 > 0) == (g2 > 0)) if act == "relu" else torch.ones_like(g0, dtype=torch.bool)
    c = c * same
    loss = lambda s: (ops.expert_gated(x + s * vx, wg + s * vg, wu + s * vu, offsets, act=act).double() * c.double()).sum()
    h, gate, up = ops.expert_gated(x, wg, wu, offsets, act=act, keep=True)
    dx, dwg, dwu = ops.expert_gated_backward(c, x, wg, wu, gate, up, offsets, act=act)
    got = sum((a.double() * b.double()).sum() for a, b in ((dx, vx), (dwg, vg), (dwu, vu)))
    diff = (loss(step) - loss(-step)) / (2 * step)
    # error of the difference: step^2 times the third derivative along the line (up to the cubes of the directions'
    # products, |v| about 6 for gate and up), and the sums' 74 terms at 2^-23 over the step
    reach = 1 + (vx.abs().double()[:, None, :] @ wg.abs().double().mean(0).T[None]).mean()
    scale = ((gate.abs() + 1).double() * (up.abs() + 1).double() * c.abs().double()).sum()
    assert abs(got - diff) <= scale * (74 * 2 * U / step + reach ** 3 * step * step), (got, diff, scale, reach)


def test_gated_past_32_bits(torch, ops):
    """320000 rows of 7168, in the 256 x 256 tiles and in the gradients."""
    gen = gen_for(torch, 22)
    rows, n, k = 320000, 136, 7168
    offsets = torch.tensor([0, 100001, 100001, 250000, rows - 7], dtype=torch.int32, device="cuda")
    x = torch.empty(rows, k, dtype=torch.bfloat16, device="cuda")
    for lo in range(0, rows, 20000):
        x[lo:lo + 20000] = normal(torch, gen, 20000, k).to(x.dtype)
    wg, wu = (normal(torch, gen, 4, n, k).mul(k ** -0.5).to(torch.bfloat16) for _ in range(2))
    h, gate, up = ops.expert_gated(x, wg, wu, offsets, keep=True)
    assert not h[-7:].any()
    dh = normal(torch, gen, rows, n).to(torch.bfloat16)
    dx, dwg, dwu = ops.expert_gated_backward(dh, x, wg, wu, gate, up, offsets)
    assert not dx[-7:].any() and not dwg[1].any() and not dwu[1].any()
    bounds = offsets.tolist()
    for s in (0, 100000, 100001, 250000, 299593, 299594, rows - 8):
        e = sum(s >= b for b in bounds[1:])
        a, mg, mu = x[s].double(), wg[e].double(), wu[e].double()
        g, u = mg @ a, mu @ a
        eg, eu = (k + 2) * 2 * U * (mg.abs() @ a.abs()), (k + 2) * 2 * U * (mu.abs() @ a.abs())
        close(gate[s], g, eg, f"gate row {s}")
        v, _ = activate(torch, g, "silu")
        close(h[s], v * u, (1.2 * eg + (8 + 2 * g.abs()) * U * g.abs()) * (u.abs() + eu) + v.abs() * eu, f"h row {s}")
        g, u, d = gate[s].double(), up[s].double(), dh[s].double()
        v, sl = activate(torch, g, "silu")
        dg, du = d * u * sl, d * v
        e1, e2 = 2.0 ** -8 * dg.abs() + 2.0 ** -18 * (d * u).abs(), 2.0 ** -8 * du.abs() + 2.0 ** -18 * d.abs() * g.abs()
        close(dx[s], dg @ mg + du @ mu, e1 @ mg.abs() + e2 @ mu.abs() + (2 * n + 2) * 2 * U * (dg.abs() @ mg.abs() + du.abs() @ mu.abs()), f"dx row {s}")
    lo, hi = bounds[3], bounds[4]
    g, u, d = gate[lo:hi, -16:].double(), up[lo:hi, -16:].double(), dh[lo:hi, -16:].double()
    v, sl = activate(torch, g, "silu")
    a = x[lo:hi, -64:].double()
    for got, t in ((dwg, d * u * sl), (dwu, d * v)):
        close(got[3, -16:, -64:], t.T @ a, (2.0 ** -8 + (hi - lo + 2) * 2 * U) * (t.abs().T @ a.abs()), "dw")


def test_gated_offsets_in_no_order_write_nothing_outside(torch, ops):
    gen = gen_for(torch, 14)
    for rows, n, k, dt in ((10, 64, 64, torch.float32), (300, 264, 328, torch.bfloat16), (2000, 520, 136, torch.float16), (900, 130, 70, torch.bfloat16)):
        for raw in ([0, rows] * 9, [rows // 2, rows, 3, -5, rows + 9, 0, rows], [2 ** 31 - 1, -2 ** 31, 5, 4, 3, 2 ** 31 - 1, 0, 7]):
            off = torch.tensor(raw, dtype=torch.int32, device="cuda")
            wg, wu = (normal(torch, gen, len(raw) - 1, n, k).to(dt) for _ in range(2))
            x, dh = normal(torch, gen, rows, k).to(dt), normal(torch, gen, rows, n).to(dt)
            full = torch.full((rows + 4, n + 16), 7.0, dtype=dt, device="cuda")
            ops.expert_gated(x, wg, wu, off, out=full[2:-2, 8:-8])
            full[2:-2, 8:-8] = 7.0
            assert (full == 7.0).all()
            h, gate, up = ops.expert_gated(x, wg, wu, off, keep=True)
            ops.expert_gated_backward(dh, x, wg, wu, gate, up, off)
    torch.cuda.synchronize()


@pytest.mark.parametrize("dtype", ["bfloat16", "float32"])
def test_gated_on_any_stream_and_in_a_graph(torch, ops, dtype):
    """Experts and a dense layer, each path by size: eager twice, on a side stream, and replayed with other inputs in between."""
    dt = getattr(torch, dtype)
    gen = gen_for(torch, 33)
    sets = []
    for counts, rest, n, k, dense in ((uneven(60, 300, 9), 3, 264, 328, False), ([3, 0, 2], 0, 72, 136, False), ([70, 5], 1, 130, 70, False),
                                      ([600], 0, 2064, 2056, True), ([600], 0, 2064, 2568, True)):
        x, dh, wg, wu, off = make(torch, gen, dt, counts, rest, n, k)
        if dense:
            wg, wu, off = wg[0], wu[0], None
        ws = [torch.empty(b, dtype=torch.uint8, device="cuda") for b in ops.expert_gated_workspace_bytes(x.shape[0], n, x, dense=dense)]
        sets.append((x, dh, wg, wu, off, ws))

    def run(own):
        out = []
        for x, dh, wg, wu, off, ws in sets:
            h, gate, up = ops.expert_gated(x, wg, wu, off, keep=True, workspace=ws[0] if own else None)
            out += [h, *ops.expert_gated_backward(dh, x, wg, wu, gate, up, off, workspace=ws[1] if own else None)]
        return out

    want = [t.clone() for t in run(False)]
    assert all(torch.equal(a, b) for a, b in zip(want, run(False)))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        other = run(True)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, other))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = run(True)
    keep = [(s[0].clone(), s[1].clone()) for s in sets]
    for i in range(4):
        for (x, dh, *_), (x0, dh0) in zip(sets, keep):
            x.copy_(x0 if i % 2 == 0 else -x0)
            dh.copy_(dh0 if i % 2 == 0 else dh0.flip(1))
        graph.replay()
        torch.cuda.synchronize()
        eager = run(False)
        assert all(torch.equal(a, b) for a, b in zip(held, eager)), i


def test_gated_on_two_streams_at_once(torch, ops):
    gen = gen_for(torch, 34)
    sets = []
    for counts, n, k, dense in (([600], 2064, 2568, True), (uneven(24, 900, 10), 264, 328, False)):
        x, dh, wg, wu, off = make(torch, gen, torch.bfloat16, counts, 0, n, k)
        if dense:
            wg, wu, off = wg[0], wu[0], None
        sets.append((x, dh, wg, wu, off, [torch.empty(b, dtype=torch.uint8, device="cuda") for b in ops.expert_gated_workspace_bytes(x.shape[0], n, x, dense=dense)]))

    def run(x, dh, wg, wu, off, ws):
        h, gate, up = ops.expert_gated(x, wg, wu, off, keep=True, workspace=ws[0])
        return [h, *ops.expert_gated_backward(dh, x, wg, wu, gate, up, off, workspace=ws[1])]

    want = [[t.clone() for t in run(*s)] for s in sets]
    streams = [torch.cuda.Stream() for _ in sets]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    for _ in range(6):
        got = []
        for s, a in zip(streams, sets):
            with torch.cuda.stream(s):
                got.append(run(*a))
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for g, w in zip(got, want) for a, b in zip(g, w))
