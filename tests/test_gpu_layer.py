"""Layer norm, rows by expert and the experts' products against their definitions in 64 bits.

Tolerances: a result is rounded once to its type, at most half a step, eps / 2 of its value; the
fp32 sums before it are off by at most (number of additions) x 2^-24 x the sum of the terms'
magnitudes (2^-23 for MFMA, whose internal rounding may truncate). Copies and plans are exact.
"""
import pytest

from helpers import say

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def torch():
    import torch as t
    if not t.cuda.is_available():
        pytest.skip("no GPU")
    return t


@pytest.fixture(scope="module")
def ops():
    from newton_schulz_matrix_muon_amd import ops as o
    o.lib()
    return o


DTYPES = ["float32", "bfloat16", "float16"]


def gen_for(torch, seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def normal(torch, gen, *shape):
    return torch.randn(*shape, generator=gen, device="cuda")


def buffer(torch, gen, dt, rows, cols, pad=0, shift=0):
    """Random rows x cols with `pad` columns behind each row and a base `shift` elements into its storage."""
    flat = normal(torch, gen, rows * (cols + pad) + shift + 8).to(dt)
    return flat[shift:shift + rows * (cols + pad)].view(rows, cols + pad)[:, :cols]


def close(got, ref, slack, what):
    """|got - ref| <= eps / 2 |ref| + slack (+ half a step more relative to the slack's own rounding)."""
    import torch
    eps = torch.finfo(got.dtype).eps
    tiny = torch.finfo(got.dtype).tiny
    got = got.double()
    bound = eps / 2 * ref.abs() + slack * (1 + eps) + tiny
    bad = ~((got - ref).abs() <= bound)
    if bad.any():
        i = int(bad.reshape(-1).nonzero()[0])
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.numel()} off, first at {i}: {got.reshape(-1)[i]} "
                             f"for {ref.reshape(-1)[i]} (bound {bound.expand_as(ref).reshape(-1)[i]:.3g})")


# ------------------------------------------------------------------------------- layer norm

NORM_SHAPES = [  # rows, cols, columns behind each row, first element
    (1, 1, 0, 0), (1, 7168, 0, 0), (3, 7, 0, 0), (5, 8, 0, 0), (17, 64, 8, 0), (64, 200, 0, 8), (65, 2047, 0, 0),
    (33, 2048, 0, 0), (129, 2056, 0, 0), (7, 2048, 3, 1), (600, 512, 0, 0), (1030, 264, 0, 0), (9, 7168, 16, 8),
    (5, 8192, 0, 0), (4, 8200, 0, 0), (3, 16384, 0, 0), (2, 33000, 0, 0), (2, 33001, 1, 0), (0, 64, 0, 0), (2500, 24, 0, 0),
]


def norm_ref(torch, x, w, b, eps):
    x = x.double()
    mean = x.mean(dim=-1)
    c = x - mean[..., None]
    rstd = 1 / torch.sqrt((c * c).mean(dim=-1) + eps)
    xh = c * rstd[..., None]
    return xh * w.double() + b.double(), mean, rstd, xh


def adds(cols):
    return cols // 64 + 40   # at most cols / 64 in a thread, the tree over the threads, and the arithmetic around it


@pytest.mark.parametrize("wide", [False, True], ids=["own", "fp32w"])
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("shape", NORM_SHAPES, ids=str)
def test_layer_norm_and_gradient(torch, ops, shape, dtype, wide):
    rows, cols, pad, shift = shape
    dt = getattr(torch, dtype)
    wdt = torch.float32 if wide else dt
    gen = gen_for(torch, rows * 31 + cols)
    x = buffer(torch, gen, dt, rows, cols, pad, shift)
    x += 0.5
    dy = buffer(torch, gen, dt, rows, cols, pad, shift)
    w = (1 + 0.1 * normal(torch, gen, cols)).to(wdt)
    b = (0.1 * normal(torch, gen, cols)).to(wdt)
    eps = 1e-5
    y, mean, rstd = ops.layer_norm(x, w, b, eps=eps)
    dx, dw, db = ops.layer_norm_backward(dy, x, mean, rstd, w)
    torch.cuda.synchronize()
    assert y.shape == x.shape and dx.shape == x.shape and dw.dtype == wdt and db.dtype == wdt
    if rows == 0:
        assert not dw.any() and not db.any()
        return
    ref, rmean, rrstd, xh = norm_ref(torch, x, w, b, eps)
    u = adds(cols) * 2.0 ** -24
    big = x.double().abs().amax(dim=1, keepdim=True)
    close(mean, rmean, u * big[:, 0], "mean")
    # the variance's terms are (x - mean)^2, each off by 2 |x - mean| times the error of the mean
    close(rstd, rrstd, rrstd * (u + 4 * u * big[:, 0] * rrstd), "rstd")
    amp = big * rrstd[:, None]
    close(y, ref, u * (3 * amp * (1 + amp) * w.double().abs() + b.double().abs()), "y")
    # the gradients from the kept statistics, as the call takes them
    mean, rstd = mean.double()[:, None], rstd.double()[:, None]
    xh = (x.double() - mean) * rstd
    g = dy.double() * w.double()
    ref = rstd * (g - g.mean(dim=1, keepdim=True) - xh * (g * xh).mean(dim=1, keepdim=True))
    ga, xa = g.abs(), ((x.double().abs() + mean.abs()) * rstd)
    close(dx, ref, u * rstd * (ga + ga.mean(dim=1, keepdim=True) * (1 + 2 * xa.amax(dim=1, keepdim=True) ** 2)), "dx")
    ur = (rows + 40) * 2.0 ** -24
    close(dw, (dy.double() * xh).sum(dim=0), ur * (dy.double().abs() * xa).sum(dim=0), "dweight")
    close(db, dy.double().sum(dim=0), ur * dy.double().abs().sum(dim=0), "dbias")


def test_layer_norm_without_parameters_batched_and_out(torch, ops):
    gen = gen_for(torch, 5)
    base = normal(torch, gen, 3, 10, 72).to(torch.bfloat16)
    x = base[:, 1:8, :64]                                     # strided batch and rows
    full = torch.full((3, 10, 72), 7.0, dtype=torch.bfloat16, device="cuda")
    y, mean, rstd = ops.layer_norm(x, out=full[:, 1:8, :64])
    flat, fm, fr = ops.layer_norm(x.reshape(-1, 64))
    assert mean.shape == (3, 7) and torch.equal(mean.reshape(-1), fm) and torch.equal(rstd.reshape(-1), fr)
    assert torch.equal(y.reshape(-1, 64), flat)
    full[:, 1:8, :64] = 7.0
    assert (full == 7.0).all()                                # nothing outside was written
    dy = normal(torch, gen, 3, 7, 64).to(torch.bfloat16)
    dx, dw, db = ops.layer_norm_backward(dy, x, mean, rstd)
    assert dw is None and db is None
    one = torch.ones(64, device="cuda", dtype=torch.bfloat16)
    dx1, dw1, db1 = ops.layer_norm_backward(dy, x, mean, rstd, one)
    assert torch.equal(dx, dx1)
    assert torch.equal(ops.layer_norm_backward(dy, x, mean, rstd, one, param_grads=False)[0], dx)
    a = ops.layer_norm_backward(dy.reshape(-1, 64), x.reshape(-1, 64), fm, fr, one)
    assert torch.equal(a[0], dx.reshape(-1, 64)) and torch.equal(a[1], dw1) and torch.equal(a[2], db1)


def test_layer_norm_constant_rows_and_non_finite_rows(torch, ops):
    """A constant row gives its bias; a row with a NaN or an infinity stays alone with it."""
    x = torch.full((4, 96), 3.0, device="cuda")
    x[1] = torch.randn(96, device="cuda")
    x[2, 5] = float("nan")
    x[3, 7] = float("inf")
    b = torch.randn(96, device="cuda")
    y, mean, rstd = ops.layer_norm(x, torch.ones(96, device="cuda"), b)
    assert torch.equal(y[0], b)
    assert torch.isfinite(y[1]).all() and torch.isnan(y[2]).all() and not torch.isfinite(y[3]).any()


def test_layer_norm_gradient_against_differences(torch, ops):
    gen = gen_for(torch, 9)
    x, v = normal(torch, gen, 6, 320), normal(torch, gen, 6, 320)
    w, b, c = normal(torch, gen, 320), normal(torch, gen, 320), normal(torch, gen, 6, 320)
    vw, vb = normal(torch, gen, 320), normal(torch, gen, 320)
    h = 2.0 ** -8   # error of the difference: h^2 times the third derivative, and 2^-24 / h of the values

    def loss(s):
        return (ops.layer_norm(x + s * v, w + s * vw, b + s * vb)[0].double() * c.double()).sum()

    y, mean, rstd = ops.layer_norm(x, w, b)
    dx, dw, db = ops.layer_norm_backward(c, x, mean, rstd, w)
    got = (dx.double() * v.double()).sum() + (dw.double() * vw.double()).sum() + (db.double() * vb.double()).sum()
    diff = (loss(h) - loss(-h)) / (2 * h)
    scale = (y.abs().double() * c.abs().double()).sum()
    assert abs(got - diff) <= scale * (2.0 ** -24 * 8 / h + 40 * h * h), (got, diff, scale)


# --------------------------------------------------------------------------- rows by expert

def plan_ref(torch, ids, experts):
    """Counting sort in Python: offsets, rank."""
    flat = ids.reshape(-1).cpu().tolist()
    lists = [[] for _ in range(experts)]
    for s, e in enumerate(flat):
        if 0 <= e < experts:
            lists[e].append(s)
    rank, offsets, at = [-1] * len(flat), [0], 0
    for l in lists:
        for s in l:
            rank[s] = at
            at += 1
        offsets.append(at)
    return torch.tensor(offsets, dtype=torch.int32), torch.tensor(rank, dtype=torch.int32).reshape(ids.shape)


SORTS = [(1, 1, 1), (1, 8, 384), (16, 8, 384), (63, 1, 2), (64, 1, 1), (65, 2, 5), (511, 1, 7), (513, 8, 64), (512, 8, 16),
         (4099, 6, 64), (700, 6, 1024), (8192, 8, 384), (30000, 5, 1000), (3000, 3, 1), (0, 2, 4)]


@pytest.mark.parametrize("ids_type", ["int32", "int64"])
@pytest.mark.parametrize("shape", SORTS, ids=str)
def test_expert_sort(torch, ops, shape, ids_type):
    tokens, k, experts = shape
    gen = gen_for(torch, tokens + k)
    ids = torch.randint(-2, experts + 2, (tokens, k), generator=gen, device="cuda").to(getattr(torch, ids_type))
    if tokens > 4:
        ids[2] = ids[3]                      # the same experts again
        ids[tokens // 2] = -1                # a padded token
        if ids_type == "int64":
            ids[1, 0] = (1 << 32)            # expert 0 in its lower half: still nobody's
    offsets, rank = ops.expert_sort(ids, experts)
    ro, rr = plan_ref(torch, ids, experts)
    assert offsets.dtype == torch.int32 and rank.dtype == torch.int32
    assert torch.equal(offsets.cpu(), ro) and torch.equal(rank.cpu(), rr)


def test_expert_sort_one_expert_takes_all_and_none_takes_any(torch, ops):
    for tokens in (100, 5000):
        ids = torch.full((tokens, 2), 3, device="cuda", dtype=torch.int32)
        offsets, rank = ops.expert_sort(ids, 5)
        assert offsets.tolist() == [0, 0, 0, 0, 2 * tokens, 2 * tokens]
        assert torch.equal(rank.reshape(-1).cpu(), torch.arange(2 * tokens, dtype=torch.int32))
        offsets, rank = ops.expert_sort(torch.full_like(ids, -1), 5)
        assert offsets.tolist() == [0] * 6 and (rank == -1).all()


ROWS = [  # tokens, k, experts, cols, columns behind each row, first element
    (1, 1, 1, 1, 0, 0), (1, 8, 384, 7168, 0, 0), (16, 8, 384, 7168, 0, 0), (5, 2, 3, 8, 0, 0), (33, 6, 64, 2048, 8, 8),
    (40, 3, 7, 65, 0, 0), (12, 9, 16, 136, 0, 0), (7, 17, 30, 24, 1, 0), (1030, 4, 10, 20, 0, 1), (300, 6, 64, 1024, 0, 0),
    (3000, 2, 4, 72, 0, 0), (0, 2, 4, 64, 0, 0),
]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("shape", ROWS, ids=str)
def test_dispatch_combine_and_gradients(torch, ops, shape, dtype):
    tokens, k, experts, cols, pad, shift = shape
    dt = getattr(torch, dtype)
    gen = gen_for(torch, tokens * 7 + cols)
    ids = torch.randint(0, experts, (tokens, k), generator=gen, device="cuda", dtype=torch.int32)
    if tokens > 2:
        ids[tokens // 3] = -1
        ids[tokens - 1, 0] = experts
    offsets, rank = ops.expert_sort(ids, experts)
    slots, kept = tokens * k, int(offsets[-1])
    x = buffer(torch, gen, dt, tokens, cols, pad, shift)
    out = buffer(torch, gen, dt, slots, cols, pad, shift).fill_(float("nan"))
    xs = ops.expert_dispatch(x, rank, offsets, out=out)
    t, j = torch.nonzero(rank >= 0, as_tuple=True)
    at = rank[t, j].long()
    ref = torch.zeros(slots, cols, dtype=dt, device="cuda")
    ref[at] = x[t]
    assert torch.equal(xs, ref)
    # its gradient: NaN in the rows of nobody must not reach a token
    dxs = buffer(torch, gen, dt, slots, cols, pad, shift)
    dxs[kept:] = float("nan")
    dx = ops.expert_dispatch_backward(dxs, rank)
    zero = torch.zeros(tokens, cols, dtype=torch.float64, device="cuda")
    ref = zero.clone().index_add_(0, t, dxs[at].double())
    mag = zero.clone().index_add_(0, t, dxs[at].double().abs())
    close(dx, ref, k * 2.0 ** -24 * mag, "dx")
    for wdt in {dt, torch.float32}:
        w = normal(torch, gen, tokens, k).to(wdt)
        w[rank < 0] = float("nan")
        y = ops.expert_combine(dxs, w, rank)
        wd = w[t, j].double()[:, None]
        ref = zero.clone().index_add_(0, t, dxs[at].double() * wd)
        mag = zero.clone().index_add_(0, t, (dxs[at].double() * wd).abs())
        close(y, ref, 2 * k * 2.0 ** -24 * mag, "y")
        dy = buffer(torch, gen, dt, tokens, cols, pad, shift)
        out.fill_(float("nan"))
        dys, dw = ops.expert_combine_backward(dy, dxs, w, rank, offsets, out=out)
        ref = torch.zeros(slots, cols, dtype=torch.float64, device="cuda")
        ref[at] = dy[t].double() * wd
        close(dys, ref, 2.0 ** -24 * ref.abs(), "dys")
        ref, mag = torch.zeros(tokens, k, dtype=torch.float64, device="cuda"), torch.zeros(tokens, k, dtype=torch.float64, device="cuda")
        prod = dy[t].double() * dxs[at].double()
        ref[t, j], mag[t, j] = prod.sum(dim=1), prod.abs().sum(dim=1)
        assert dw.dtype == wdt
        close(dw, ref, adds(cols) * 2.0 ** -24 * mag, "dweights")


def test_ranks_out_of_range_are_no_rows(torch, ops):
    """A rank buffer that expert_sort did not write: what is out of range counts as no row."""
    x = torch.randn(6, 64, device="cuda")
    rank = torch.tensor([[0, 99], [-5, 1], [2, 12], [3, -2 ** 31], [2 ** 31 - 1, 4], [5, -1]], dtype=torch.int32, device="cuda")
    offsets = torch.tensor([0, 6, 6], dtype=torch.int32, device="cuda")
    xs = ops.expert_dispatch(x, rank, offsets)
    assert torch.equal(xs[:6], x) and not xs[6:].any()
    assert torch.equal(ops.expert_dispatch_backward(xs, rank), x)
    dys, dw = ops.expert_combine_backward(x, xs, torch.ones(6, 2, device="cuda"), rank, offsets)
    assert torch.equal(dys, xs)
    assert ((dw != 0) == ((rank >= 0) & (rank < 12))).all()


# ------------------------------------------------------------------------------- products

PRODUCTS = [  # rows per expert, rows of nobody, N, K
    ([1], 0, 1, 1), ([6], 0, 64, 64), ([1, 1, 0, 1], 0, 136, 264), ([3, 0, 5], 2, 17, 33), ([130, 0, 127, 1], 3, 128, 128),
    ([257, 128, 0, 300], 40, 264, 520), ([40, 70], 0, 65, 130), ([0, 0, 0], 9, 72, 64), ([1000], 0, 256, 2048),
    ([300, 20, 600, 0, 77], 5, 520, 776), ([5, 2, 9, 1, 0, 3], 0, 1408, 2048), ([33] * 40, 0, 128, 192), ([700, 411], 1, 1000, 264),
    ([64, 3], 0, 2047, 1021), ([513, 255, 256, 1, 0, 31], 7, 768, 1096),
]


def make_product(torch, gen, dt, counts, rest, n, k, pad=0, shift=0):
    rows = sum(counts) + rest
    x = buffer(torch, gen, dt, rows, k, pad, shift)
    dy = buffer(torch, gen, dt, rows, n, pad, shift)
    w = buffer(torch, gen, dt, len(counts) * n, k, pad, shift)
    w = w.as_strided((len(counts), n, k), (n * w.stride(0), w.stride(0), 1), w.storage_offset())
    offsets = torch.tensor([0] + counts, device="cuda").cumsum(0).to(torch.int32)
    return x, dy, w, offsets


def check_product(torch, ops, x, dy, w, counts, offsets):
    rows, n, k = x.shape[0], w.shape[1], w.shape[2]
    y = ops.expert_matmul(x, w, offsets)
    dx, dw = ops.expert_matmul_backward(dy, x, w, offsets)
    u = 2.0 ** -23
    at = 0
    for e, c in enumerate(counts):
        a, g, m = x[at:at + c].double(), dy[at:at + c].double(), w[e].double()
        close(y[at:at + c], a @ m.T, (k + 2) * u * (a.abs() @ m.abs().T), f"y of expert {e}")
        close(dx[at:at + c], g @ m, (n + 2) * u * (g.abs() @ m.abs()), f"dx of expert {e}")
        close(dw[e], g.T @ a, (c + 2) * u * (g.abs().T @ a.abs()), f"dw of expert {e}")
        at += c
    assert not y[at:].any() and not dx[at:].any()


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("case", PRODUCTS, ids=lambda c: f"{len(c[0])}x{sum(c[0])}+{c[1]}_{c[2]}x{c[3]}")
def test_expert_products(torch, ops, case, dtype):
    counts, rest, n, k = case
    gen = gen_for(torch, n + k)
    x, dy, w, offsets = make_product(torch, gen, getattr(torch, dtype), counts, rest, n, k)
    x[sum(counts):] = float("nan")           # rows of nobody are not read into anything
    dy[sum(counts):] = float("nan")
    check_product(torch, ops, x, dy, w, counts, offsets)


def uneven(experts, most, seed, empty=5):
    """Row counts 0 .. most, every empty-th expert without rows."""
    import torch
    c = torch.randint(0, most + 1, (experts,), generator=torch.Generator().manual_seed(seed))
    c[::empty] = 0
    return c.tolist()


# many experts: half a chip of 256 x 256 tiles and more, several a workgroup; contractions of one
# chunk, one stage, a stage and a bit, an odd and an even number of stages
MANY = [
    (uneven(70, 600, 1), 3, 264, 8), (uneven(70, 300, 2), 0, 520, 64), (uneven(90, 300, 3), 300, 392, 72), (uneven(40, 500, 4), 5, 1032, 200),
    (uneven(33, 200, 5), 0, 2048, 256), (uneven(200, 40, 6), 1, 136, 1096), (uneven(1024, 3, 7), 2, 264, 136), ([0] * 20 + [9000] + [0] * 19, 9, 256, 328),
    ([256] * 130, 0, 256, 320), ([0] * 150, 700, 144, 160), (uneven(150, 130, 8, 2), 0, 144, 160),
]


@pytest.mark.parametrize("dtype", ["bfloat16", "float16"])
@pytest.mark.parametrize("case", MANY, ids=lambda c: f"{len(c[0])}x{sum(c[0])}+{c[1]}_{c[2]}x{c[3]}")
def test_expert_products_of_many_experts(torch, ops, case, dtype):
    counts, rest, n, k = case
    gen = gen_for(torch, n + k)
    x, dy, w, offsets = make_product(torch, gen, getattr(torch, dtype), counts, rest, n, k, pad=8)
    x[sum(counts):] = float("nan")
    dy[sum(counts):] = float("nan")
    check_product(torch, ops, x, dy, w, counts, offsets)


def test_expert_products_write_nothing_outside(torch, ops):
    """Strided results: the columns behind each row and the rows around stay as they were."""
    gen = gen_for(torch, 12)
    for counts, n, k in (([40, 0, 70], 72, 136), (uneven(60, 300, 9), 264, 328)):
        rows = sum(counts)
        x, dy, w, offsets = make_product(torch, gen, torch.bfloat16, counts, 0, n, k)
        for call, r, c in ((lambda o: ops.expert_matmul(x, w, offsets, out=o), rows, n),
                           (lambda o: ops.expert_matmul_grad_input(dy, w, offsets, out=o), rows, k)):
            full = torch.full((r + 4, c + 16), 7.0, dtype=torch.bfloat16, device="cuda")
            got = call(full[2:-2, 8:-8]).clone()
            full[2:-2, 8:-8] = 7.0
            assert (full == 7.0).all() and torch.equal(got, call(None))
        full = torch.full((len(counts), n + 4, k + 16), 7.0, dtype=torch.bfloat16, device="cuda")
        got = ops.expert_matmul_grad_weight(dy, x, offsets, out=full[:, 2:-2, 8:-8]).clone()
        full[:, 2:-2, 8:-8] = 7.0
        assert (full == 7.0).all() and torch.equal(got, ops.expert_matmul_grad_weight(dy, x, offsets))


@pytest.mark.parametrize("dtype", DTYPES)
def test_no_rows_at_all(torch, ops, dtype):
    dt = getattr(torch, dtype)
    for experts in (3, 200):
        w = torch.randn(experts, 136, 264, device="cuda").to(dt)
        off = torch.zeros(experts + 1, dtype=torch.int32, device="cuda")
        x, dy = torch.empty(0, 264, dtype=dt, device="cuda"), torch.empty(0, 136, dtype=dt, device="cuda")
        assert ops.expert_matmul(x, w, off).shape == (0, 136)
        dx, dw = ops.expert_matmul_backward(dy, x, w, off)
        assert dx.shape == (0, 264) and dw.shape == w.shape and not dw.any()


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("pad,shift", [(8, 0), (3, 0), (8, 1), (0, 8), (1, 3)])
def test_expert_products_strided_and_unaligned(torch, ops, dtype, pad, shift):
    gen = gen_for(torch, 3)
    counts = [70, 0, 200, 1]
    x, dy, w, offsets = make_product(torch, gen, getattr(torch, dtype), counts, 4, 264, 328, pad, shift)
    check_product(torch, ops, x, dy, w, counts, offsets)


NARROW = [(1, 9), (3, 8), (4, 4), (5, 7), (7, 5), (8, 3), (9, 1), (9, 17), (12, 31), (130, 15), (15, 130), (257, 33), (33, 2067),
          (300, 5), (301, 261)]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("counts,rest", [([2, 0, 1], 1), ([17, 0, 3, 40], 0), ([70, 0, 130], 2), ([400, 0, 390], 1)], ids=str)
@pytest.mark.parametrize("n,k", NARROW)
def test_expert_products_of_rows_shorter_than_a_load(torch, ops, n, k, counts, rest, dtype):
    """Widths around 16 bytes and rows that begin at any element, their neighbours not finite."""
    dt = getattr(torch, dtype)
    gen = gen_for(torch, 31 * n + k)

    def rows(r, c):                    # a base one element into the storage, one column behind each row
        flat = torch.full((r * (c + 1) + 2,), float("nan"), device="cuda", dtype=dt)
        out = flat[1:1 + r * (c + 1)].view(r, c + 1)[:, :c]
        out.copy_(normal(torch, gen, r, c))
        return out
    total = sum(counts) + rest
    x, dy, w = rows(total, k), rows(total, n), rows(len(counts) * n, k)
    w = w.as_strided((len(counts), n, k), (n * w.stride(0), w.stride(0), 1), w.storage_offset())
    offsets = torch.tensor([0] + counts, device="cuda").cumsum(0).to(torch.int32)
    check_product(torch, ops, x, dy, w, counts, offsets)


@pytest.mark.parametrize("dtype", ["bfloat16", "float16"])
def test_expert_products_at_model_widths(torch, ops, dtype):
    """27 experts of 2048 x 7168, skewed, with one empty: the sizes a card of the 216-expert layer holds."""
    gen = gen_for(torch, 8)
    counts = torch.randint(1, 120, (27,), generator=torch.Generator().manual_seed(1)).tolist()
    counts[4], counts[9] = 0, 700
    x, dy, w, offsets = make_product(torch, gen, getattr(torch, dtype), counts, 11, 2048, 7168)
    check_product(torch, ops, x, dy, w, counts, offsets)


def test_expert_products_keep_non_finite_values_in_place(torch, ops):
    """An infinity in one row of one expert reaches that row, and that expert's weight gradient, alone."""
    gen = gen_for(torch, 4)
    x, dy, w, offsets = make_product(torch, gen, torch.bfloat16, [40, 50, 60], 0, 72, 136)
    x[45, 3] = float("inf")
    y = ops.expert_matmul(x, w, offsets)
    ok = torch.isfinite(y).all(dim=1)
    assert not ok[45] and ok.sum() == 149
    dw = ops.expert_matmul_grad_weight(dy, x, offsets)
    bad = ~torch.isfinite(dw)
    assert bad[1, :, 3].all() and bad.sum() == 72


def test_offsets_out_of_range_are_cut(torch, ops):
    x = torch.randn(10, 64, device="cuda")
    w = torch.randn(3, 64, 64, device="cuda")
    whole = ops.expert_matmul(x, w, torch.tensor([0, 4, 4, 10], dtype=torch.int32, device="cuda"))
    cut = ops.expert_matmul(x, w, torch.tensor([-3, 4, 4, 99], dtype=torch.int32, device="cuda"))
    assert torch.equal(whole, cut)
    back = torch.tensor([0, 10, 4, 10], dtype=torch.int32, device="cuda")   # expert 1 ends before it begins
    assert not ops.expert_matmul_grad_weight(x, x, back)[1].any()
    xs = ops.expert_dispatch(x[:5], torch.full((5, 2), -1, dtype=torch.int32, device="cuda"),
                             torch.tensor([0, -7], dtype=torch.int32, device="cuda"))
    assert not xs.any()


def test_offsets_in_no_order_write_nothing_outside(torch, ops):
    """Experts that share rows: the results are unspecified, what lies around them stays."""
    gen = gen_for(torch, 14)
    for rows, n, k, dt in ((10, 64, 64, torch.float32), (300, 264, 328, torch.bfloat16), (700, 520, 136, torch.float16), (900, 130, 70, torch.bfloat16)):
        for raw in ([0, rows] * 9, [rows // 2, rows, 3, -5, rows + 9, 0, rows], [2 ** 31 - 1, -2 ** 31, 5, 4, 3, 2 ** 31 - 1, 0, 7]):
            off = torch.tensor(raw, dtype=torch.int32, device="cuda")
            w = normal(torch, gen, len(raw) - 1, n, k).to(dt)
            x, dy = normal(torch, gen, rows, k).to(dt), normal(torch, gen, rows, n).to(dt)
            for call, r, c in ((lambda o: ops.expert_matmul(x, w, off, out=o), rows, n),
                               (lambda o: ops.expert_matmul_grad_input(dy, w, off, out=o), rows, k)):
                full = torch.full((r + 4, c + 16), 7.0, dtype=dt, device="cuda")
                call(full[2:-2, 8:-8])
                full[2:-2, 8:-8] = 7.0
                assert (full == 7.0).all()
            dw = ops.expert_matmul_grad_weight(dy, x, off)   # each expert's own rows, shared or not
            for e, (lo, hi) in enumerate(zip(raw, raw[1:])):
                lo = min(max(lo, 0), rows)
                hi = min(max(hi, lo), rows)
                g, a = dy[lo:hi].double(), x[lo:hi].double()
                close(dw[e], g.T @ a, (hi - lo + 2) * 2.0 ** -23 * (g.abs().T @ a.abs()), f"dw of expert {e}")


def test_row_buffers_past_32_bits(torch, ops):
    """40000 tokens of 7168 with 8 picks: the row side holds 2.3e9 elements."""
    gen = gen_for(torch, 6)
    tokens, k, cols, experts = 40000, 8, 7168, 3
    x = normal(torch, gen, tokens, cols).to(torch.bfloat16)
    ids = torch.randint(0, experts, (tokens, k), generator=gen, device="cuda", dtype=torch.int32)
    ids[7] = -1
    offsets, rank = ops.expert_sort(ids, experts)
    xs = ops.expert_dispatch(x, rank, offsets)
    assert xs.numel() > 2 ** 31
    for t in (0, 6, 8, tokens - 1):
        assert (xs[rank[t].long()] == x[t]).all()
    assert not xs[-8:].any()
    w8 = torch.full((tokens, k), 0.125, device="cuda")
    y = ops.expert_combine(xs, w8, rank)
    keep = torch.arange(tokens, device="cuda") != 7
    assert torch.equal(y[keep], x[keep]) and not y[7].any()
    assert torch.equal(ops.expert_dispatch_backward(xs, rank)[keep], 8 * x[keep])
    dys, dw = ops.expert_combine_backward(x, xs, w8, rank, offsets)
    assert torch.equal(dys[:-8], (xs[:-8].float() * 0.125).to(torch.bfloat16))
    del dys, y
    w = normal(torch, gen, experts, 72, cols).to(torch.bfloat16)
    out = ops.expert_matmul(xs, w, offsets)
    for s in (0, int(offsets[1]), int(offsets[2]) + 5, int(offsets[-1]) - 1):
        e = int((offsets[1:] <= s).sum())
        a, m = xs[s].double(), w[e].double()
        close(out[s], m @ a, (cols + 2) * 2.0 ** -23 * (m.abs() @ a.abs()), f"row {s}")
    dwt = ops.expert_matmul_grad_weight(out, xs, offsets)
    lo = int(offsets[2])
    g, a = out[lo:, :8].double(), xs[lo:, -64:].double()
    close(dwt[2, :8, -64:], g.T @ a, (g.shape[0] + 2) * 2.0 ** -23 * (g.abs().T @ a.abs()), "dw")
    del xs, x
    dx = ops.expert_matmul_grad_input(out, w, offsets)
    for s in (3, int(offsets[2]) + 5, int(offsets[-1]) - 1):
        e = int((offsets[1:] <= s).sum())
        g, m = out[s].double(), w[e].double()
        close(dx[s], g @ m, 74 * 2.0 ** -23 * (g.abs() @ m.abs()), f"dx row {s}")


def test_more_threads_than_a_grid_dimension_holds(torch, ops):
    """A workgroup per token of 2^24 tokens, and a thread per element of 2^22 x 1025 that begin anywhere."""
    gen = gen_for(torch, 8)
    tokens, experts = 1 << 24, 5
    x = normal(torch, gen, tokens, 1)
    ids = torch.randint(-1, experts, (tokens, 1), generator=gen, device="cuda", dtype=torch.int32)
    offsets, rank = ops.expert_sort(ids, experts)
    some = (ids >= 0).view(-1)
    at = rank.view(-1).long()[some]
    xs = ops.expert_dispatch(x, rank, offsets)
    assert torch.equal(xs[at], x[some]) and not xs[int(offsets[-1]):].any()
    w = normal(torch, gen, tokens, 1)
    y = ops.expert_combine(xs, w, rank)
    assert torch.equal(y[some], (w * x)[some]) and not y[~some].any()
    dys, dw = ops.expert_combine_backward(x, xs, w, rank, offsets)
    assert torch.equal(dys[at], (w * x)[some]) and not dys[int(offsets[-1]):].any()
    assert torch.equal(dw[some], (x * x)[some]) and not dw[~some].any()
    del x, xs, w, y, dys, dw

    tokens, cols = 1 << 22, 1025
    x = torch.arange(tokens, device="cuda", dtype=torch.int32).to(torch.bfloat16).view(-1, 1).expand(tokens, cols).contiguous()
    offsets, rank = ops.expert_sort(ids[:tokens], experts)
    xs = ops.expert_dispatch(x, rank, offsets)
    some = (ids[:tokens] >= 0).view(-1)
    at = rank.view(-1).long()[some]
    for c in (0, cols - 1):
        assert torch.equal(xs[:, c][at], x[:, c][some]) and not xs[int(offsets[-1]):, c].any()
    dx = ops.expert_dispatch_backward(xs, rank)
    for c in (0, cols - 1):
        assert torch.equal(dx[:, c][some], x[:, c][some]) and not dx[:, c][~some].any()


def test_layer_norm_past_32_bits(torch, ops):
    rows, cols = 300000, 7168
    x = torch.zeros(rows, cols, dtype=torch.bfloat16, device="cuda")
    x[-1] = torch.randn(cols, device="cuda").to(torch.bfloat16)
    x[5] = x[-1]
    w, b = torch.ones(cols, device="cuda"), torch.zeros(cols, device="cuda")
    y, mean, rstd = ops.layer_norm(x, w, b)
    assert torch.equal(y[5], y[-1]) and y[-1].any() and not y[6:-1].any()
    dx, dw, db = ops.layer_norm_backward(y, x, mean, rstd, w)
    assert torch.equal(dx[5], dx[-1]) and torch.equal(db, 2 * y[5].float())


@pytest.mark.parametrize("dtype", DTYPES)
def test_halves_of_one_buffer_as_input_and_output(torch, ops, dtype):
    """Columns of one wider buffer, and every other matrix of one batch, on both sides of a call."""
    dt = getattr(torch, dtype)
    gen = gen_for(torch, 15)
    for rows, cols, e in ((70, 64, 3), (301, 33, 2), (2000, 264, 5)):
        both = lambda r: normal(torch, gen, r, 2 * cols).to(dt)
        buf = both(rows)
        x = buf[:, :cols].clone()
        y, mean, rstd = ops.layer_norm(buf[:, :cols], out=buf[:, cols:])
        assert torch.equal(y, ops.layer_norm(x)[0]) and torch.equal(buf[:, :cols], x)
        buf = both(rows)
        dy, want = buf[:, cols:].clone(), ops.layer_norm_backward(buf[:, cols:].clone(), x, mean, rstd)[0]
        assert torch.equal(ops.layer_norm_backward(buf[:, cols:], x, mean, rstd, out=buf[:, :cols])[0], want) and torch.equal(buf[:, cols:], dy)
        off = torch.linspace(0, rows, e + 1, device="cuda").to(torch.int32)
        w = normal(torch, gen, e, cols, cols).to(dt)
        buf = both(rows)
        x, want = buf[:, :cols].clone(), ops.expert_matmul(buf[:, :cols].clone(), w, off)
        assert torch.equal(ops.expert_matmul(buf[:, :cols], w, off, out=buf[:, cols:]), want) and torch.equal(buf[:, :cols], x)
        want = ops.expert_matmul_grad_input(x, w, off)
        assert torch.equal(ops.expert_matmul_grad_input(buf[:, :cols], w, off, out=buf[:, cols:]), want) and torch.equal(buf[:, :cols], x)
        with pytest.raises(RuntimeError, match="MNS_ERR_ARG"):
            ops.expert_matmul(buf[:, :cols], w, off, out=buf[:, cols - 1:-1])
        ids = torch.randint(-1, e, (rows, 1), generator=gen, device="cuda", dtype=torch.int32)
        offsets, rank = ops.expert_sort(ids, e)
        want = ops.expert_dispatch(x, rank, offsets)
        assert torch.equal(ops.expert_dispatch(buf[:, :cols], rank, offsets, out=buf[:, cols:]), want) and torch.equal(buf[:, :cols], x)
        pairs = normal(torch, gen, 3, 2, rows, cols).to(dt)
        x = pairs[:, 0].clone()
        assert torch.equal(ops.layer_norm(pairs[:, 0], out=pairs[:, 1])[0], ops.layer_norm(x)[0]) and torch.equal(pairs[:, 0], x)


# ------------------------------------------------------------------------- streams, graphs

def layer_inputs(torch, dt, seed=2, tokens=200, k=4, experts=10, dim=256, inner=192):
    gen = gen_for(torch, seed)
    s = {"x": normal(torch, gen, tokens, dim).to(dt), "nw": (1 + 0.1 * normal(torch, gen, dim)).to(dt), "nb": (0.1 * normal(torch, gen, dim)).to(dt),
         "router": normal(torch, gen, dim, experts) * dim ** -0.5, "up": (normal(torch, gen, experts, inner, dim) * dim ** -0.5).to(dt),
         "down": (normal(torch, gen, experts, dim, inner) * inner ** -0.5).to(dt), "c": normal(torch, gen, tokens, dim).to(dt), "k": k,
         "experts": experts}
    picks = torch.topk(normal(torch, gen, tokens, experts), k, dim=1)
    s["ids"], s["weights"] = picks.indices, torch.softmax(picks.values, dim=1)
    s["ids"][tokens - 9:] = -1
    return s


def layer_pass(ops, s, ws=None):
    """Norm, dispatch, up, square of the positive part, down, combine; then every gradient for the loss sum(c y)."""
    h, mean, rstd = ops.layer_norm(s["x"], s["nw"], s["nb"])
    offsets, rank = ops.expert_sort(s["ids"], s["experts"], workspace=None if ws is None else ws[0])
    xs = ops.expert_dispatch(h, rank, offsets)
    up = ops.expert_matmul(xs, s["up"], offsets)
    act = up.clamp(min=0).square()
    ys = ops.expert_matmul(act, s["down"], offsets)
    y = ops.expert_combine(ys, s["weights"], rank)
    dys, dweights = ops.expert_combine_backward(s["c"], ys, s["weights"], rank, offsets)
    dact, ddown = ops.expert_matmul_backward(dys, act, s["down"], offsets)
    dup = dact * 2 * up.clamp(min=0)
    dxs, dw_up = ops.expert_matmul_backward(dup, xs, s["up"], offsets)
    dh = ops.expert_dispatch_backward(dxs, rank)
    dx, dnw, dnb = ops.layer_norm_backward(dh, s["x"], mean, rstd, s["nw"], workspace=None if ws is None else ws[1])
    return y, dweights, ddown, dw_up, dx, dnw, dnb


def test_the_layer_against_autograd_in_64_bits_and_its_gradients_in_the_optimizer(torch, ops):
    s = layer_inputs(torch, torch.float32)
    got = layer_pass(ops, s)
    leaf = {n: s[n].double().cpu().requires_grad_() for n in ("x", "nw", "nb", "up", "down", "weights")}
    h = (leaf["x"] - leaf["x"].mean(1, keepdim=True))
    h = h / torch.sqrt((h * h).mean(1, keepdim=True) + 1e-5) * leaf["nw"] + leaf["nb"]
    rows = []
    for t, ids in enumerate(s["ids"].cpu().tolist()):
        acc = torch.zeros(h.shape[1], dtype=torch.float64)
        for j, e in enumerate(ids):
            if e >= 0:
                acc = acc + leaf["weights"][t, j] * (leaf["down"][e] @ (leaf["up"][e] @ h[t]).clamp(min=0).square())
        rows.append(acc)
    y = torch.stack(rows)
    (y * s["c"].double().cpu()).sum().backward()
    want = (y.detach(), leaf["weights"].grad, leaf["down"].grad, leaf["up"].grad, leaf["x"].grad, leaf["nw"].grad, leaf["nb"].grad)
    for name, a, r in zip(("y", "dweights", "ddown", "dup", "dx", "dnorm_w", "dnorm_b"), got, want):
        e = float((a.double().cpu() - r).norm() / r.norm())
        say(f"layer {name}: rel {e:.2e}")
        # a chain of six fp32 sums of at most 800 terms of random sign: 6 sqrt(800) 2^-23, and as much again for the
        # square's slope
        assert e < 4e-5, name
    # the gradients go into the optimizer as they are
    mats = [(s["up"].clone(), got[3], torch.zeros_like(s["up"])), (s["down"].clone(), got[2], torch.zeros_like(s["down"]))]
    vecs = [(s["nw"].clone(), got[5], torch.zeros(256, device="cuda"), torch.zeros(256, device="cuda"))]
    before = mats[0][0].clone()
    ops.hybrid_step(mats, vecs, muon=dict(lr=0.02, momentum=0.95, weight_decay=0.1), adamw=dict(lr=1e-3))
    assert torch.isfinite(mats[0][0]).all() and torch.isfinite(mats[1][0]).all() and torch.isfinite(vecs[0][0]).all()
    moved = (mats[0][0] - before).flatten(1).norm(dim=1)
    assert (moved > 0).all()


@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
def test_the_layer_is_deterministic_on_any_stream_and_in_a_graph(torch, ops, dtype):
    s = layer_inputs(torch, getattr(torch, dtype), tokens=1100)   # sort on several workgroups
    want = [t.clone() for t in layer_pass(ops, s)]
    again = layer_pass(ops, s)
    assert all(torch.equal(a, b) for a, b in zip(want, again))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        other = layer_pass(ops, s)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, other))
    ws = [torch.empty(ops.expert_sort_workspace_bytes(s["ids"].numel(), s["experts"]), dtype=torch.uint8, device="cuda"),
          torch.empty(ops.layer_norm_workspace_bytes(s["x"]), dtype=torch.uint8, device="cuda")]
    with torch.cuda.stream(side):
        layer_pass(ops, s, ws)
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = layer_pass(ops, s, ws)
    x0, ids0 = s["x"].clone(), s["ids"].clone()
    for i in range(4):
        s["x"].copy_(x0 if i % 2 == 0 else x0.flip(0))
        s["ids"].copy_(ids0 if i % 2 == 0 else ids0.flip(0))
        graph.replay()
        torch.cuda.synchronize()
        eager = layer_pass(ops, s)
        assert all(torch.equal(a, b) for a, b in zip(held, eager)), i
