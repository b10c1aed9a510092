"""The layer's kernels where a workgroup takes more than one row or tile: the rows fetched ahead and the two
reduction buffers of the norm's gradients, the walk of the products' tile lists, and products past 2^31 elements.
Checked as in test_gpu_layer.py, with its tolerances."""
import pytest

from test_gpu_layer import (DTYPES, adds, check_product, close, gen_for, make_product, normal, ops,  # noqa: F401 (fixtures)
                            test_layer_norm_and_gradient as check_norm, torch, uneven)

pytestmark = pytest.mark.gpu

# rows, cols, columns behind each row, first element: each variant by length, several rows a workgroup (the first alone
# has one), rows of whole 16-byte chunks and rows that begin anywhere
NORM = [
    (5, 768, 0, 0), (2500, 1024, 0, 0), (4500, 1000, 8, 8), (2500, 1021, 1, 1), (5000, 513, 0, 3),
    (700, 1536, 0, 0), (2300, 2048, 0, 0), (1500, 1500, 0, 0), (1600, 1503, 0, 0), (1200, 3000, 0, 0), (1200, 2999, 2, 0), (600, 4096, 8, 0),
    (1100, 7168, 0, 0), (1100, 7165, 0, 1), (700, 8192, 0, 8), (600, 8200, 0, 0), (600, 8201, 3, 0), (1500, 12000, 0, 0), (700, 12001, 0, 0),
    (520, 16384, 0, 0), (600, 16392, 0, 0), (1100, 16395, 1, 0),
]


@pytest.mark.parametrize("wide", [False, True], ids=["own", "fp32w"])
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("shape", NORM, ids=str)
def test_norm_of_several_rows_a_workgroup(torch, ops, shape, dtype, wide):
    check_norm(torch, ops, shape, dtype, wide)


def test_norm_gradients_past_32_bits(torch, ops):
    rows, cols = 300000, 7168
    gen = gen_for(torch, 21)
    x = torch.empty(rows, cols, dtype=torch.bfloat16, device="cuda")
    dy = torch.empty_like(x)
    for lo in range(0, rows, 20000):
        x[lo:lo + 20000] = normal(torch, gen, 20000, cols).to(x.dtype)
        dy[lo:lo + 20000] = normal(torch, gen, 20000, cols).to(x.dtype)
    w = 1 + 0.1 * normal(torch, gen, cols)
    _, mean, rstd = ops.layer_norm(x, w)
    dx, dw, db = ops.layer_norm_backward(dy, x, mean, rstd, w)
    sums = torch.zeros(4, cols, dtype=torch.float64, device="cuda")
    for lo in range(0, rows, 20000):
        m, r = mean[lo:lo + 20000].double()[:, None], rstd[lo:lo + 20000].double()[:, None]
        g, a = dy[lo:lo + 20000].double(), x[lo:lo + 20000].double()
        sums += torch.stack([(g * (a - m) * r).sum(0), (g.abs() * (a.abs() + m.abs()) * r).sum(0), g.sum(0), g.abs().sum(0)])
    # a column's sum: a workgroup of 512 adds up every 512th row, then 32 parts a wave and 16 waves
    u = (rows / 512 + 32 + 16 + 40) * 2.0 ** -24
    close(dw, sums[0], u * sums[1], "dweight")
    close(db, sums[2], u * sums[3], "dbias")
    at = torch.tensor([0, 511, 512, 149999, 299487, 299488, rows - 1], device="cuda")
    m, r = mean[at].double()[:, None], rstd[at].double()[:, None]
    xh, g = (x[at].double() - m) * r, dy[at].double() * w.double()
    ref = r * (g - g.mean(1, keepdim=True) - xh * (g * xh).mean(1, keepdim=True))
    ga, xa = g.abs(), (x[at].double().abs() + m.abs()) * r
    close(dx[at], ref, adds(cols) * 2.0 ** -24 * r * (ga + ga.mean(1, keepdim=True) * (1 + 2 * xa.amax(1, keepdim=True) ** 2)), "dx")


# counts, rows of nobody, N, K, columns behind each row, first element. Rows that begin anywhere take 128 x 128 tiles: more
# than 1000 of them for at most 512 workgroups, experts of several bands of eight tile rows, and few tiles (split ones)
LOOPS = [
    (uneven(64, 300, 11), 5, 1405, 1421, 1, 1), ([5000, 17, 0, 1400, 3003], 3, 1405, 1333, 0, 0), (uneven(300, 100, 12), 0, 333, 525, 3, 0),
    ([65] * 8, 1, 1341, 523, 1, 0), (uneven(16, 200, 13), 0, 1405, 1021, 0, 3),
]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("case", LOOPS, ids=lambda c: f"{len(c[0])}x{sum(c[0])}+{c[1]}_{c[2]}x{c[3]}")
def test_products_of_several_tiles_a_workgroup(torch, ops, case, dtype):
    counts, rest, n, k, pad, shift = case
    x, dy, w, offsets = make_product(torch, gen_for(torch, n + k), getattr(torch, dtype), counts, rest, n, k, pad, shift)
    x[sum(counts):] = float("nan")
    dy[sum(counts):] = float("nan")
    check_product(torch, ops, x, dy, w, counts, offsets)


# the same with whole 16-byte chunks: fp32 tiles of both kinds
ALIGNED = [(uneven(64, 300, 14), 5, 1408, 1424), ([5000, 17, 0, 1400, 3003], 3, 1408, 1336), (uneven(16, 200, 15), 0, 1408, 1024)]


@pytest.mark.parametrize("case", ALIGNED, ids=lambda c: f"{len(c[0])}x{sum(c[0])}+{c[1]}_{c[2]}x{c[3]}")
def test_fp32_products_of_several_tiles_a_workgroup(torch, ops, case):
    counts, rest, n, k = case
    x, dy, w, offsets = make_product(torch, gen_for(torch, n + k), torch.float32, counts, rest, n, k)
    x[sum(counts):] = float("nan")
    dy[sum(counts):] = float("nan")
    check_product(torch, ops, x, dy, w, counts, offsets)


def test_products_past_32_bits(torch, ops):
    """320000 rows of 7168 against experts of 264 x 7168: the 256 x 256 tiles on operands and results past 2^31 elements."""
    gen = gen_for(torch, 22)
    rows, n, k = 320000, 264, 7168
    offsets = torch.tensor([0, 100001, 100001, 250000, rows - 7], dtype=torch.int32, device="cuda")
    x = torch.empty(rows, k, dtype=torch.bfloat16, device="cuda")
    for lo in range(0, rows, 20000):
        x[lo:lo + 20000] = normal(torch, gen, 20000, k).to(x.dtype)
    assert x.numel() > 2 ** 31
    w = normal(torch, gen, 4, n, k).to(torch.bfloat16)
    y = ops.expert_matmul(x, w, offsets)
    assert not y[-7:].any()
    bounds = offsets.tolist()
    rows_of = torch.tensor([0, 100000, 100001, 249999, 250000, 299594, 299595, rows - 8], device="cuda")   # 2^31 elements end in row 299593
    expert = [sum(s >= b for b in bounds[1:]) for s in rows_of.tolist()]
    for s, e in zip(rows_of.tolist(), expert):
        a, m = x[s].double(), w[e].double()
        close(y[s], m @ a, (k + 2) * 2.0 ** -23 * (m.abs() @ a.abs()), f"row {s}")
    dw = ops.expert_matmul_grad_weight(y, x, offsets)
    assert not dw[1].any()
    for e in (0, 2, 3):
        lo, hi = bounds[e], bounds[e + 1]
        for r, c in ((slice(0, 16), slice(0, 64)), (slice(n - 16, n), slice(k - 64, k))):
            g, a = y[lo:hi, r].double(), x[lo:hi, c].double()
            close(dw[e, r, c], g.T @ a, (hi - lo + 2) * 2.0 ** -23 * (g.abs().T @ a.abs()), f"dw of expert {e}")
    dx = ops.expert_matmul_grad_input(y, w, offsets, out=x)
    assert not dx[-7:].any()
    for s, e in zip(rows_of.tolist(), expert):
        g, m = y[s].double(), w[e].double()
        close(dx[s], g @ m, (n + 2) * 2.0 ** -23 * (g.abs() @ m.abs()), f"dx row {s}")
