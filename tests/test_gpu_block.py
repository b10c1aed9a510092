"""Rms norm, token embeddings and AdamW in 8 bits against their definitions in 64 bits.

Tolerances: a result is rounded once to its type, at most half a step (eps / 2 of its value, for e4m3 2^-4 or half of its
smallest step 2^-9); the fp32 sums before it are off by at most (number of additions) x 2^-24 x the sum of the terms'
magnitudes. Copies, powers of two and the order of sums are exact.
"""
import math

import pytest

from test_gpu_layer import DTYPES, adds, buffer, close, gen_for, normal, ops, torch  # noqa: F401 (fixtures)

pytestmark = pytest.mark.gpu

U = 2.0 ** -24

# --------------------------------------------------------------------------------- rms norm

# rows, cols, columns behind each row, first element: each kernel by length, rows that begin anywhere, rows shorter than a load,
# several rows a workgroup in the backward pass
RMS = [
    (1, 1, 0, 0), (1, 7168, 0, 0), (3, 3, 0, 0), (5, 7, 2, 1), (5, 8, 0, 0), (9, 9, 0, 0), (17, 64, 8, 0), (64, 200, 0, 8), (65, 511, 0, 1),
    (33, 512, 0, 0), (2500, 1021, 1, 1), (1030, 264, 0, 0), (65, 2047, 0, 0), (2300, 2048, 0, 0), (129, 2056, 0, 0), (7, 2048, 3, 1),
    (700, 3001, 0, 0), (600, 4096, 8, 0), (1100, 7168, 0, 0), (9, 7168, 16, 8), (600, 7165, 0, 1), (4, 8200, 0, 0), (520, 12001, 0, 0),
    (3, 16384, 0, 0), (2, 16385, 0, 0), (600, 16395, 1, 0), (2, 33000, 0, 0), (2, 70001, 1, 3), (0, 64, 0, 0), (5000, 24, 0, 0), (700, 2, 0, 1),
]


def rms_inputs(torch, shape, dtype, wide):
    rows, cols, pad, shift = shape
    dt = getattr(torch, dtype)
    gen = gen_for(torch, rows * 31 + cols)
    x, r, dy, dh = (buffer(torch, gen, dt, rows, cols, pad, shift) for _ in range(4))
    w = (1 + 0.1 * normal(torch, gen, cols)).to(torch.float32 if wide else dt)
    return x, r, dy, dh, w


def rms_ref(torch, h, w, eps):
    h = h.double()
    rstd = (h.square().mean(dim=-1) + eps).rsqrt()
    return h * rstd[..., None] * w.double(), rstd


@pytest.mark.parametrize("wide", [False, True], ids=["own", "fp32w"])
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("shape", RMS, ids=str)
def test_rms_norm_and_gradient(torch, ops, shape, dtype, wide):
    x, r, dy, dh, w = rms_inputs(torch, shape, dtype, wide)
    rows, cols = x.shape
    y, h, rstd = ops.rms_norm(x, w, residual=r, eps=1e-6)
    dx, dw = ops.rms_norm_backward(dy, h, rstd, w, dh=dh)
    torch.cuda.synchronize()
    assert y.shape == h.shape == dx.shape == x.shape and dw.dtype == w.dtype and rstd.dtype == torch.float32
    assert torch.equal(h, (x.float() + r.float()).to(x.dtype))
    if rows == 0:
        assert not dw.any()
        return
    ref, rrstd = rms_ref(torch, h, w, 1e-6)
    u = adds(cols) * U
    close(rstd, rrstd, rrstd * u, "rstd")
    close(y, ref, ref.abs() * (u + 3 * U), "y")
    # without a residual x is h; without a weight 1
    y1, h1, rstd1 = ops.rms_norm(h, w, eps=1e-6)
    assert h1 is h and torch.equal(y1, y) and torch.equal(rstd1, rstd)
    # the gradients from the kept statistic, as the call takes it
    rs = rstd.double()[:, None]
    xh, g = h.double() * rs, dy.double() * w.double()
    part = rs * (g.abs() + xh.abs() * (g * xh).abs().mean(dim=1, keepdim=True))
    ref = rs * (g - xh * (g * xh).mean(dim=1, keepdim=True))
    close(dx, ref + dh.double(), (u + 4 * U) * part + U * dh.double().abs(), "dx")
    close(ops.rms_norm_backward(dy, h, rstd, w)[0], ref, (u + 4 * U) * part, "dx without a stream")
    close(dw, (dy.double() * xh).sum(dim=0), (rows + 40) * U * (dy.double() * xh).abs().sum(dim=0), "dweight")


def decoded(torch, q, scales):
    wide = scales.double().repeat_interleave(32, dim=-1)[..., :q.shape[-1]]
    return q.double() * wide


@pytest.mark.parametrize("wide", [False, True], ids=["own", "fp32w"])
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("shape", RMS, ids=str)
def test_rms_norm_in_8_bits(torch, ops, shape, dtype, wide):
    x, r, _, _, w = rms_inputs(torch, shape, dtype, wide)
    rows, cols = x.shape
    if rows > 4:
        x[1], r[1] = 0, 0                                     # a row of zeros
        x[2] = torch.where(torch.arange(cols, device="cuda") % 64 < 32, x[2], torch.zeros((), device="cuda", dtype=x.dtype))
        r[2] = 0                                              # blocks of zeros
    q, scales, h, rstd = ops.rms_norm_mx8(x, w, residual=r, eps=1e-6)
    assert q.dtype == torch.float8_e4m3fn and scales.dtype == torch.float8_e8m0fnu and scales.shape == (rows, -(-cols // 32))
    y, h1, rstd1 = ops.rms_norm(x, w, residual=r, eps=1e-6)
    assert torch.equal(h, h1) and torch.equal(rstd, rstd1)
    if rows == 0:
        return
    ref, _ = rms_ref(torch, h, w, 1e-6)
    off = (adds(cols) + 3) * U
    top = torch.nn.functional.pad(ref.abs(), (0, -cols % 32)).view(rows, -1, 32).amax(dim=2)
    s = scales.double()
    byte = scales.view(torch.uint8)
    assert (top * (1 - off) <= 448 * s).all() and ((top * (1 + off) > 224 * s) | (byte == 0)).all()
    assert (byte[top == 0] == 0).all()
    wide_s = s.repeat_interleave(32, dim=1)[:, :cols]
    half = torch.maximum(ref.abs() * 2.0 ** -4, wide_s * 2.0 ** -10)
    assert ((decoded(torch, q, scales) - ref).abs() <= half * (1 + off) + off * ref.abs()).all()


def test_rms_norm_8_bit_codes_are_the_nearest(torch, ops):
    """Ties to even and every exponent, from rows whose norm is known: 64 values of +-1 scaled by the weight (eps 0)."""
    codes = torch.arange(0, 127, device="cuda", dtype=torch.uint8).view(torch.float8_e4m3fn).float()   # 0 .. 448
    mid = (codes[:-1] + codes[1:]) / 2                        # halfway: the even code
    for lo in range(0, 126, 31):
        v = torch.cat([mid[lo:lo + 31], torch.full((1,), 448.0, device="cuda")])
        w = torch.cat([v, torch.zeros(64 - v.numel(), device="cuda")])
        x = torch.ones(1, 64, device="cuda")
        q, s, _, rstd = ops.rms_norm_mx8(x, w, eps=0.0)
        assert rstd.item() == 1 and s.view(torch.uint8)[0, 0] == 127
        assert torch.equal(q[0, :v.numel()].float(), v.to(torch.float8_e4m3fn).float())
    # 448 2^k fits its block's power, the next fp32 number does not
    for k in (-40, 0, 40):
        w = torch.full((64,), 2.0 ** -60, device="cuda")
        w[0] = 448.0 * 2.0 ** k
        w[32] = torch.nextafter(w[0], w.new_tensor(math.inf))
        s = ops.rms_norm_mx8(torch.ones(1, 64, device="cuda"), w, eps=0.0)[1].view(torch.uint8)[0].tolist()
        assert s == [127 + k, 128 + k]


def test_rms_norm_non_finite_and_zero_rows(torch, ops):
    x = torch.randn(5, 96, device="cuda")
    x[1, 5] = float("nan")
    x[2, 7] = float("inf")
    x[3] = 0
    y, _, rstd = ops.rms_norm(x)
    assert torch.isnan(y[1]).all() and rstd[2] == 0 and torch.isnan(y[2, 7]) and not y[2, :7].any()
    assert not y[3].any() and torch.isfinite(y[[0, 4]]).all()
    # in 8 bits a value that is not finite is a NaN and leaves its block alone
    w = torch.ones(96, device="cuda")
    w[40], w[41] = float("inf"), float("nan")
    q, s, _, _ = ops.rms_norm_mx8(x[:1], w)
    q1, s1, _, _ = ops.rms_norm_mx8(x[:1], torch.where(torch.isfinite(w), w, torch.zeros((), device="cuda")))
    bad = torch.isnan(q.float())[0]
    assert bad.nonzero()[:, 0].tolist() == [40, 41]
    assert torch.equal(q.float()[0][~bad], q1.float()[0][~bad]) and torch.equal(s.view(torch.uint8), s1.view(torch.uint8))


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("cols", [40, 1000, 7168, 8191, 20001])
def test_rms_norm_in_place_strided_and_batched(torch, ops, cols, dtype):
    dt = getattr(torch, dtype)
    gen = gen_for(torch, cols)
    base = normal(torch, gen, 2, 9, cols + 7).to(dt)
    x, stream = base[:, 1:8, :cols], normal(torch, gen, 2, 9, cols + 3).to(dt)
    r = stream[:, 1:8, 3:]
    w = normal(torch, gen, cols).to(dt)
    y, h, rstd = ops.rms_norm(x, w, residual=r.clone())
    assert rstd.shape == (2, 7)
    q, s, _, _ = ops.rms_norm_mx8(x, w, residual=r.clone())
    for call in ("rms_norm", "rms_norm_mx8"):
        held = stream.clone()
        part = held[:, 1:8, 3:]
        got = getattr(ops, call)(x, w, residual=part, residual_out=part)
        assert got[-2] is part and torch.equal(part, h)
        part.copy_(r)
        assert torch.equal(held, stream)                      # nothing outside was written
        if call == "rms_norm":
            assert torch.equal(got[0], y)
        else:
            assert torch.equal(got[0].view(torch.uint8), q.view(torch.uint8)) and torch.equal(got[1].view(torch.uint8), s.view(torch.uint8))
    full = torch.full((2, 9, cols + 2), 7.0, dtype=dt, device="cuda")
    assert torch.equal(ops.rms_norm(x, w, residual=r, out=full[:, 1:8, 1:-1])[0], y)
    dy, dh = normal(torch, gen, 2, 7, cols).to(dt), normal(torch, gen, 2, 7, cols).to(dt)
    dx, dw = ops.rms_norm_backward(dy, h, rstd, w, dh=dh)
    dx1, dw1 = ops.rms_norm_backward(dy, h, rstd, w, dh=dh, out=dh)
    assert dx1 is dh and torch.equal(dx, dh) and torch.equal(dw, dw1)
    full[:, 1:8, 1:-1] = 7.0
    ops.rms_norm_backward(dy, h, rstd, w, out=full[:, 1:8, 1:-1])
    full[:, 1:8, 1:-1] = 7.0
    assert (full == 7.0).all()
    assert ops.rms_norm_backward(dy, h, rstd)[1] is None and ops.rms_norm_backward(dy, h, rstd, w, param_grads=False)[1] is None


def test_rms_norm_gradient_against_differences(torch, ops):
    gen = gen_for(torch, 9)
    x, r, v, c, d = (normal(torch, gen, 6, 320) for _ in range(5))
    w, vw = normal(torch, gen, 320), normal(torch, gen, 320)
    step = 2.0 ** -8   # error of the difference: step^2 times the third derivative, and 2^-24 / step of the values

    def loss(s):
        y, h, _ = ops.rms_norm(x + s * v, w + s * vw, residual=r)
        return (y.double() * c.double()).sum() + (h.double() * d.double()).sum()

    y, h, rstd = ops.rms_norm(x, w, residual=r)
    dx, dw = ops.rms_norm_backward(c, h, rstd, w, dh=d)
    got = (dx.double() * v.double()).sum() + (dw.double() * vw.double()).sum()
    diff = (loss(step) - loss(-step)) / (2 * step)
    scale = (y.abs().double() * c.abs().double()).sum() + (h.abs().double() * d.abs().double()).sum()
    assert abs(got - diff) <= scale * (U * 8 / step + 40 * step * step), (got, diff, scale)


def test_rms_norm_past_32_bits(torch, ops):
    rows, cols = 300000, 7168
    x = torch.zeros(rows, cols, dtype=torch.bfloat16, device="cuda")
    x[-1] = torch.randn(cols, device="cuda").to(torch.bfloat16)
    x[5] = x[-1]
    w = torch.ones(cols, device="cuda")
    y, h, rstd = ops.rms_norm(x, w, residual=x, eps=1e-6)
    assert torch.equal(h[-1], 2 * x[-1]) and torch.equal(y[5], y[-1]) and y[-1].any() and not y[6:-1].any()
    del x
    q, s, _, _ = ops.rms_norm_mx8(h, w)
    assert torch.equal(q[5].view(torch.uint8), q[-1].view(torch.uint8)) and torch.equal(s[5].view(torch.uint8), s[-1].view(torch.uint8))
    assert not q[6:-1].view(torch.uint8).any()
    dx, dw = ops.rms_norm_backward(y, h, rstd, w, dh=y)
    assert torch.equal(dx[5], dx[-1]) and dx[-1].any()


def test_rms_norm_of_more_rows_than_a_grid_dimension(torch, ops):
    rows = 1 << 24
    x = torch.arange(1, rows + 1, device="cuda", dtype=torch.float32)[:, None]
    y, _, rstd = ops.rms_norm(x, eps=0.0)
    assert ((y - 1).abs() <= 4 * U).all()
    dx, _ = ops.rms_norm_backward(y, x, rstd, dh=x)
    assert ((dx - x).abs() <= 8 * U * (1 + x)).all()          # the norm of one column does not move


# ------------------------------------------------------------------------------- embeddings

# tokens, vocabulary, cols, columns behind each row, first element
EMBED = [
    (1, 1, 1, 0, 0), (1, 163840, 64, 0, 0), (5, 3, 7, 0, 0), (31, 40, 8, 0, 0), (32, 40, 3, 1, 1), (33, 2, 4, 0, 1), (64, 1, 65, 0, 0), (65, 300, 2047, 0, 0),
    (100, 70000, 24, 8, 8), (1000, 1000, 512, 0, 0), (4099, 1023, 513, 0, 3), (4099, 1024, 128, 0, 0), (4096, 8191, 40, 0, 0), (4097, 70000, 12, 0, 8), (16384, 8191, 40, 0, 0),
    (16385, 8191, 40, 0, 0), (50000, 120, 33, 3, 0), (70000, 1100000, 9, 0, 0), (0, 50, 64, 0, 0), (3000, 5, 1024, 0, 0), (300000, 300, 2, 0, 0),
]


def token_ids(torch, gen, n, vocab, dtype):
    """Tokens of falling frequency, with padding and ids outside the vocabulary among them."""
    rank = torch.exp(torch.rand(n, generator=gen, device="cuda", dtype=torch.float64) * math.log(vocab + 1)).long().clamp(1, vocab) - 1
    if n > 4:
        rank[n // 2], rank[n // 3], rank[-1] = -1, vocab, -2 ** 31
        if dtype == torch.int64:
            rank[1] = 1 << 32                # token 0 in its lower half: still nobody's
    return rank.to(dtype)


@pytest.mark.parametrize("ids", ["int32", "int64"])
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("shape", EMBED, ids=str)
def test_embed_and_gradient(torch, ops, shape, dtype, ids):
    n, vocab, cols, pad, shift = shape
    dt = getattr(torch, dtype)
    gen = gen_for(torch, n + cols)
    tokens = token_ids(torch, gen, n, vocab, getattr(torch, ids))
    have = (tokens >= 0) & (tokens < vocab)
    table = buffer(torch, gen, dt, vocab, cols, pad, shift)
    scale = math.sqrt(cols)
    y = ops.embed(tokens, table, scale=scale)
    ref = torch.zeros(n, cols, device="cuda", dtype=dt)
    ref[have] = (table[tokens[have].long()].float() * torch.tensor(scale, device="cuda")).to(dt)
    assert torch.equal(y, ref)
    dy = buffer(torch, gen, dt, n, cols, pad, shift)
    dy[~have] = float("nan")                 # the gradient at padding reaches nothing
    out = buffer(torch, gen, dt, vocab, cols, pad, shift).fill_(float("nan"))
    got = ops.embed_backward(dy, tokens, vocab, scale=scale, out=out)
    assert got is out
    ref = torch.zeros(vocab, cols, dtype=torch.float64, device="cuda")
    mag, count = ref.clone(), torch.zeros(vocab, 1, dtype=torch.float64, device="cuda")
    at, rows = tokens[have].long(), dy[have].double()
    ref.index_add_(0, at, rows)
    mag.index_add_(0, at, rows.abs())
    count.index_add_(0, at, torch.ones(at.numel(), 1, dtype=torch.float64, device="cuda"))
    # a token of c rows: c additions at most (tiles of 32, then the tiles' parts), and the scale's product
    s32 = float(torch.tensor(scale))
    close(got, ref * s32, (count + 4) * U * mag * s32, "dtable")
    again = ops.embed_backward(dy, tokens, vocab, scale=scale)
    assert torch.equal(again, got)


@pytest.mark.parametrize("n", [10, 1000, 20000, 90000])
def test_embed_gradient_counts_exactly(torch, ops, n):
    """Whole numbers: every row reaches its token once, whatever runs of a token do at the ends of tiles."""
    gen = gen_for(torch, n)
    kinds = [torch.zeros(n), torch.arange(n) % 7, torch.arange(n) // 32, torch.arange(n) // 33, torch.arange(n) // 31, torch.arange(n) // 64,
             torch.arange(n) // 1000, torch.arange(n).flip(0), torch.where(torch.arange(n) < n // 2, 3, 2 ** 20)]
    for tokens in kinds:
        tokens = tokens.long().cuda()
        tokens = tokens[torch.randperm(n, generator=gen, device="cuda")]
        vocab = int(tokens.max()) + 2
        dy = torch.randint(-8, 9, (n, 5), generator=gen, device="cuda").float()
        ref = torch.zeros(vocab, 5, dtype=torch.float64, device="cuda").index_add_(0, tokens, dy.double())
        assert torch.equal(ops.embed_backward(dy, tokens, vocab).double(), ref)


@pytest.mark.parametrize("n", [32736, 32737, 70001])
def test_embed_gradient_counts_long_runs_exactly(torch, ops, n):
    """Runs of a token over whole groups of 64 tiles, that begin and end anywhere in a group."""
    gen = gen_for(torch, n)
    at = torch.arange(n, device="cuda")
    for run, first in ((2048, 0), (2048, 1), (2047, 0), (2049, 31), (2079, 0), (2080, 32), (4095, 32), (4128, 2016), (6200, 33), (30000, 2047), (n, 0), (n - 1, n - 1)):
        tokens = (at + (run - first)) // run
        tokens = tokens[torch.randperm(n, generator=gen, device="cuda")]
        vocab = int(tokens.max()) + 1
        dy = torch.randint(-8, 9, (n, 3), generator=gen, device="cuda").float()
        ref = torch.zeros(vocab, 3, dtype=torch.float64, device="cuda").index_add_(0, tokens, dy.double())
        assert torch.equal(ops.embed_backward(dy, tokens, vocab).double(), ref)


@pytest.mark.parametrize("vocab", [3, (1 << 24) - 1])
def test_embed_gradient_of_the_most_positions(torch, ops, vocab):
    """2^24 positions of one column: sums of whole numbers below 2^24, which fp32 holds."""
    n = 1 << 24
    gen = gen_for(torch, vocab)
    tokens = torch.randint(0, vocab, (n,), generator=gen, device="cuda", dtype=torch.int32)
    dy = torch.randint(0, 2, (n, 1), generator=gen, device="cuda").float()
    ref = torch.bincount(tokens, weights=dy[:, 0].double(), minlength=vocab)
    assert torch.equal(ops.embed_backward(dy, tokens, vocab)[:, 0].double(), ref)


def test_embed_shapes_out_and_nothing_outside(torch, ops):
    gen = gen_for(torch, 3)
    table = normal(torch, gen, 50, 72).to(torch.bfloat16)
    tokens = torch.randint(-1, 51, (3, 5), generator=gen, device="cuda")
    y = ops.embed(tokens, table)
    assert y.shape == (3, 5, 72) and torch.equal(y.view(15, 72), ops.embed(tokens.view(-1), table))
    assert ops.embed(tokens[0, 0], table).shape == (72,)
    full = torch.full((19, 90), 7.0, dtype=torch.bfloat16, device="cuda")
    assert torch.equal(ops.embed(tokens, table, out=full[2:-2, 8:-10]), y.view(15, 72))
    full[2:-2, 8:-10] = 7.0
    assert (full == 7.0).all()
    dy = normal(torch, gen, 3, 5, 72).to(torch.bfloat16)
    dt = ops.embed_backward(dy, tokens, 50, scale=0.5)
    full = torch.full((54, 90), 7.0, dtype=torch.bfloat16, device="cuda")
    ws = torch.empty(ops.embed_workspace_bytes(15, 50, 72), dtype=torch.uint8, device="cuda").fill_(255)
    assert torch.equal(ops.embed_backward(dy.view(15, 72), tokens, 50, scale=0.5, out=full[2:-2, 8:-10], workspace=ws), dt)
    full[2:-2, 8:-10] = 7.0
    assert (full == 7.0).all()
    # no token at all: nothing but zeros
    assert not ops.embed_backward(dy[:0].view(0, 72), tokens[:0].reshape(0), 50).any()
    assert not ops.embed_backward(dy, torch.full_like(tokens, -1), 50).any()
    assert not ops.embed(torch.full_like(tokens, 50), table).any()


def test_embed_past_32_bits(torch, ops):
    vocab, cols = 320000, 7168                # 2.3e9 elements
    table = torch.zeros(vocab, cols, dtype=torch.bfloat16, device="cuda")
    gen = gen_for(torch, 4)
    some = normal(torch, gen, 3, cols).to(torch.bfloat16)
    at = torch.tensor([0, 299999, vocab - 1], device="cuda")
    table[at] = some
    assert torch.equal(ops.embed(at, table), some)
    del table
    dt = ops.embed_backward(some, at, vocab, scale=2.0)
    assert torch.equal(dt[at], 2 * some)
    dt[at] = 0
    assert not dt.view(torch.int16).any()
    del dt
    tokens = torch.arange(vocab, device="cuda") % 1000
    y = ops.embed(tokens, some.repeat(400, 1))
    assert torch.equal(y[-1], some[999 % 3]) and torch.equal(y[299999], some[999 % 3]) and torch.equal(y[301000], some[0])
    ones = y.fill_(1)
    dt = ops.embed_backward(ones, tokens, 1000)
    assert (dt == 320).all()


# ----------------------------------------------------------------------------- AdamW, 8 bits

def mix(x):
    x = x ^ (x >> 16)
    x = (x * 0x3dd219bf) & 0xffffffff
    x = x ^ (x >> 15)
    x = (x * 0xafd7c8e5) & 0xffffffff
    return x ^ (x >> 16)


def random_bits(torch, seed, step, place, n):
    key = mix(mix(mix(mix(seed & 0xffffffff) ^ (seed >> 32)) ^ step) ^ place)
    i = torch.arange(n, device="cuda")
    x = mix((i * 0xdf50e7c3 + key) & 0xffffffff)
    return x & 0xffff, x >> 16


def state_values(torch, codes, scales):
    return decoded(torch, codes.view(torch.float8_e4m3fn).view(1, -1), scales.view(torch.float8_e8m0fnu).view(1, -1))[0]


def check_adamw8(torch, p0, g, s0, p1, s1, hp, place, dtype):
    """One step of one tensor from its inputs' copies; hp as ops.adamw8_step takes them."""
    f32 = lambda v: float(torch.tensor(v, dtype=torch.float32))
    lr, b1, b2, eps = (f32(hp[k]) for k in ("lr", "beta1", "beta2", "eps"))
    c1, c2, keep = f32(1 - hp["beta1"]), f32(1 - hp["beta2"]), f32(1 - hp["lr"] * hp["weight_decay"])
    n = p0.numel()
    if n == 0:
        return
    p0, g = p0.double(), g.double()
    m0, r0 = state_values(torch, s0[0], s0[1]), state_values(torch, s0[2], s0[3])
    m, v = b1 * m0 + c1 * g, b2 * r0 ** 2 + c2 * g ** 2
    r = v.sqrt()
    fix = (1 - hp["beta1"] ** hp["step"], math.sqrt(1 - hp["beta2"] ** hp["step"])) if hp["bias_correction"] else (1.0, 1.0)
    dm = 4 * U * (b1 * m0.abs() + c1 * g.abs()) + 1e-38
    upd = (m / fix[0]) / (r / fix[1] + eps)
    # r: three roundings under the root, halved, and the root's own; the quotient three more
    slack = 4 * U * (keep * p0.abs() + lr * upd.abs()) + lr * (dm / fix[0] / (r / fix[1] + eps) + 8 * U * upd.abs())
    close(p1, keep * p0 - lr * upd, slack, "parameter")
    rm, rr = random_bits(torch, hp["seed"], hp["step"], place, n)
    for name, val, off, codes, scales, rnd, least in (("m", m, dm, s1[0], s1[1], rm, 0.0), ("r", r, 4 * U * r + 1e-38, s1[2], s1[3], rr, 2.0 ** -9)):
        top = torch.nn.functional.pad(val.abs(), (0, -n % 32)).view(-1, 32).amax(dim=1)
        s = scales.view(torch.float8_e8m0fnu).double()
        byte = scales.view(torch.uint8)
        assert (top * (1 - 8 * U) <= 448 * s).all() and ((top * (1 + 8 * U) > 224 * s) | (byte == 0)).all(), name
        s = s.repeat_interleave(32)[:n]
        x = val.abs() / s
        _, e = torch.frexp(x)
        step = torch.exp2((e - 1).clamp(min=-6).double() - 3)
        got = codes.view(torch.float8_e4m3fn).double().abs()
        want = torch.floor(x / step + rnd.double() / 65536) * step
        want = torch.where((val != 0) & (want < least), torch.full_like(want, least), want)
        # only a number that lands within the fp32 errors of a whole step may go either way
        near = x / step + rnd.double() / 65536
        free = (near - near.round()).abs() <= (off / s) / step + 2.0 ** -20
        assert ((got == want) | (free & ((got - want).abs() <= step))).all(), (name, int((got != want).sum()))
        assert ((codes.view(torch.float8_e4m3fn).double().sign() == val.sign()) | (got == 0)).all()


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("correct", [False, True])
def test_adamw8_of_many_tensors_and_steps(torch, ops, dtype, correct):
    """More tensors than one launch's table, of any length and alignment, over three steps from zero states."""
    dt = getattr(torch, dtype)
    gen = gen_for(torch, 21)
    sizes = [0, 1, 7, 8, 31, 32, 33, 4095, 4096, 4097, 100_003] + [5, 300, 64] * 20
    base = normal(torch, gen, sum(sizes) + 3 * len(sizes) + 8).to(dt)
    ps, at = [], 1
    for n in sizes:                          # views that begin anywhere, three elements apart
        ps.append(base[at:at + n])
        at += n + 3
    outside = torch.ones(base.numel(), dtype=torch.bool, device="cuda")
    at = 1
    for n in sizes:
        outside[at:at + n] = False
        at += n + 3
    kept = base[outside].clone()
    states = [ops.adamw8_state(p) for p in ps]
    for step in (1, 2, 3):
        gs = [(normal(torch, gen, n) * 10.0 ** (i % 9 - 6)).to(dt) for i, n in enumerate(sizes)]
        if step == 2:
            gs[10][:5000] = 0                # moments that only decay
            gs[9].zero_()
        before = [(p.clone(), [t.clone() for t in s]) for p, s in zip(ps, states)]
        hp = dict(lr=3e-3, beta1=0.9, beta2=0.95, eps=1e-8, weight_decay=0.1, step=step, bias_correction=correct, seed=0x123456789abcdef + step)
        ops.adamw8_step(ps, gs, states, **hp)
        for i, ((p0, s0), g, p, s) in enumerate(zip(before, gs, ps, states)):
            check_adamw8(torch, p0, g, s0, p, s, hp, i, dt)
    assert torch.equal(base[outside], kept)


def test_adamw8_fp32_states_follow_the_formula_bit_for_bit(torch, ops):
    """Every operation of the moments rounded to fp32 as torch's are: no rounding goes to another code, in millions of elements."""
    gen = gen_for(torch, 22)
    n = 3_000_000
    p = normal(torch, gen, n)
    state = ops.adamw8_state(p)
    scale = 10.0 ** (torch.arange(n, device="cuda") // 32 % 7 - 6)
    for step in (1, 2, 3, 4):
        g = normal(torch, gen, n) * scale
        held = [state_values(torch, state[i], state[i + 1]).float() for i in (0, 2)]
        ops.adamw8_step([p], [g], [state], lr=1e-3, step=step, beta1=0.9, beta2=0.95, seed=77)
        m = 0.9 * held[0] + (1 - 0.9) * g
        r = torch.sqrt(0.95 * held[1].square() + (1 - 0.95) * (g * g))
        for val, i, rnd, least in zip((m, r), (0, 2), random_bits(torch, 77, step, 0, n), (0.0, 2.0 ** -9)):
            byte = state[i + 1].view(torch.uint8).repeat_interleave(32)[:n]
            x = (val.abs().double() * torch.exp2(127 - byte.double())).float()
            fine = torch.floor(x.double() * 512 + rnd.double() * 2.0 ** -16) * 2.0 ** -9
            size = torch.where(x < 2.0 ** -6, fine.float(), ((x.view(torch.int32) + (rnd.int() << 4)) & ~0xfffff).view(torch.float32))
            size = torch.where((val != 0) & (size < least), torch.full_like(size, least), size)
            got = state[i].view(torch.float8_e4m3fn).float().abs()
            # below 2^-6 the number is added to 2^-6 first, one rounding more: at most one in 10^5 of them ends elsewhere
            off = got != size
            assert not (off & (x >= 2.0 ** -6)).any() and off.sum() <= 1 + 1e-5 * (x < 2.0 ** -6).sum(), int(off.sum())


def test_adamw8_moments_keep_their_mean(torch, ops):
    """A million elements of one value: the states' mean follows the recursion, also where a step's change is below
    half a code (r decays by 2.5 % a step without gradients; the nearest code would never move)."""
    n = 1 << 20
    p = torch.zeros(n, device="cuda")
    s = ops.adamw8_state(p)
    g = torch.full((n,), 0.37, device="cuda")
    m = r2 = 0.0
    for step in range(1, 21):
        if step == 6:
            g.zero_()
        ops.adamw8_step([p], [g], [s], lr=1e-3, beta1=0.95, beta2=0.95, step=step, seed=5)
        x = float(g[0])
        m, r2 = 0.95 * m + 0.05 * x, 0.95 * r2 + 0.05 * x * x
        # the rounding of each step is off by at most a step of the code, 1/8 of the value, of random sign: a mean of 2^20 of
        # them by less than 6 / 8 / 2^10 of it, some steps of it left in the moment (1 / (1 - beta) = 20); r^2 gains the variance
        # of r's roundings, at most 1/256 of it a step, and loses 5 % of it
        assert abs(float(state_values(torch, s[0], s[1]).mean()) / m - 1) < 20 * 6 / 8 / 1024, step
        got = float(state_values(torch, s[2], s[3]).square().mean())
        assert -0.02 < got / r2 - 1 < 1.06 * 20 / 256, (step, got, r2)


def test_adamw8_values_that_are_not_finite_and_tiny_gradients(torch, ops):
    n = 96
    p = torch.ones(n, device="cuda")
    s = ops.adamw8_state(p)
    g = torch.full((n,), 1e-3, device="cuda")
    g[5], g[40] = float("nan"), float("inf")
    ops.adamw8_step([p], [g], [s], lr=1e-3, step=1)
    bad = torch.isnan(p)
    assert bad[5] and bad[40] and bad.sum() == 2              # inf / inf
    for codes, scales in ((s[0], s[1]), (s[2], s[3])):
        v = state_values(torch, codes, scales)
        assert torch.isnan(v).nonzero()[:, 0].tolist() == [5, 40] and (v[~bad] > 0).all()
    # an element far below its block's largest keeps a root that is not zero, and its step stays bounded
    p, g = torch.zeros(32, device="cuda"), torch.full((32,), 1e-9, device="cuda")
    g[0] = 1.0
    s = ops.adamw8_state(p)
    ops.adamw8_step([p], [g], [s], lr=1e-3, step=1)
    assert (s[2].float() > 0).all()
    for step in range(2, 40):
        before = p.clone()
        ops.adamw8_step([p], [torch.zeros_like(g)], [s], lr=1e-3, weight_decay=0.0, step=step)
        assert ((p - before).abs() <= 1e-3 * 3).all()         # m / r: m of a smallest code is 2^-9 times a power at most m's top / 224


def test_adamw8_beside_adamw_and_in_the_hybrid_step(torch, ops):
    """One step from the same zero state gives adamw_step's parameters; entries of both kinds in one hybrid step."""
    gen = gen_for(torch, 8)
    p = normal(torch, gen, 5000).to(torch.bfloat16)
    g = (1e-3 * normal(torch, gen, 5000)).to(torch.bfloat16)
    a, b = p.clone(), p.clone()
    hp = dict(lr=1e-2, step=1, bias_correction=True)
    m, v, s = torch.zeros(5000, device="cuda"), torch.zeros(5000, device="cuda"), ops.adamw8_state(p)
    ops.adamw_step([a], [g], [m], [v], **hp)
    ops.adamw8_step([b], [g], [s], **hp)
    assert ((a.float() - b.float()).abs() <= a.float().abs() * 2.0 ** -7).all() and (a != b).float().mean() < 0.01
    c, d = p.clone(), p.clone()
    W = normal(torch, gen, 2, 64, 96).to(torch.bfloat16)
    states = [torch.zeros(5000, device="cuda"), torch.zeros(5000, device="cuda"), ops.adamw8_state(p)]
    ops.hybrid_step([(W, W.clone(), torch.zeros(2, 64, 96, device="cuda"))], [(c, g, states[0], states[1]), (d, g, states[2])],
                    muon=dict(lr=0.02, momentum=0.95, weight_decay=0.1), adamw=hp)
    assert torch.equal(c, a) and torch.equal(d, b) and torch.equal(states[2][0].view(torch.uint8), s[0].view(torch.uint8))
    ops.hybrid_step([], [(d, g, states[2])], muon={}, adamw=dict(hp, step=2), seed=3)
    assert torch.isfinite(d).all()


def test_adamw8_past_32_bits(torch, ops):
    """2^32 + 100 elements: places past 32 bits have random numbers of their own."""
    n = 2 ** 32 + 100
    p = torch.ones(n, dtype=torch.bfloat16, device="cuda")
    g = torch.full((n,), 0.37, dtype=torch.bfloat16, device="cuda")
    s = ops.adamw8_state(p)
    ops.adamw8_step([p], [g], [s], lr=0.5, weight_decay=0.0, step=1)
    assert (p[-200:] == p[0]).all() and p[0] != 1
    codes = s[0].view(torch.uint8)
    assert len(codes[-96:].unique()) <= 2 and len(s[1].view(torch.uint8)[-4:].unique()) == 1 and s[1].view(torch.uint8)[-1] == s[1].view(torch.uint8)[0]
    low, high = codes[:96], codes[2 ** 32:2 ** 32 + 96]
    assert not torch.equal(low, high)


# ------------------------------------------------------------------------- streams, graphs

def test_streams_and_graphs(torch, ops):
    """Every call on a side stream and replayed from a graph, against eager calls, with other inputs in between."""
    gen = gen_for(torch, 30)
    n, vocab, cols = 20000, 5000, 200
    tokens = token_ids(torch, gen, n, vocab, torch.int64)
    table = normal(torch, gen, vocab, cols).to(torch.bfloat16)
    w = normal(torch, gen, cols)
    stream_in = normal(torch, gen, n, cols).to(torch.bfloat16)
    p0, small = normal(torch, gen, 5000).to(torch.bfloat16), tokens[:500]

    def run(ws=(None, None, None)):
        x = ops.embed(tokens, table, scale=3.0)
        y, h, rstd = ops.rms_norm(x, w, residual=stream_in)
        q, s, _, _ = ops.rms_norm_mx8(x, w, residual=stream_in)
        dx, dw = ops.rms_norm_backward(y, h, rstd, w, dh=x, workspace=ws[0])
        dt = ops.embed_backward(dx, tokens, vocab, scale=3.0, workspace=ws[1])
        dt1 = ops.embed_backward(dx[:500], small, vocab, workspace=ws[2])
        p, state = p0.clone(), ops.adamw8_state(p0)
        ops.adamw8_step([p], [dt.view(-1)[:5000]], [state], lr=1e-2, step=3, seed=11)
        return [y, h, rstd, q.view(torch.uint8), s.view(torch.uint8), dx, dw, dt, dt1, p] + [t.view(torch.uint8) for t in state]

    want = [t.clone() for t in run()]
    assert all(torch.equal(a, b) for a, b in zip(want, run()))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    ws = [torch.empty(b, dtype=torch.uint8, device="cuda") for b in
          (ops.rms_norm_workspace_bytes(stream_in), ops.embed_workspace_bytes(n, vocab, cols), ops.embed_workspace_bytes(500, vocab, cols))]
    with torch.cuda.stream(side):
        other = run(ws)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, other))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = run(ws)
    t0, s0 = tokens.clone(), stream_in.clone()
    for i in range(4):
        tokens.copy_(t0 if i % 2 == 0 else t0.flip(0))
        stream_in.copy_(s0 if i % 2 == 0 else s0.flip(0))
        graph.replay()
        torch.cuda.synchronize()
        eager = run()
        assert all(torch.equal(a, b) for a, b in zip(held, eager)), i


def test_two_streams_at_once(torch, ops):
    """Calls of one kind on two streams, one of them replayed from a graph, with workspaces of their own: long runs of tokens among them."""
    sets = []
    for seed, n in ((41, 40000), (42, 70000)):
        gen = gen_for(torch, seed)
        tokens = torch.where(torch.rand(n, generator=gen, device="cuda") < 0.7, 11, token_ids(torch, gen, n, 3000, torch.int32))
        dy = normal(torch, gen, n, 136).to(torch.bfloat16)
        ws = [torch.empty(b, dtype=torch.uint8, device="cuda") for b in (ops.embed_workspace_bytes(n, 3000, 136), ops.rms_norm_workspace_bytes(dy))]
        sets.append((tokens.to(torch.int32), dy, normal(torch, gen, 136), ws))

    def run(tokens, dy, w, ws):
        y, h, rstd = ops.rms_norm(dy, w)
        return [y, ops.embed_backward(dy, tokens, 3000, workspace=ws[0]), *ops.rms_norm_backward(y, h, rstd, w, workspace=ws[1])]

    want = [[t.clone() for t in run(*s)] for s in sets]
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = run(*sets[0])
    one, two = torch.cuda.Stream(), torch.cuda.Stream()
    one.wait_stream(torch.cuda.current_stream())
    two.wait_stream(torch.cuda.current_stream())
    for _ in range(6):
        with torch.cuda.stream(one):
            graph.replay()
        with torch.cuda.stream(two):
            other = run(*sets[1])
        one.synchronize()
        two.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(want[0], held))
        assert all(torch.equal(a, b) for a, b in zip(want[1], other))
