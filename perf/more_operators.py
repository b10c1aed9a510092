"""Cases that measure the operators around a mixture-of-experts layer and its optimizer.

Four operators: root-mean-square norm with the residual's addition (``rms_norm``, ``rms_norm_mx8`` with an
output in 8 bits, ``rms_norm_backward``), token embeddings (``embed``, ``embed_backward``), the experts' gated
projections (``expert_gated``, ``expert_gated_backward``) and AdamW with states in 8 bits (``adamw8_step``).
``run`` computes them in plain torch where ``own`` is false and through ``newton_schulz_matrix_muon_amd.ops``
where it is true.

8-bit values are e4m3 with a power of two per block of 32 (e8m0): the smallest that brings the block's
largest finite magnitude to 448 or less.
"""
import math

import torch

own = False

DTYPE = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
BYTES = {"f32": 4, "bf16": 2, "f16": 2}


# ------------------------------------------------------------------------------------ cases

def _rms(pass_, tokens, dim, dtype, wdtype):
    """pass_: "fwd", "mx8" (forward with an 8-bit output), "bwd"; all with a residual stream."""
    return {"op": "rms", "pass": pass_, "tokens": tokens, "dim": dim, "dtype": dtype, "wdtype": wdtype}


def _embed(pass_, tokens, pad, vocab, dim, dtype):
    return {"op": "embed", "pass": pass_, "tokens": tokens, "pad": pad, "vocab": vocab, "dim": dim, "dtype": dtype}


def _gated(pass_, tokens, pad, k, experts, rows, cols, dtype, act):
    """experts = 0: a dense block, every token through the one pair of matrices. pass_: "fwd", "keep" (forward that
    keeps both projections for the backward pass), "bwd"."""
    return {"op": "gated", "pass": pass_, "tokens": tokens, "pad": pad, "k": k, "experts": experts, "rows": rows, "cols": cols,
            "dtype": dtype, "act": act}


def _adamw8(count, size, more, dtype, correct):
    """count tensors of size elements and one of more."""
    return {"op": "adamw8", "count": count, "size": size, "more": more, "dtype": dtype, "correct": correct}


def listed():
    cases = [
        # one token while text is generated: latency alone
        ("rms_fwd_1x7168_bf16", _rms("fwd", 1, 7168, "bf16", "bf16")),
        # a training micro-batch at the 7168-wide model's hidden size, its output in 8 bits
        ("rms_mx8_16384x7168_bf16", _rms("mx8", 16384, 7168, "bf16", "f32")),
        # the backward pass of a ragged batch, rows that no aligned load fits
        ("rms_bwd_16383x2047_f16", _rms("bwd", 16383, 2047, "f16", "f32")),
        # the tokens of a micro-batch in the 163840 x 7168 embedding
        ("embed_fwd_16384_of_163840x7168_bf16", _embed("fwd", 16384, 0, 163840, 7168, "bf16")),
        # its gradient: most of the time goes into the rows of tokens that do not occur
        ("embed_bwd_8192_of_163840x7168_bf16", _embed("bwd", 8192, 0, 163840, 7168, "bf16")),
        # a small model's, padded, with odd sizes: tokens that occur many times
        ("embed_bwd_30011_of_8191x1021_f32", _embed("bwd", 30011, 1000, 8191, 1021, "f32")),
        # one token through its 6 experts of 64: the weights are read once, nothing else counts
        ("gated_fwd_1_k6_e64_1408x2048_bf16", _gated("fwd", 1, 0, 6, 64, 1408, 2048, "bf16", "silu")),
        # one card's 27 experts of 2048 x 7168, a training micro-batch
        ("gated_keep_4096_k8_e27_2048x7168_bf16", _gated("keep", 4096, 0, 8, 27, 2048, 7168, "bf16", "silu")),
        # all gradients of 64 experts of 1408 x 2048 on a padded batch of odd length
        ("gated_bwd_4099_k6_e64_1408x2048_f16", _gated("bwd", 4099, 131, 6, 64, 1408, 2048, "f16", "silu")),
        # a piece of a prompt through the dense block of the 7168-wide model
        ("gated_fwd_509_dense_18432x7168_bf16", _gated("fwd", 509, 0, 1, 0, 18432, 7168, "bf16", "gelu")),
        # 122 norm scales of 7168: one launch, latency
        ("adamw8_122x7168_bf16", _adamw8(122, 7168, 33, "bf16", False)),
        # an eighth of the 163840 x 7168 embedding and eight routers of 384 x 7168
        ("adamw8_20480x7168_bf16", _adamw8(8, 384 * 7168, 20480 * 7168, "bf16", True)),
    ]
    return [dict(c, name=n) for n, c in cases]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _width(rng, lo, hi):
    """Mostly multiples of 8, as models have them; one in four is any number."""
    n = _log(rng, lo, hi)
    return n if rng.random() < 0.25 else max(8, n // 8 * 8)


def draw(rng):
    op = rng.choice(["rms", "embed", "gated", "adamw8"])
    dtype = rng.choice(["bf16", "bf16", "f16", "f32"])
    if op == "rms":
        dim = _width(rng, 64, 16384)
        tokens = _log(rng, 1, min(65536, 16384 * 7168 * 2 // (BYTES[dtype] * dim)))
        return _rms(rng.choice(["fwd", "mx8", "bwd"]), tokens, dim, dtype, rng.choice([dtype, "f32"]))
    if op == "embed":
        dim = _width(rng, 64, 7168)
        vocab = _log(rng, 256, min(163840, 163840 * 7168 * 2 // (BYTES[dtype] * dim)))
        tokens = _log(rng, 1, min(65536, 16384 * 7168 * 2 // (BYTES[dtype] * dim)))
        return _embed(rng.choice(["fwd", "bwd"]), tokens, rng.choice([0, tokens // 16]), vocab, dim, dtype)
    if op == "gated":
        pass_ = rng.choice(["fwd", "keep", "bwd"])
        rows, cols = _width(rng, 64, 7168), _width(rng, 64, 7168)
        experts = rng.choice([0, _log(rng, 4, 384)])
        # no dearer than the largest listed product, whose work is 4 * 32768 * 2048 * 7168 flops
        experts = min(experts, max(1, 27 * 2048 * 7168 * 2 // (rows * cols * BYTES[dtype] * 2)))
        k = rng.randint(1, min(8, experts)) if experts else 1
        most = 32768 * 2048 * 7168 // (rows * cols * k * (2 if pass_ == "bwd" else 1) * (8 if dtype == "f32" else 1))
        tokens = _log(rng, 1, max(1, min(8192, most)))
        return _gated(pass_, tokens, rng.choice([0, tokens // 16]) if experts else 0, k, experts, rows, cols, dtype, rng.choice(["silu", "silu", "gelu", "relu"]))
    count = _log(rng, 1, 100)
    return _adamw8(count, _log(rng, 1, 60000000 // count), _log(rng, 1, 60000000), dtype, rng.choice([False, True]))


# ----------------------------------------------------------------------------------- inputs

def _normal(gen, *shape):
    return torch.randn(*shape, generator=gen, device="cuda")


def _prepare_rms(s, case, gen, dt):
    t, d, wdt = case["tokens"], case["dim"], DTYPE[case["wdtype"]]
    # a residual stream with channels of different scale, and a few that stand out
    scale = 0.5 + torch.rand(d, generator=gen, device="cuda") + 8 * (torch.rand(d, generator=gen, device="cuda") > 0.995)
    s["residual"] = (_normal(gen, t, d) * scale).to(dt)
    s["weight"] = (1 + 0.1 * _normal(gen, d)).to(wdt)
    s["eps"] = 1e-6
    if case["pass"] != "bwd":
        s["x"] = (0.3 * _normal(gen, t, d)).to(dt)
    else:  # the sum and its statistic as the forward pass kept them, the gradients of the norm's output and of the stream
        s["dy"] = (1e-2 * _normal(gen, t, d)).to(dt)
        s["dh"] = (1e-2 * _normal(gen, t, d)).to(dt)
        s["rstd"] = torch.rsqrt(s["residual"].float().square().mean(dim=1) + s["eps"])


def _prepare_embed(s, case, gen, dt):
    t, v, d = case["tokens"], case["vocab"], case["dim"]
    # word frequencies fall with the word's rank, whose place in the vocabulary is arbitrary
    rank = torch.exp(torch.rand(t, generator=gen, device="cuda", dtype=torch.float64) * math.log(v)).long().clamp(1, v) - 1
    s["tokens"] = torch.randperm(v, generator=gen, device="cuda")[rank]
    if case["pad"]:
        s["tokens"][t - case["pad"]:] = -1
    s["scale"] = math.sqrt(d)
    if case["pass"] == "fwd":
        s["table"] = _normal(gen, v, d).mul_(0.02).to(dt)
    else:
        s["dy"] = (1e-2 * _normal(gen, t, d)).to(dt)


def _prepare_gated(s, case, gen, dt):
    t, e, k, n, c = case["tokens"], max(1, case["experts"]), case["k"], case["rows"], case["cols"]
    slots, kept = t * k, (t - case["pad"]) * k
    if case["experts"]:  # rows per expert as routers spread them: some experts are liked more than others
        score = _normal(gen, t - case["pad"], e) + 0.5 * _normal(gen, e)
        count = torch.bincount(torch.topk(score, k, dim=1).indices.reshape(-1), minlength=e)
    else:
        count = torch.full((1,), slots, device="cuda")
    offsets = torch.cat([count.new_zeros(1), count.cumsum(0)])
    s["offsets"] = offsets.to(torch.int32) if case["experts"] else None
    here = (torch.arange(slots, device="cuda") < kept)[:, None]
    shape = (e, n, c) if case["experts"] else (n, c)
    s["w_gate"], s["w_up"] = ((_normal(gen, *shape) * (1.5 * c ** -0.5)).to(dt) for _ in range(2))
    s["x"] = _normal(gen, slots, c).to(dt)
    if case["pass"] == "bwd":  # what the forward pass kept, and the gradient that arrives
        s["gate"], s["up"] = ((_normal(gen, slots, n) * 1.5 * here).to(dt) for _ in range(2))
        s["dh"] = (1e-2 * _normal(gen, slots, n)).to(dt)
    # the plain form's own plan: experts with rows, their rows padded to the longest, and back
    s["active"] = torch.nonzero(count)[:, 0]
    longest = max(1, int(count.max()))
    at = offsets[s["active"]][:, None] + torch.arange(longest, device="cuda")
    s["grid"] = torch.where(at < offsets[s["active"] + 1][:, None], at, torch.full_like(at, slots))
    back = torch.full((slots + 1,), s["grid"].numel(), device="cuda", dtype=torch.long)
    back[s["grid"].reshape(-1)] = torch.arange(s["grid"].numel(), device="cuda")
    s["back"] = back[:slots].clone()
    s["back"][kept:] = s["grid"].numel()


def _prepare_adamw8(s, case, gen, dt):
    sizes = [case["size"]] * case["count"] + [case["more"]]
    starts = [0]
    for n in sizes:  # tensors of one buffer, each at a multiple of 32 elements; zeros between them
        starts.append(starts[-1] + (n + 31) // 32 * 32)
    total = starts[-1]
    s["starts"], s["sizes"] = starts, sizes
    here = torch.ones(total, device="cuda")
    if case["size"] % 32:
        here[:starts[-2]].view(case["count"], -1)[:, case["size"]:] = 0
    here[starts[-2] + case["more"]:] = 0
    # gradients whose scale differs from block to block, and moments of the same scale
    scale = 1e-3 * torch.exp(_normal(gen, total // 32))
    exps = (torch.log2(scale) + 127 - 8).round().to(torch.uint8)
    s["grad"] = (_normal(gen, total // 32, 32) * scale[:, None]).view(-1).mul_(here).to(dt)
    codes = (_normal(gen, total) * 128).clamp(-448, 448).mul_(here).to(torch.float8_e4m3fn)
    roots = (_normal(gen, total).abs() * 128).clamp(2.0 ** -9, 448).mul_(here).to(torch.float8_e4m3fn)
    param = (0.02 * _normal(gen, total)).mul_(here).to(dt)
    s["flat"] = (param, codes, exps.view(torch.float8_e8m0fnu), roots, (exps + 1).view(torch.float8_e8m0fnu))
    part = lambda t, i: t[starts[i]:starts[i] + sizes[i]]  # noqa: E731
    blocks = lambda t, i: t[starts[i] // 32:starts[i + 1] // 32]  # noqa: E731
    s["params"], s["grads"] = ([part(t, i) for i in range(len(sizes))] for t in (param, s["grad"]))
    s["states"] = [(part(codes, i), blocks(s["flat"][2], i), part(roots, i), blocks(s["flat"][4], i)) for i in range(len(sizes))]
    s["hyper"] = {"lr": 1e-3, "beta1": 0.9, "beta2": 0.95, "eps": 1e-8, "weight_decay": 0.1, "step": 7, "bias_correction": case["correct"]}
    s["seed"] = int(torch.randint(0, 2 ** 62, (1,), generator=gen, device="cuda"))


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(int(seed))
    s = {"case": case}
    make = {"rms": _prepare_rms, "embed": _prepare_embed, "gated": _prepare_gated, "adamw8": _prepare_adamw8}
    make[case["op"]](s, case, gen, DTYPE[case["dtype"]])
    return s


# ------------------------------------------------------------------------------ plain forms

def _scale_byte(top):
    """The exponent byte of the smallest power of two that brings top (fp32, finite) to 448 = 1.75 * 2^8 or less."""
    bits = top.view(torch.int32)
    return ((bits >> 23) - 8 + ((bits & 0x7fffff) > 0x600000).int()).clamp(min=0)


def _times(x, power):
    """x * 2^power, exactly, for blocks of 32 (power int32 per block)."""
    return x * ((power + 127) << 23).view(torch.float32)[..., None]


def _blocks(x):
    """fp32 [rows, n] in blocks of 32, zeros behind the end: (values [rows, blocks, 32], exponent bytes)."""
    rows, n = x.shape
    full = torch.zeros(rows, (n + 31) // 32 * 32, device=x.device)
    full[:, :n] = x
    full = full.view(rows, -1, 32)
    size = full.abs()
    byte = _scale_byte(torch.where(torch.isfinite(size), size, torch.zeros_like(size)).amax(dim=2))
    return full, byte


def _plain_rms(s):
    case, w = s["case"], s["weight"].float()
    if case["pass"] == "bwd":
        h, dy, rstd = s["residual"].float(), s["dy"].float(), s["rstd"][:, None]
        xh = h * rstd
        g = dy * w
        dx = (g - xh * ((g * xh).sum(dim=1, keepdim=True) / h.shape[1])) * rstd + s["dh"].float()
        return dx.to(s["residual"].dtype), (dy * xh).sum(dim=0).to(s["weight"].dtype)
    h = (s["x"].float() + s["residual"].float()).to(s["x"].dtype)
    f = h.float()
    rstd = 1 / torch.sqrt((f * f).sum(dim=1) / f.shape[1] + s["eps"])
    y = f * rstd[:, None] * w
    if case["pass"] == "fwd":
        return y.to(h.dtype), h, rstd
    full, byte = _blocks(y)
    q = _times(full, 127 - byte).to(torch.float8_e4m3fn).view(y.shape[0], -1)[:, :y.shape[1]]
    return q, byte.to(torch.uint8).view(torch.float8_e8m0fnu), h, rstd


def _plain_embed(s):
    case, tokens = s["case"], s["tokens"]
    have = (tokens >= 0) & (tokens < case["vocab"])
    if case["pass"] == "fwd":
        rows = s["table"][tokens.clamp(0, case["vocab"] - 1)].float() * s["scale"]
        return torch.where(have[:, None], rows, torch.zeros((), device="cuda")).to(s["table"].dtype)
    out = torch.zeros(case["vocab"] + 1, case["dim"], device="cuda")
    out.index_add_(0, torch.where(have, tokens, torch.full_like(tokens, case["vocab"])), s["dy"].float())
    return (out[:-1] * s["scale"]).to(s["dy"].dtype)


def _padded(rows, grid):
    """The experts' rows in 32 bits, each expert's padded with zeros to the longest: [A, L, D]."""
    return torch.cat([rows.float(), torch.zeros(1, rows.shape[1], device=rows.device)])[grid]


def _unpadded(values, s):
    flat = torch.cat([values.reshape(-1, values.shape[-1]), torch.zeros(1, values.shape[-1], device=values.device)])
    return flat[s["back"]].to(s["x"].dtype)


def _plain_act(g, act):
    """The activation and its slope."""
    if act == "relu":
        return g.clamp(min=0), (g > 0).to(g.dtype)
    if act == "silu":
        p = 1 / (1 + torch.exp(-g))
        return g * p, p * (1 + g * (1 - p))
    p = 0.5 * (1 + torch.erf(g * math.sqrt(0.5)))
    return g * p, p + g * torch.exp(-0.5 * g * g) * (1 / math.sqrt(2 * math.pi))


def _plain_gated(s):
    case, pick = s["case"], s["active"]
    wg, wu = (w.view(-1, case["rows"], case["cols"])[pick].float() for w in (s["w_gate"], s["w_up"]))
    x = _padded(s["x"], s["grid"])
    if case["pass"] != "bwd":
        gate = torch.matmul(x, wg.transpose(1, 2).contiguous())
        up = torch.matmul(x, wu.transpose(1, 2).contiguous())
        h = _unpadded(_plain_act(gate, case["act"])[0] * up, s)
        return (h, _unpadded(gate, s), _unpadded(up, s)) if case["pass"] == "keep" else h
    dh, gate, up = (_padded(s[n], s["grid"]) for n in ("dh", "gate", "up"))
    a, slope = _plain_act(gate, case["act"])
    dgate, dup = dh * up * slope, dh * a
    dx = _unpadded(torch.matmul(dgate, wg) + torch.matmul(dup, wu), s)
    dwg, dwu = torch.zeros_like(s["w_gate"]), torch.zeros_like(s["w_up"])
    dwg.view(-1, case["rows"], case["cols"])[pick] = torch.matmul(dgate.transpose(1, 2).contiguous(), x).to(dwg.dtype)
    dwu.view(-1, case["rows"], case["cols"])[pick] = torch.matmul(dup.transpose(1, 2).contiguous(), x).to(dwu.dtype)
    return dx, dwg, dwu


# Rounding up or down at random, in proportion, by 16 bits for each state of an element: the number is
# mixed from the call's seed, its step, the tensor's place in the list and the element's in the tensor.
_MIX = (0xdf50e7c3, 0x3dd219bf, 0xafd7c8e5)


def _mixed(x):
    """32 bits (held in 64) mixed; python numbers and int64 tensors."""
    x = x ^ (x >> 16)
    x = (x * _MIX[1]) & 0xffffffff
    x = x ^ (x >> 15)
    x = (x * _MIX[2]) & 0xffffffff
    return x ^ (x >> 16)


def _random16(s):
    """The two numbers of every element of the buffer that holds the tensors."""
    seed = s["seed"]
    key = _mixed(_mixed(_mixed(seed & 0xffffffff) ^ (seed >> 32 & 0xffffffff)) ^ s["hyper"]["step"])
    starts = torch.tensor(s["starts"], device="cuda")
    keys = _mixed(torch.arange(len(s["sizes"]), device="cuda") ^ key) - starts[:-1] * _MIX[0]
    x = torch.arange(s["starts"][-1], device="cuda").view(-1, 32) * _MIX[0] + keys.repeat_interleave(starts.diff() // 32)[:, None]
    x = _mixed(x.view(-1) & 0xffffffff)
    return (x & 0xffff).int(), (x >> 16).int()


def _to_e4m3(x, rnd):
    """Magnitudes x (at most 448): a multiple of the step of e4m3 below or above, above by the chance rnd / 2^16 gives."""
    high = ((x.view(torch.int32) + (rnd << 4)) & ~0xfffff).view(torch.float32)
    low = torch.floor(x * 512 + rnd * 2.0 ** -16) * 2.0 ** -9
    return torch.where(x < 2.0 ** -6, low, high)


def _plain_adamw8(s):
    h, (p, codes, exps, roots, root_exps) = s["hyper"], s["flat"]
    c1 = 1 / (1 - h["beta1"] ** h["step"]) if h["bias_correction"] else 1.0
    c2 = math.sqrt(1 / (1 - h["beta2"] ** h["step"])) if h["bias_correction"] else 1.0
    f, (r_m, r_r) = s["grad"].float(), _random16(s)
    wide = lambda q, e: (q.float().view(-1, 32) * e.float()[:, None]).view(-1)  # noqa: E731
    m = h["beta1"] * wide(codes, exps) + (1 - h["beta1"]) * f
    r = torch.sqrt(h["beta2"] * wide(roots, root_exps).square() + (1 - h["beta2"]) * (f * f))
    p.copy_(((1 - h["lr"] * h["weight_decay"]) * p.float() - h["lr"] * ((m * c1) / (r * c2 + h["eps"]))).to(p.dtype))
    full, byte = _blocks(m[None])
    size = _to_e4m3(_times(full, 127 - byte).abs().view(-1), r_m)
    codes.copy_(torch.where(m < 0, -size, size).to(codes.dtype))
    exps.copy_(byte[0].to(torch.uint8).view(exps.dtype))
    full, byte = _blocks(r[None])
    size = _to_e4m3(_times(full, 127 - byte).view(-1), r_r)
    # a root that is not zero keeps the smallest value at least: a step never divides by eps alone where it did not before
    roots.copy_(torch.where(r > 0, size.clamp(min=2.0 ** -9), size).to(roots.dtype))
    root_exps.copy_(byte[0].to(torch.uint8).view(root_exps.dtype))
    return s["flat"]


# --------------------------------------------------------------------------------------- run

def run(state):
    s, case = state, state["case"]
    if not own:
        return {"rms": _plain_rms, "embed": _plain_embed, "gated": _plain_gated, "adamw8": _plain_adamw8}[case["op"]](s)
    from newton_schulz_matrix_muon_amd import ops
    if case["op"] == "rms":
        if case["pass"] == "bwd":
            return ops.rms_norm_backward(s["dy"], s["residual"], s["rstd"], s["weight"], dh=s["dh"])
        call = ops.rms_norm if case["pass"] == "fwd" else ops.rms_norm_mx8
        return call(s["x"], s["weight"], residual=s["residual"], eps=s["eps"])
    if case["op"] == "embed":
        if case["pass"] == "fwd":
            return ops.embed(s["tokens"], s["table"], scale=s["scale"])
        return ops.embed_backward(s["dy"], s["tokens"], case["vocab"], scale=s["scale"])
    if case["op"] == "gated":
        if case["pass"] != "bwd":
            return ops.expert_gated(s["x"], s["w_gate"], s["w_up"], s["offsets"], act=case["act"], keep=case["pass"] == "keep")
        return ops.expert_gated_backward(s["dh"], s["x"], s["w_gate"], s["w_up"], s["gate"], s["up"], s["offsets"], act=case["act"])
    ops.adamw8_step(s["params"], s["grads"], s["states"], seed=s["seed"], **s["hyper"])
    return s["flat"]


# -------------------------------------------------------------------------------------- work

def work(case):
    es = BYTES[case["dtype"]]
    if case["op"] == "adamw8":  # parameter, gradient and both codes with their blocks' exponents
        n = case["count"] * case["size"] + case["more"]
        return {"bytes": n * (3 * es + 4) + n // 8, "flops": 16 * n}
    t, pad = case["tokens"], case.get("pad", 0)
    if case["op"] == "rms":
        d, w = case["dim"], case["dim"] * BYTES[case["wdtype"]]
        if case["pass"] == "bwd":  # dy, h, dh, weight, rstd -> dx, dweight
            return {"bytes": 4 * t * d * es + 2 * w + 4 * t, "flops": 9 * t * d}
        out = t * d * es if case["pass"] == "fwd" else t * d + t * ((d + 31) // 32)
        return {"bytes": 3 * t * d * es + out + w + 4 * t, "flops": 5 * t * d}  # x, residual, weight -> y, h, rstd
    if case["op"] == "embed":
        d = case["dim"]
        if case["pass"] == "fwd":
            return {"bytes": (2 * t - pad) * d * es + 8 * t, "flops": t * d}
        return {"bytes": (t - pad + case["vocab"]) * d * es + 8 * t, "flops": t * d}
    n, c, e = case["rows"], case["cols"], max(1, case["experts"])
    slots, kept = t * case["k"], (t - pad) * case["k"]
    active = min(e, kept)
    if case["pass"] != "bwd":
        return {"bytes": (kept * c + 2 * active * n * c + slots * n * (3 if case["pass"] == "keep" else 1)) * es, "flops": 4 * kept * n * c}
    return {"bytes": (kept * (3 * n + c) + 2 * active * n * c + slots * c + 2 * e * n * c) * es, "flops": 8 * kept * n * c}


# ------------------------------------------------------------------------------------- exact

def _nearest(x, pick):
    """64-bit values as e4m3 stands for them, |x| <= 448; pick(steps) chooses whole steps."""
    _, e = torch.frexp(x.abs())
    step = torch.exp2((e - 1).clamp(min=-6).double() - 3)
    return pick(x / step) * step


def _exponents(x):
    """(64-bit values [rows, n] in blocks of 32, the blocks' powers of two)."""
    rows, n = x.shape
    x = torch.nn.functional.pad(x, (0, -n % 32)).view(rows, -1, 32)
    part, e = torch.frexp(x.abs().amax(dim=2))  # part in [1/2, 1): 448 is 0.875 * 2^9
    power = torch.where(part == 0, -127, (e - 9 + (part > 0.875).int()).clamp(min=-127))
    return x, torch.exp2(power.double())


def exact(case, seed):
    """The definitions in 64 bits: one expert after the other, gradients summed through an incidence of sorted tokens."""
    s = prepare(case, seed)
    if case["op"] == "rms":
        w = s["weight"].double()
        if case["pass"] == "bwd":
            h, dy, r = s["residual"].double(), s["dy"].double(), s["rstd"].double()[:, None]
            dot = torch.linalg.vecdot(dy * w, h)[:, None]
            return torch.addcmul(s["dh"].double(), r, dy * w) - h * dot * (r ** 3 / h.shape[1]), torch.linalg.vecdot(dy, h * r, dim=0)
        total = s["x"].double() + s["residual"].double()
        h = total.to(s["x"].dtype).double()
        rstd = (h.pow(2).mean(dim=1) + s["eps"]).pow(-0.5)
        y = h * rstd[:, None] * w
        if case["pass"] == "fwd":
            return y, total, rstd
        x, scale = _exponents(y)
        return _nearest(x / scale[..., None], torch.round).flatten(1)[:, :y.shape[1]], scale, total, rstd
    if case["op"] == "embed":
        tokens = s["tokens"]
        if case["pass"] == "fwd":
            out = torch.zeros(case["tokens"], case["dim"], dtype=torch.float64, device="cuda")
            have = torch.nonzero(tokens >= 0)[:, 0]
            out[have] = s["table"][tokens[have]].double() * s["scale"]
            return out
        order = torch.argsort(tokens)
        order = order[tokens[order] >= 0]
        words, counts = torch.unique_consecutive(tokens[order], return_counts=True)
        ends = counts.cumsum(0)
        out = torch.zeros(case["vocab"], case["dim"], dtype=torch.float64, device="cuda")
        sums = torch.segment_reduce(s["dy"][order].double(), "sum", offsets=torch.cat([ends.new_zeros(1), ends]), axis=0)
        out[words] = sums * s["scale"]
        return out
    if case["op"] == "gated":
        x, n, c = s["x"], case["rows"], case["cols"]
        wg, wu = s["w_gate"].view(-1, n, c), s["w_up"].view(-1, n, c)
        off = s["offsets"].tolist() if s["offsets"] is not None else [0, x.shape[0]]
        spans = [(e, slice(lo, hi)) for e, (lo, hi) in enumerate(zip(off, off[1:])) if hi > lo]
        zeros = lambda *shape: torch.zeros(*shape, dtype=torch.float64, device="cuda")  # noqa: E731

        def act(g):  # the activation and its slope
            if case["act"] == "relu":
                return torch.where(g > 0, g, 0), torch.heaviside(g, zeros(1))
            if case["act"] == "silu":
                p = torch.sigmoid(g)
                return g * p, p + g * p * torch.sigmoid(-g)
            p = 0.5 * torch.erfc(-g / math.sqrt(2))
            return g * p, p + g * torch.exp(-g * g / 2) / math.sqrt(2 * math.pi)
        if case["pass"] != "bwd":
            h, gate, up = (zeros(x.shape[0], n) for _ in range(3))
            for e, r in spans:
                gate[r], up[r] = x[r].double() @ wg[e].double().T, x[r].double() @ wu[e].double().T
                h[r] = act(gate[r])[0] * up[r]
            return (h, gate, up) if case["pass"] == "keep" else h
        dx, dwg, dwu = zeros(x.shape), zeros(wg.shape), zeros(wu.shape)
        for e, r in spans:
            a, slope = act(s["gate"][r].double())
            dg, du = s["dh"][r].double() * s["up"][r].double() * slope, s["dh"][r].double() * a
            dx[r] = dg @ wg[e].double() + du @ wu[e].double()
            dwg[e], dwu[e] = dg.T @ x[r].double(), du.T @ x[r].double()
        return dx, dwg.view(s["w_gate"].shape), dwu.view(s["w_up"].shape)
    h, (p, codes, exps, roots, root_exps) = s["hyper"], (t.double() for t in s["flat"])
    g, held = s["grad"].double(), []
    m = torch.lerp(g, codes * exps.repeat_interleave(32), h["beta1"])
    r = torch.lerp(g ** 2, (roots * root_exps.repeat_interleave(32)) ** 2, h["beta2"]).sqrt()
    fix = (1 - h["beta1"] ** h["step"], (1 - h["beta2"] ** h["step"]) ** 0.5) if h["bias_correction"] else (1, 1)
    p = p * (1 - h["lr"] * h["weight_decay"]) - h["lr"] * (m / fix[0]) / (r / fix[1] + h["eps"])
    for v, least, rnd in zip((m, r), (0.0, 2.0 ** -9), _random16(s)):
        x, scale = _exponents(v[None])
        x = (x / scale[..., None]).view(-1)
        q = _nearest(x.abs(), lambda steps: torch.floor(steps + rnd.double() / 65536))
        held += [torch.copysign(torch.where(v != 0, q.clamp(min=least), q), x), scale[0]]
    return (p, *held)
