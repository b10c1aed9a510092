"""Cases that measure the operators of a mixture-of-experts layer's training and serving path.

Four operators, each with its gradient: layer norm, rows sorted by expert (``expert_dispatch``),
rows summed back with their weights (``expert_combine``) and the experts' matrix products
(``expert_matmul``). ``run`` computes them in plain torch where ``own`` is false and through
``newton_schulz_matrix_muon_amd.ops`` where it is true.

T tokens choose k of E experts each; a padded token chooses none (id -1). The S = T k slots are
sorted by expert, ties by slot; rows behind the last expert's are zero.
"""
import math

import torch

own = False

DTYPE = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
BYTES = {"f32": 4, "bf16": 2, "f16": 2}


# ------------------------------------------------------------------------------------ cases

def _norm(pass_, tokens, dim, dtype, wdtype):
    return {"op": "norm", "pass": pass_, "tokens": tokens, "dim": dim, "dtype": dtype, "wdtype": wdtype}


def _rows(op, pass_, tokens, pad, k, experts, dim, dtype):
    return {"op": op, "pass": pass_, "tokens": tokens, "pad": pad, "k": k, "experts": experts, "dim": dim, "dtype": dtype}


def _matmul(pass_, tokens, pad, k, experts, rows, cols, dtype):
    return {"op": "matmul", "pass": pass_, "tokens": tokens, "pad": pad, "k": k, "experts": experts, "rows": rows,
            "cols": cols, "dtype": dtype}


def listed():
    cases = [
        # one token while text is generated: latency alone
        ("norm_fwd_1x7168_bf16", _norm("fwd", 1, 7168, "bf16", "bf16")),
        # a training micro-batch of 16384 tokens at the 7168-wide model's hidden size
        ("norm_fwd_16384x7168_bf16", _norm("fwd", 16384, 7168, "bf16", "bf16")),
        # its backward pass, with fp32 master weights for the norm
        ("norm_bwd_16384x7168_bf16", _norm("bwd", 16384, 7168, "bf16", "f32")),
        # odd sizes in fp32: rows that no vector load fits
        ("norm_bwd_1021x2047_f32", _norm("bwd", 1021, 2047, "f32", "f32")),
        # a decoding batch of 16 sequences over 384 experts
        ("dispatch_fwd_16_k8_e384_7168_bf16", _rows("dispatch", "fwd", 16, 0, 8, 384, 7168, "bf16")),
        # a training micro-batch over 384 experts
        ("dispatch_fwd_8192_k8_e384_7168_bf16", _rows("dispatch", "fwd", 8192, 0, 8, 384, 7168, "bf16")),
        # the gradient of a padded batch of odd length, 64 experts of the 2048-wide model, top 6
        ("dispatch_bwd_4099_k6_e64_2048_f16", _rows("dispatch", "bwd", 4099, 131, 6, 64, 2048, "f16")),
        ("combine_fwd_8192_k8_e384_7168_bf16", _rows("combine", "fwd", 8192, 0, 8, 384, 7168, "bf16")),
        ("combine_bwd_4099_k6_e64_2048_f16", _rows("combine", "bwd", 4099, 131, 6, 64, 2048, "f16")),
        # one token through its 6 experts of 64: the weights are read once, nothing else counts
        ("matmul_fwd_1_k6_e64_1408x2048_bf16", _matmul("fwd", 1, 0, 6, 64, 1408, 2048, "bf16")),
        # one card's 27 experts of 2048 x 7168 (a 216-expert layer over 8 cards)
        ("matmul_fwd_4096_k8_e27_2048x7168_bf16", _matmul("fwd", 4096, 0, 8, 27, 2048, 7168, "bf16")),
        # both gradients of 64 experts of 1408 x 2048 on a padded batch of odd length
        ("matmul_bwd_4099_k6_e64_1408x2048_f16", _matmul("bwd", 4099, 131, 6, 64, 1408, 2048, "f16")),
    ]
    return [dict(c, name=n) for n, c in cases]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _width(rng, lo, hi):
    """Mostly multiples of 8, as models have them; one in four is any number."""
    n = _log(rng, lo, hi)
    return n if rng.random() < 0.25 else max(8, n // 8 * 8)


def draw(rng):
    op = rng.choice(["norm", "dispatch", "combine", "matmul"])
    pass_ = rng.choice(["fwd", "bwd"])
    dtype = rng.choice(["bf16", "bf16", "f16", "f32"])
    if op == "norm":
        dim = _width(rng, 64, 16384)
        tokens = _log(rng, 1, min(65536, 16384 * 7168 * 2 // (BYTES[dtype] * dim)))
        return _norm(pass_, tokens, dim, dtype, rng.choice([dtype, "f32"]))
    experts = _log(rng, 4, 384)
    k = rng.randint(1, min(8, experts))
    if op != "matmul":
        dim = _width(rng, 64, 7168)
        tokens = _log(rng, 1, min(32768, 8192 * 8 * 7168 * 2 // (2 * BYTES[dtype] * dim * k)))
        return _rows(op, pass_, tokens, rng.choice([0, tokens // 16]), k, experts, dim, dtype)
    rows, cols = _width(rng, 64, 7168), _width(rng, 64, 7168)
    # no dearer than the largest listed product, whose work is 2 * 32768 * 2048 * 7168 * 2 bytes or flops
    experts = max(1, min(experts, 27 * 2048 * 7168 * 2 // (rows * cols * BYTES[dtype] * 2)))
    k = min(k, experts)
    most = 32768 * 2048 * 7168 // (rows * cols * k * (2 if pass_ == "bwd" else 1) * (8 if dtype == "f32" else 1))
    tokens = _log(rng, 1, max(1, min(8192, most)))
    return _matmul(pass_, tokens, rng.choice([0, tokens // 16]), k, experts, rows, cols, dtype)


# ----------------------------------------------------------------------------------- inputs

def _normal(gen, *shape):
    return torch.randn(*shape, generator=gen, device="cuda")


def _choices(gen, case):
    """The experts that each token's router picks, int32 [T, k]: some experts are liked more than others."""
    t, e = case["tokens"], case["experts"]
    score = _normal(gen, t, e) + 0.5 * _normal(gen, e)
    top = torch.topk(score, case["k"], dim=1)
    ids = top.indices.to(torch.int32)
    if case["pad"]:
        ids[t - case["pad"]:] = -1
    return ids, torch.softmax(top.values, dim=1)


def _sorted(ids, experts):
    """(offsets int32 [E + 1], rank int32 [T, k]): where each expert's rows begin, and each slot's row (-1: none)."""
    flat = ids.reshape(-1).long()
    key = torch.where((flat >= 0) & (flat < experts), flat, torch.full_like(flat, experts))
    order = torch.argsort(key, stable=True)
    rank = torch.empty_like(order)
    rank[order] = torch.arange(order.numel(), device=order.device)
    rank = torch.where(key < experts, rank, torch.full_like(rank, -1))
    offsets = torch.searchsorted(key[order], torch.arange(experts + 1, device=key.device), right=False)
    return offsets.to(torch.int32), rank.to(torch.int32).view(ids.shape)


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(int(seed))
    dt = DTYPE[case["dtype"]]
    s = {"case": case}
    if case["op"] == "norm":
        t, d, wdt = case["tokens"], case["dim"], DTYPE[case["wdtype"]]
        # activations: channels of different scale around an offset
        s["x"] = (_normal(gen, t, d) * (0.5 + torch.rand(d, generator=gen, device="cuda")) + 0.3 * _normal(gen, d)).to(dt)
        s["weight"] = (1 + 0.1 * _normal(gen, d)).to(wdt)
        s["bias"] = (0.1 * _normal(gen, d)).to(wdt)
        s["eps"] = 1e-5
        if case["pass"] == "bwd":  # the gradient that arrives and what the forward pass kept
            s["dy"] = (1e-2 * _normal(gen, t, d)).to(dt)
            x = s["x"].float()
            s["mean"] = x.mean(dim=1)
            s["rstd"] = torch.rsqrt((x - s["mean"][:, None]).square().mean(dim=1) + s["eps"])
        return s
    ids, weights = _choices(gen, case)
    offsets, rank = _sorted(ids, case["experts"])
    slots = ids.numel()
    if case["op"] == "matmul":
        n, k, e = case["rows"], case["cols"], case["experts"]
        s["offsets"] = offsets
        s["w"] = (_normal(gen, e, n, k) * 0.02).to(dt)
        s["x"] = _normal(gen, slots, k).to(dt)
        if case["pass"] == "bwd":
            s["dy"] = (1e-2 * _normal(gen, slots, n)).to(dt)
        # the plain form's own plan: experts with rows, their rows padded to the longest, and back
        count = (offsets[1:] - offsets[:-1]).long()
        s["active"] = torch.nonzero(count)[:, 0]
        longest = max(1, int(count.max()))
        at = offsets[s["active"]].long()[:, None] + torch.arange(longest, device="cuda")
        s["grid"] = torch.where(at < offsets[s["active"] + 1][:, None], at, torch.full_like(at, slots))
        back = torch.full((slots + 1,), s["grid"].numel(), device="cuda", dtype=torch.long)
        back[s["grid"].reshape(-1)] = torch.arange(s["grid"].numel(), device="cuda")
        back[slots] = s["grid"].numel()
        s["back"] = back[:slots]
        return s
    d = case["dim"]
    s["experts"] = case["experts"]
    if case["op"] == "dispatch" and case["pass"] == "fwd":
        s["x"], s["ids"] = _normal(gen, case["tokens"], d).to(dt), ids
        return s
    s["offsets"], s["rank"], s["weights"] = offsets, rank, weights
    kept = torch.arange(slots, device="cuda") < offsets[-1]
    if case["op"] == "dispatch":
        s["dxs"] = (1e-2 * _normal(gen, slots, d) * kept[:, None]).to(dt)
    else:
        s["ys"] = (_normal(gen, slots, d) * kept[:, None]).to(dt)
        if case["pass"] == "bwd":
            s["dy"] = (1e-2 * _normal(gen, case["tokens"], d)).to(dt)
    return s


# ------------------------------------------------------------------------------ plain forms

def _plain_norm(s):
    x, w, b = s["x"].float(), s["weight"].float(), s["bias"].float()
    if s["case"]["pass"] == "fwd":
        mean = x.sum(dim=1) / x.shape[1]
        c = x - mean[:, None]
        rstd = 1 / torch.sqrt((c * c).sum(dim=1) / x.shape[1] + s["eps"])
        return (c * rstd[:, None] * w + b).to(s["x"].dtype), mean, rstd
    dy = s["dy"].float()
    xh = (x - s["mean"][:, None]) * s["rstd"][:, None]
    g = dy * w
    m1 = g.sum(dim=1, keepdim=True) / x.shape[1]
    m2 = (g * xh).sum(dim=1, keepdim=True) / x.shape[1]
    dx = (g - m1 - xh * m2) * s["rstd"][:, None]
    return dx.to(s["x"].dtype), (dy * xh).sum(dim=0).to(s["weight"].dtype), dy.sum(dim=0).to(s["weight"].dtype)


def _gathered(rows, rank):
    """rows[rank] in 32 bits, zero where a slot has no row: [T, k, D]."""
    got = rows[rank.clamp(min=0).long().reshape(-1)].view(*rank.shape, -1).float()
    return torch.where((rank >= 0)[..., None], got, torch.zeros((), device=got.device))


def _scattered(values, rank, dtype):
    """values [T, k, D] at their rows, the others zero: [S, D]."""
    out = torch.zeros(rank.numel() + 1, values.shape[-1], dtype=dtype, device=values.device)
    flat = rank.reshape(-1).long()
    out[torch.where(flat >= 0, flat, torch.full_like(flat, rank.numel()))] = values.reshape(flat.numel(), -1).to(dtype)
    return out[:-1]


def _plain_dispatch(s):
    if s["case"]["pass"] == "bwd":
        return _gathered(s["dxs"], s["rank"]).sum(dim=1).to(s["dxs"].dtype)
    offsets, rank = _sorted(s["ids"], s["experts"])
    x = s["x"]
    return _scattered(x[:, None].expand(-1, rank.shape[1], -1), rank, x.dtype), offsets, rank


def _plain_combine(s):
    ys = _gathered(s["ys"], s["rank"])
    if s["case"]["pass"] == "fwd":
        return (ys * s["weights"][..., None]).sum(dim=1).to(s["ys"].dtype)
    dy = s["dy"].float()[:, None]
    return _scattered(dy * s["weights"][..., None], s["rank"], s["ys"].dtype), (ys * dy).sum(dim=2)


def _padded(rows, grid):
    """The experts' rows in 32 bits, each expert's padded with zeros to the longest: [A, L, D]."""
    return torch.cat([rows.float(), torch.zeros(1, rows.shape[1], device=rows.device)])[grid]


def _unpadded(values, s):
    flat = torch.cat([values.reshape(-1, values.shape[-1]), torch.zeros(1, values.shape[-1], device=values.device)])
    return flat[s["back"]].to(s["w"].dtype)


def _plain_matmul(s):
    w = s["w"][s["active"]].float()
    x = _padded(s["x"], s["grid"])
    if s["case"]["pass"] == "fwd":
        return _unpadded(torch.matmul(x, w.transpose(1, 2).contiguous()), s)
    dy = _padded(s["dy"], s["grid"])
    dw = torch.zeros_like(s["w"])
    dw[s["active"]] = torch.matmul(dy.transpose(1, 2).contiguous(), x).to(dw.dtype)
    return _unpadded(torch.matmul(dy, w), s), dw


# --------------------------------------------------------------------------------------- run

def run(state):
    s, case = state, state["case"]
    if not own:
        return {"norm": _plain_norm, "dispatch": _plain_dispatch, "combine": _plain_combine, "matmul": _plain_matmul}[case["op"]](s)
    from newton_schulz_matrix_muon_amd import ops
    forward = case["pass"] == "fwd"
    if case["op"] == "norm":
        if forward:
            return ops.layer_norm(s["x"], s["weight"], s["bias"], eps=s["eps"])
        return ops.layer_norm_backward(s["dy"], s["x"], s["mean"], s["rstd"], s["weight"])
    if case["op"] == "dispatch":
        if not forward:
            return ops.expert_dispatch_backward(s["dxs"], s["rank"])
        offsets, rank = ops.expert_sort(s["ids"], s["experts"])
        return ops.expert_dispatch(s["x"], rank, offsets), offsets, rank
    if case["op"] == "combine":
        if forward:
            return ops.expert_combine(s["ys"], s["weights"], s["rank"])
        return ops.expert_combine_backward(s["dy"], s["ys"], s["weights"], s["rank"], s["offsets"])
    if forward:
        return ops.expert_matmul(s["x"], s["w"], s["offsets"])
    return ops.expert_matmul_backward(s["dy"], s["x"], s["w"], s["offsets"])


# -------------------------------------------------------------------------------------- work

def work(case):
    es, t = BYTES[case["dtype"]], case["tokens"]
    if case["op"] == "norm":
        d, wes = case["dim"], BYTES[case["wdtype"]]
        if case["pass"] == "fwd":  # x, weight, bias -> y, mean, rstd
            return {"bytes": 2 * t * d * es + 2 * d * wes + 8 * t, "flops": 8 * t * d}
        return {"bytes": 3 * t * d * es + 3 * d * wes + 8 * t, "flops": 14 * t * d}  # dy, x, weight, mean, rstd -> dx, dweight, dbias
    slots, kept, e = t * case["k"], (t - case["pad"]) * case["k"], case["experts"]
    if case["op"] == "matmul":
        n, k, active = case["rows"], case["cols"], min(e, kept)
        if case["pass"] == "fwd":
            return {"bytes": (kept * k + active * n * k + slots * n) * es + 4 * (e + 1), "flops": 2 * kept * n * k}
        return {"bytes": (kept * (n + k) + active * n * k + slots * k + e * n * k) * es + 4 * (e + 1), "flops": 4 * kept * n * k}
    d = case["dim"]
    plan = 4 * slots + 4 * (e + 1)
    if case["op"] == "dispatch":
        if case["pass"] == "fwd":
            return {"bytes": (t * d + slots * d) * es + 4 * slots + plan, "flops": 0}
        return {"bytes": (kept * d + t * d) * es + 4 * slots, "flops": kept * d}
    if case["pass"] == "fwd":
        return {"bytes": (kept * d + t * d) * es + 8 * slots, "flops": 2 * kept * d}
    return {"bytes": (kept * d + t * d + slots * d) * es + 4 * slots + plan + 4 * slots, "flops": 3 * kept * d}


# ------------------------------------------------------------------------------------- exact

def exact(case, seed):
    """The definitions in 64 bits: one expert after the other, ranks from sorted pairs (expert, slot)."""
    s = prepare(case, seed)
    if case["op"] == "norm":
        x, w = s["x"].double(), s["weight"].double()
        if case["pass"] == "fwd":
            mean, var = x.mean(dim=1), x.var(dim=1, unbiased=False)
            rstd = (var + s["eps"]).pow(-0.5)
            return torch.addcmul(s["bias"].double(), (x - mean[:, None]) * rstd[:, None], w), mean, rstd
        mean, rstd, dy = s["mean"].double()[:, None], s["rstd"].double()[:, None], s["dy"].double()
        n = x.shape[1]
        xh = (x - mean) * rstd
        a, b = torch.mv(dy, w) / n, torch.mv(dy * xh, w) / n
        return rstd * (dy * w - a[:, None] - b[:, None] * xh), torch.linalg.vecdot(dy, xh, dim=0), dy.sum(dim=0)
    if case["op"] == "matmul":
        x, off = s["x"], s["offsets"].tolist()
        spans = [(e, lo, hi) for e, (lo, hi) in enumerate(zip(off, off[1:])) if hi > lo]
        if case["pass"] == "fwd":
            y = torch.zeros(x.shape[0], case["rows"], dtype=torch.float64, device="cuda")
            for e, lo, hi in spans:
                y[lo:hi] = x[lo:hi].double() @ s["w"][e].double().T
            return y
        dx = torch.zeros(x.shape[0], case["cols"], dtype=torch.float64, device="cuda")
        dw = torch.zeros(s["w"].shape, dtype=torch.float64, device="cuda")
        for e, lo, hi in spans:
            dx[lo:hi] = s["dy"][lo:hi].double() @ s["w"][e].double()
            dw[e] = s["dy"][lo:hi].double().T @ x[lo:hi].double()
        return dx, dw
    if case["op"] == "dispatch" and case["pass"] == "fwd":
        ids, slots = s["ids"].long().reshape(-1), s["ids"].numel()
        pair = torch.where(ids >= 0, ids, case["experts"]) * slots + torch.arange(slots, device="cuda")
        slot = torch.sort(pair).values % slots
        kept = int((ids >= 0).sum())
        xs = torch.zeros(slots, case["dim"], dtype=torch.float64, device="cuda")
        xs[:kept] = s["x"].double()[slot[:kept] // case["k"]]
        return xs, None, None
    rank, slots = s["rank"], s["rank"].numel()
    rows = s["dxs"] if case["op"] == "dispatch" else s["ys"]
    t, j = torch.nonzero(rank >= 0, as_tuple=True)
    at = rank[t, j].long()
    if case["pass"] == "fwd" or case["op"] == "dispatch":
        share = s["weights"][t, j].double() if case["op"] == "combine" else torch.ones(len(t), dtype=torch.float64, device="cuda")
        out = torch.zeros(case["tokens"], case["dim"], dtype=torch.float64, device="cuda")
        return out.index_add_(0, t, rows[at].double() * share[:, None])
    dy = s["dy"].double()
    dys = torch.zeros(slots, case["dim"], dtype=torch.float64, device="cuda")
    dys[at] = dy[t] * s["weights"][t, j].double()[:, None]
    dw = torch.zeros(rank.shape, dtype=torch.float64, device="cuda")
    dw[t, j] = torch.linalg.vecdot(rows[at].double(), dy[t])
    return dys, dw
