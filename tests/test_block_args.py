"""The operators around the layer (rms norm, embeddings, AdamW in 8 bits) refuse what they do not take, in the binding and
in the C ABI, before any HIP call (no GPU is needed); the ABI's refusals also run on the host-sanitized copy."""
import ctypes
import os
import subprocess
import sys

import pytest

from test_hostsan import CHILD, ROOT, TESTS, asan_runtime
from test_layer_args import ARG, BF16, DTYPE, F16, F32, L, OK, SHAPE, WS, ops, t, torch  # noqa: F401 (fixtures)

P, Q, R, S, U = 0x10000, 0x8000000, 0x10000000, 0x18000000, 0x20000000   # addresses that are never followed


def test_rms_norm_refusals(L):
    f = L.rms_norm
    x, r, y, h = t(P, 4, 64), t(Q, 4, 64), t(R, 4, 64), t(S, 4, 64)
    args = lambda **k: (k.get("x", x), k.get("r", r), k.get("w"), k.get("wdt", F32), k.get("eps", 1e-6), k.get("y", y), k.get("h", h),
                        k.get("rstd", U), None)
    assert f(*args(x=None)) == ARG
    assert f(*args(r=None)) == ARG and f(*args(h=None)) == ARG               # one without the other
    assert f(*args(r=t(Q, 4, 64, dtype=F32))) == DTYPE
    assert f(*args(h=t(S, 4, 64, dtype=F16))) == DTYPE
    assert f(*args(y=t(R, 4, 64, dtype=F32))) == DTYPE
    assert f(*args(wdt=F16)) == DTYPE
    assert f(*args(r=t(Q, 3, 64))) == SHAPE
    assert f(*args(h=t(S, 4, 63))) == SHAPE
    assert f(*args(y=t(R, 4, 65))) == SHAPE
    assert f(*args(x=t(P, 4, 64, ld=63))) == SHAPE
    assert f(*args(eps=-1.0)) == ARG and f(*args(eps=float("inf"))) == ARG
    assert f(*args(rstd=None)) == ARG and f(*args(rstd=U + 2)) == ARG
    assert f(*args(w=U + 2)) == ARG
    assert f(*args(y=x)) == ARG and f(*args(h=x)) == ARG and f(*args(y=h)) == ARG
    assert f(*args(y=t(Q + 128, 4, 64))) == ARG                              # over the residual
    assert f(*args(h=t(Q + 128, 4, 64))) == ARG                              # in the residual's buffer, but not it
    assert f(*args(h=t(Q, 4, 64, ld=128), r=t(Q, 4, 64))) == ARG             # the same address, other rows
    assert f(*args(rstd=R + 8)) == ARG and f(*args(rstd=S)) == ARG
    assert f(*args(w=S, wdt=BF16)) == ARG                                    # the weight in h
    e = t(None, 0, 64)
    assert f(*args(x=e, r=e, y=e, h=e, rstd=None)) == OK
    assert f(e, None, None, F32, 1e-6, e, None, None, None) == OK


def test_rms_norm_mx8_refusals(L):
    f = L.rms_norm_mx8
    x, r, h = t(P, 4, 65), t(Q, 4, 65), t(S, 4, 65)
    args = lambda **k: (k.get("x", x), k.get("r", r), None, F32, 1e-6, k.get("q", R), k.get("sc", R + 4096), k.get("h", h), k.get("rstd", U), None)
    assert f(*args(q=None)) == ARG and f(*args(sc=None)) == ARG and f(*args(rstd=None)) == ARG
    assert f(*args(r=None)) == ARG
    assert f(*args(sc=R + 4 * 65 - 1)) == ARG                                # the scales begin in the codes
    assert f(*args(q=P + 1)) == ARG and f(*args(q=Q + 4)) == ARG and f(*args(sc=S + 1)) == ARG
    assert f(*args(rstd=R + 4096)) == ARG
    assert f(*args(x=t(P, 4, 65, dtype=9))) == DTYPE


def test_rms_norm_backward_refusals(L):
    f = L.rms_norm_backward
    n = ctypes.c_size_t()
    assert L.mns_rms_norm_workspace_bytes(t(None, 4, 64), ctypes.byref(n)) == OK and n.value >= 4 * 64
    assert L.mns_rms_norm_workspace_bytes(None, ctypes.byref(n)) == ARG
    assert L.mns_rms_norm_workspace_bytes(t(None, 4, 64), None) == ARG
    assert L.mns_rms_norm_workspace_bytes(t(None, -1, 64), ctypes.byref(n)) == SHAPE
    dy, h, dh, dx = t(P, 4, 64), t(P + 4096, 4, 64), t(Q, 4, 64), t(Q + 4096, 4, 64)
    args = lambda **k: (k.get("dy", dy), k.get("h", h), k.get("rstd", R), k.get("w", R + 4096), k.get("wdt", F32), k.get("dh", dh),
                        k.get("dx", dx), k.get("dw", R + 8192), k.get("ws", S), k.get("n", n.value), None)
    assert f(*args(dy=None)) == ARG and f(*args(dy=None, dh=None)) == ARG and f(*args(h=None)) == ARG and f(*args(dx=None)) == ARG
    assert f(*args(rstd=None)) == ARG
    assert f(*args(ws=None)) == WS and f(*args(n=n.value - 1)) == WS and f(*args(ws=S + 8)) == WS
    assert f(*args(dx=dy)) == ARG and f(*args(dx=h)) == ARG
    assert f(*args(dx=t(Q + 64, 4, 64))) == ARG                              # in dh's buffer, but not it
    assert f(*args(dw=Q)) == ARG and f(*args(dw=R + 4096)) == ARG and f(*args(ws=Q)) == ARG and f(*args(dw=S)) == ARG
    assert f(*args(dh=t(Q, 4, 64, dtype=F32))) == DTYPE and f(*args(dh=t(Q, 5, 64))) == SHAPE
    assert f(*args(wdt=F16)) == DTYPE and f(*args(dw=R + 8194)) == ARG


def test_embed_refusals(L):
    f = L.embed
    table, y = t(P, 100, 64), t(Q, 8, 64)
    args = lambda **k: (k.get("tok", R), k.get("b", 4), k.get("table", table), k.get("scale", 1.0), k.get("y", y), None)
    assert f(*args(tok=None)) == ARG and f(*args(tok=R + 2)) == ARG and f(*args(tok=R + 4, b=8)) == ARG
    assert f(*args(b=2)) == DTYPE
    assert f(*args(table=None)) == ARG and f(*args(y=None)) == ARG
    assert f(*args(y=t(Q, 8, 64, dtype=F32))) == DTYPE
    assert f(*args(y=t(Q, 8, 63))) == SHAPE and f(*args(table=t(P, 0, 64))) == SHAPE
    assert f(*args(table=t(P, 100, 64, batch=2))) == SHAPE and f(*args(y=t(Q, 8, 64, batch=2))) == SHAPE
    assert f(*args(scale=float("nan"))) == ARG
    assert f(*args(y=t(P + 640, 8, 64))) == ARG and f(*args(tok=Q + 64)) == ARG
    assert f(*args(y=t(None, 0, 64), tok=None)) == OK


def test_embed_backward_refusals(L):
    n = ctypes.c_size_t()
    w = L.mns_embed_workspace_bytes
    assert w(8, 100, 64, ctypes.byref(n)) == OK and n.value >= 100 + 4 * 4 * 8
    assert w(8, 100, 64, None) == ARG
    for bad in ((-1, 100, 64), (8, 0, 64), (8, 100, 0), ((1 << 24) + 1, 100, 64), (8, (1 << 24) + 1, 64), (8, 100, (1 << 20) + 1)):
        assert w(*bad, ctypes.byref(n)) == SHAPE
    assert w(1 << 24, 1 << 24, 1 << 20, ctypes.byref(n)) == OK and n.value > 1 << 40
    assert w(8, 100, 64, ctypes.byref(n)) == OK
    f = L.embed_backward
    dy, dt = t(P, 8, 64), t(Q, 100, 64)
    args = lambda **k: (k.get("dy", dy), k.get("tok", R), k.get("b", 8), k.get("scale", 1.0), k.get("dt", dt), k.get("ws", S), k.get("n", n.value), None)
    assert f(*args(tok=None)) == ARG and f(*args(b=1)) == DTYPE and f(*args(tok=R + 4)) == ARG
    assert f(*args(dt=t(Q, 100, 64, dtype=F32))) == DTYPE and f(*args(dt=t(Q, 100, 65))) == SHAPE and f(*args(dt=t(Q, 0, 64))) == SHAPE
    assert f(*args(ws=None)) == WS and f(*args(n=n.value - 1)) == WS and f(*args(ws=S + 4)) == WS
    assert f(*args(dt=t(P + 512, 100, 64))) == ARG and f(*args(ws=P)) == ARG and f(*args(ws=Q + 64)) == ARG and f(*args(tok=S + 8)) == ARG
    assert f(*args(scale=float("inf"))) == ARG


def test_adamw8_refusals(L):
    from newton_schulz_matrix_muon_amd.ops import MnsAdamw8Params
    arr = lambda *v: (ctypes.c_void_p * len(v))(*v)
    good = dict(n=2, p=(P, P + 4096), g=(Q, Q + 4096), m=(R, R + 101), ms=(R + 4096, R + 4100), r=(S, S + 4096), rs=(S + 8192, S + 8300),
                numels=(100, 50), dt=BF16)

    def call(hyper=(1e-3, 0.9, 0.95, 1e-8, 0.1, 1, 0, 0), **k):
        a = {**good, **k}
        lists = [None if a[i] is None else arr(*a[i]) for i in ("p", "g", "m", "ms", "r", "rs")]
        return L.adamw8_step(a["n"], *lists, (ctypes.c_int64 * len(a["numels"]))(*a["numels"]), a["dt"], ctypes.byref(MnsAdamw8Params(*hyper)), None)
    for name in ("p", "g", "m", "ms", "r", "rs"):
        assert call(**{name: None}) == ARG
        assert call(**{name: (None, good[name][1])}) == ARG
    assert call(n=0) == ARG and call(dt=5) == DTYPE and call(numels=(-1, 5)) == ARG and call(numels=((1 << 34) + 1, 5)) == SHAPE
    assert call(p=(P + 1, P + 4096)) == ARG and call(g=(Q, Q + 4097)) == ARG
    assert call(m=(R, R + 99)) == ARG                                        # the second tensor's codes begin in the first's
    assert call(rs=(S + 8192, S + 8195)) == ARG                              # ... and its powers
    assert call(p=(P, P)) == ARG and call(g=(P, Q)) == ARG and call(r=(R + 4096, S)) == ARG
    for i, bad in ((0, float("nan")), (0, 1e39), (1, 1.0), (1, -0.1), (2, 1.0), (3, -1e-8), (4, float("inf")), (5, 0), (6, 2)):
        h = [1e-3, 0.9, 0.95, 1e-8, 0.1, 1, 0, 0]
        h[i] = bad
        assert call(hyper=tuple(h)) == ARG, (i, bad)
    none = (None, None)
    assert call(numels=(0, 0), p=none, g=none, m=none, ms=none, r=none, rs=none) == OK


def test_abi_refusals_under_host_sanitizers():
    from newton_schulz_matrix_muon_amd import build as b
    rt = asan_runtime()
    if os.path.exists("/dev/kfd") or rt is None or not os.path.exists(b.LIB):
        pytest.skip("needs the CPU, an ASan runtime and the built library")
    if not os.path.exists(b.HOSTSAN_LIB) or os.path.getmtime(b.HOSTSAN_LIB) < os.path.getmtime(b.LIB):
        b.build_hostsan()
    env = dict(os.environ, ASAN_OPTIONS="detect_leaks=0:halt_on_error=1:verify_asan_link_order=0",
               UBSAN_OPTIONS="halt_on_error=1:print_stacktrace=1")
    env["LD_PRELOAD"] = rt + (":" + env["LD_PRELOAD"] if env.get("LD_PRELOAD") else "")
    code = CHILD.replace("test_abi", "test_block_args").format(root=ROOT, tests=TESTS, path=b.HOSTSAN_LIB)
    r = subprocess.run([sys.executable, "-c", code], env=env, capture_output=True, text=True, timeout=300)
    out = r.stdout + r.stderr
    assert r.returncode == 0 and "AddressSanitizer" not in out and "runtime error:" not in out, out[-4000:]
    assert "ran 6 " in r.stdout, out[-2000:]


# ------------------------------------------------------------------------------- the binding

def test_binding_refuses_shapes_types_and_host_tensors(torch, ops):
    x, w, r = torch.zeros(4, 64), torch.ones(64), torch.zeros(4)
    device = pytest.raises(ValueError, match="device tensors")
    for call in (lambda: ops.rms_norm(x, w, residual=x.clone()), lambda: ops.rms_norm_mx8(x), lambda: ops.rms_norm_backward(x, x, r, w, dh=x),
                 lambda: ops.embed(torch.zeros(3, 2, dtype=torch.int64), x), lambda: ops.embed_backward(x, torch.zeros(4, dtype=torch.int32), 9)):
        with device:
            call()
    for match, call in [("weight has shape", lambda: ops.rms_norm(x, w[:5])), ("residual has shape", lambda: ops.rms_norm(x, w, residual=x[:3])),
                        ("without residual", lambda: ops.rms_norm(x, w, residual_out=x)), ("out has shape", lambda: ops.rms_norm(x, w, out=x[:2])),
                        ("rstd has shape", lambda: ops.rms_norm_backward(x, x, r[:3], w)), ("dh has shape", lambda: ops.rms_norm_backward(x, x, r, w, dh=x[:1])),
                        ("contiguous", lambda: ops.rms_norm(x.t())), ("no rows", lambda: ops.embed(torch.zeros(3, dtype=torch.int64), x[:0])),
                        ("out has shape", lambda: ops.embed(torch.zeros(3, dtype=torch.int64), x, out=x)),
                        ("dy has shape", lambda: ops.embed_backward(x, torch.zeros(3, dtype=torch.int64), 9)),
                        ("rows must be", lambda: ops.embed_backward(x, torch.zeros(4, dtype=torch.int64), 0)),
                        ("out has shape", lambda: ops.embed_backward(x, torch.zeros(4, dtype=torch.int64), 9, out=x)),
                        ("contiguous", lambda: ops.embed(torch.zeros(6, 2, dtype=torch.int64).t(), x)),
                        ("2-D", lambda: ops.embed_backward(torch.zeros(2, 2, 64), torch.zeros(4, dtype=torch.int64), 9))]:
        with pytest.raises(ValueError, match=match):
            call()
    for call in (lambda: ops.rms_norm(x.double()), lambda: ops.rms_norm(x, w.half()), lambda: ops.rms_norm(x, residual=x.half()),
                 lambda: ops.rms_norm(x, out=x.bfloat16()), lambda: ops.rms_norm_backward(x.half(), x, r), lambda: ops.rms_norm_backward(x, x, r.double()),
                 lambda: ops.embed(torch.zeros(3), x), lambda: ops.embed(torch.zeros(3, dtype=torch.int16), x),
                 lambda: ops.embed_backward(x, torch.zeros(4, dtype=torch.int64), 9, out=torch.zeros(9, 64).half())):
        with pytest.raises(TypeError):
            call()


def test_binding_refuses_adamw8_lists(torch, ops):
    p = torch.zeros(100)
    s = ops.adamw8_state(p)
    ok = lambda **k: ops.adamw8_step(**{**dict(params=[p], grads=[p.clone()], states=[s], lr=1e-3, step=1), **k})
    with pytest.raises(ValueError, match="device tensors"):
        ok()
    with pytest.raises(TypeError):
        ops.adamw8_step([p], [p], [s], lr=1e-3)                              # no step
    for match, k in (("equal length", dict(grads=[])), ("equal length", dict(params=[], grads=[], states=[])), ("step", dict(step=0)),
                     ("seed", dict(seed=-1)), ("seed", dict(seed=2 ** 64)), ("four tensors", dict(states=[s[:3]])),
                     ("elements", dict(states=[ops.adamw8_state(p[:99])])), ("elements", dict(grads=[p[:99]])),
                     ("contiguous", dict(grads=[torch.zeros(200)[::2]]))):
        with pytest.raises(ValueError, match=match):
            ok(**k)
    for k in (dict(grads=[p.half()]), dict(params=[p.double()], grads=[p.double()]), dict(states=[(p, *s[1:])]),
              dict(states=[(s[0], s[0].view(torch.uint8)[:4].float(), *s[2:])]), dict(params=[p, p.half()], grads=[p, p.half()], states=[s, s])):
        with pytest.raises(TypeError):
            ok(**k)
    a = ops.adamw8_state(torch.zeros(0))
    assert [t.numel() for t in a] == [0, 0, 0, 0]


def test_binding_refuses_what_autograd_would_have_to_record(torch, ops):
    leaf = lambda *shape: torch.zeros(*shape, requires_grad=True)
    x, r, tok = torch.zeros(8, 64), torch.zeros(8), torch.zeros(8, dtype=torch.int64)
    calls = [lambda: ops.rms_norm(leaf(8, 64)), lambda: ops.rms_norm(x, leaf(64)), lambda: ops.rms_norm(x, residual=leaf(8, 64)),
             lambda: ops.rms_norm(x, out=leaf(8, 64)), lambda: ops.rms_norm(x, residual=x, residual_out=leaf(8, 64)),
             lambda: ops.rms_norm_mx8(leaf(8, 64)), lambda: ops.rms_norm_backward(leaf(8, 64), x, r), lambda: ops.rms_norm_backward(x, x, leaf(8)),
             lambda: ops.rms_norm_backward(x, x, r, dh=leaf(8, 64)), lambda: ops.rms_norm_backward(x, x, r, out=leaf(8, 64)),
             lambda: ops.embed(tok, leaf(9, 64)), lambda: ops.embed(tok, x, out=leaf(8, 64)), lambda: ops.embed_backward(leaf(8, 64), tok, 9),
             lambda: ops.embed_backward(x, tok, 9, out=leaf(9, 64))]
    for i, call in enumerate(calls):
        with pytest.raises(RuntimeError, match="autograd"):
            call()
            pytest.fail(f"call {i}")
        with torch.no_grad(), pytest.raises(ValueError, match="device tensors"):
            call()
    from torch.autograd import forward_ad as fwad
    with fwad.dual_level():
        dual = fwad.make_dual(x, torch.ones_like(x))
        for call in (lambda: ops.rms_norm(dual), lambda: ops.rms_norm(x, residual=dual), lambda: ops.rms_norm_mx8(dual),
                     lambda: ops.rms_norm_backward(dual, x, r), lambda: ops.embed(tok, dual), lambda: ops.embed_backward(dual, tok, 9)):
            with pytest.raises(RuntimeError, match="forward-mode"):
                call()
