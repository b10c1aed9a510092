"""The gated block refuses what it does not take, in the binding and in the C ABI, before any HIP call (no GPU is
needed); the ABI's refusals also run on the host-sanitized copy."""
import ctypes
import os
import subprocess
import sys

import pytest

from test_hostsan import CHILD, ROOT, TESTS, asan_runtime
from test_layer_args import ARG, BF16, DTYPE, F16, F32, L, OK, SHAPE, WS, ops, t, torch  # noqa: F401 (fixtures)

P, Q, R, S, V = 0x10000, 0x8000000, 0x10000000, 0x18000000, 0x20000000   # addresses that are never followed


def test_gated_refusals(L):
    f = L.expert_gated
    x, wg, wu, h, g, u = t(P, 8, 64), t(Q, 32, 64, batch=3), t(R, 32, 64, batch=3), t(S, 8, 32), t(S + 4096, 8, 32), t(S + 8192, 8, 32)
    args = lambda **k: (k.get("x", x), k.get("wg", wg), k.get("wu", wu), k.get("off", V), k.get("act", 0), k.get("h", h), k.get("g", g), k.get("u", u), k.get("ws"), k.get("n", 0), None)
    for name in ("x", "wg", "wu", "h", "g", "u"):
        assert f(*args(**{name: None})) == ARG, name
    assert f(*args(off=None)) == ARG and f(*args(off=V + 2)) == ARG
    for act in (-1, 3, 99):
        assert f(*args(act=act)) == ARG
    for name, bad in (("x", t(P, 8, 64, dtype=F32)), ("wg", t(Q, 32, 64, batch=3, dtype=F16)), ("wu", t(R, 32, 64, batch=3, dtype=F32)),
                      ("h", t(S, 8, 32, dtype=F16)), ("g", t(S + 4096, 8, 32, dtype=F32)), ("u", t(S + 8192, 8, 32, dtype=F32))):
        assert f(*args(**{name: bad})) == DTYPE, name
    for name, bad in (("x", t(P, 8, 63)), ("x", t(P, 8, 64, batch=2)), ("wg", t(Q, 31, 64, batch=3)), ("wu", t(R, 32, 64, batch=2)), ("wu", t(R, 32, 65, batch=3)),
                      ("h", t(S, 7, 32)), ("h", t(S, 8, 33)), ("g", t(S + 4096, 9, 32)), ("u", t(S + 8192, 8, 31)),
                      ("wu", t(R, 32, 64, batch=3, stride=100))):
        assert f(*args(**{name: bad})) == SHAPE, name
    many = dict(wg=t(Q, 32, 64, batch=1025), wu=t(R, 32, 64, batch=1025))
    assert f(*args(**many)) == SHAPE
    assert f(*args(h=t(P + 64, 8, 32))) == ARG and f(*args(h=t(Q + 64, 8, 32))) == ARG and f(*args(g=t(R + 64, 8, 32))) == ARG
    assert f(*args(g=h)) == ARG and f(*args(u=g)) == ARG and f(*args(u=t(V, 8, 32))) == ARG
    one = dict(wg=t(Q, 32, 64), wu=t(R, 32, 64), off=None)
    assert f(*args(**one, ws=V + 8, n=1 << 30)) == WS                        # not aligned
    assert f(*args(**one, ws=S, n=1 << 30)) == ARG and f(*args(**one, ws=P, n=1 << 30)) == ARG
    empty = dict(x=t(None, 0, 64), h=t(None, 0, 32), g=t(None, 0, 32), u=t(None, 0, 32))
    assert f(*args(**one, **empty)) == OK and f(*args(**empty)) == OK
    assert f(*args(**one, x=t(P, 8, 63))) == SHAPE


def test_gated_backward_refusals(L):
    n = ctypes.c_size_t()
    m = ctypes.c_size_t()
    w = lambda rows, inner, dt, e=3: L.mns_expert_gated_workspace_bytes(rows, inner, e, dt, ctypes.byref(m), ctypes.byref(n))
    assert w(8, 32, BF16) == OK and n.value >= 2 * 8 * 32 * 2 and m.value == 0
    assert L.mns_expert_gated_workspace_bytes(8, 32, 3, BF16, None, ctypes.byref(n)) == ARG
    assert L.mns_expert_gated_workspace_bytes(8, 32, 3, BF16, ctypes.byref(m), None) == ARG
    assert w(8, 32, 5) == DTYPE
    for bad in ((-1, 32), (8, 0), ((1 << 24) + 1, 32), (8, (1 << 20) + 1), (8, 32, -1), (8, 32, 1025)):
        assert w(bad[0], bad[1], F32, *bad[2:]) == SHAPE
    assert w(1 << 24, 1 << 20, F32) == OK and n.value == 1 << 47
    assert w(8, 32, BF16, 0) == OK and m.value > 0 and n.value == m.value + 2 * 8 * 32 * 2
    assert w(8, 32, F32, 0) == OK and m.value == 0
    assert w(8, 32, BF16) == OK
    f = L.expert_gated_backward
    x, wg, wu, dh, g, u = t(P, 8, 64), t(Q, 32, 64, batch=3), t(R, 32, 64, batch=3), t(S, 8, 32), t(S + 4096, 8, 32), t(S + 8192, 8, 32)
    dx, dwg, dwu = t(P + 65536, 8, 64), t(Q + (1 << 20), 32, 64, batch=3), t(R + (1 << 20), 32, 64, batch=3)
    names = dict(dh=dh, x=x, wg=wg, wu=wu, g=g, u=u, off=V, act=0, dx=dx, dwg=dwg, dwu=dwu, ws=V + 65536, n=n.value)
    args = lambda **k: (*{**names, **k}.values(), None)
    for name in ("dh", "x", "wg", "wu", "g", "u", "dwg", "dwu", "off"):
        assert f(*args(**{name: None})) == ARG, name
    assert f(*args(dx=None, dwg=None, dwu=None)) == ARG
    assert f(*args(act=7)) == ARG
    assert f(*args(ws=None)) == WS and f(*args(n=n.value - 1)) == WS and f(*args(ws=V + 65544)) == WS
    for name, bad in (("dx", t(P + 65536, 8, 65)), ("dx", t(P + 65536, 7, 64)), ("dwg", t(Q + (1 << 20), 32, 64, batch=2)),
                      ("dwu", t(R + (1 << 20), 33, 64, batch=3)), ("dh", t(S, 8, 31)), ("g", t(S + 4096, 7, 32)), ("u", t(S + 8192, 8, 33))):
        assert f(*args(**{name: bad})) == SHAPE, name
    for name, bad in (("dx", t(P + 65536, 8, 64, dtype=F32)), ("dwu", t(R + (1 << 20), 32, 64, batch=3, dtype=F32)), ("dh", t(S, 8, 32, dtype=F16))):
        assert f(*args(**{name: bad})) == DTYPE, name
    assert f(*args(dx=x)) == ARG and f(*args(dwg=wg)) == ARG and f(*args(dwu=dwg)) == ARG and f(*args(ws=S)) == ARG and f(*args(ws=P + 65536)) == ARG
    empty = dict(dh=t(None, 0, 32), x=t(None, 0, 64), g=t(None, 0, 32), u=t(None, 0, 32), dx=t(None, 0, 64), ws=None, n=0)
    assert f(*args(**empty, dwg=None, dwu=None)) == OK


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
    code = CHILD.replace("test_abi", "test_gated_args").format(root=ROOT, tests=TESTS, path=b.HOSTSAN_LIB)
    r = subprocess.run([sys.executable, "-c", code], env=env, capture_output=True, text=True, timeout=300)
    out = r.stdout + r.stderr
    assert r.returncode == 0 and "AddressSanitizer" not in out and "runtime error:" not in out, out[-4000:]
    assert "ran 2 " in r.stdout, out[-2000:]


def test_binding_refuses(torch, ops):
    x, w, off = torch.zeros(8, 64), torch.zeros(3, 32, 64), torch.zeros(4, dtype=torch.int32)
    g = torch.zeros(8, 32)
    for call in (lambda: ops.expert_gated(x, w, w.clone(), off), lambda: ops.expert_gated(x, w[0], w[1], keep=True),
                 lambda: ops.expert_gated_backward(g, x, w, w, g, g, off)):
        with pytest.raises(ValueError, match="device tensors"):
            call()
    for match, call in (("act must", lambda: ops.expert_gated(x, w, w, off, act="tanh")), ("need offsets", lambda: ops.expert_gated(x, w, w)),
                        ("experts, offsets", lambda: ops.expert_gated(x, w[:2], w[:2], off)), ("w_up has shape", lambda: ops.expert_gated(x, w, w[:, :5], off)),
                        ("x has shape", lambda: ops.expert_gated(x[:, :60], w, w, off)), ("out has shape", lambda: ops.expert_gated(x, w, w, off, out=x)),
                        ("w_gate must", lambda: ops.expert_gated(x, w[0, 0], w[0, 0])), ("gate has shape", lambda: ops.expert_gated_backward(g, x, w, w, g[:5], g, off)),
                        ("dh has shape", lambda: ops.expert_gated_backward(x, x, w, w, g, g, off)),
                        ("nothing wanted", lambda: ops.expert_gated_backward(g, x, w, w, g, g, off, need_input=False, need_weights=False))):
        with pytest.raises(ValueError, match=match):
            call()
    for call in (lambda: ops.expert_gated(x.half(), w, w, off), lambda: ops.expert_gated(x, w, w.half(), off), lambda: ops.expert_gated(x, w, w, off, out=g.half()),
                 lambda: ops.expert_gated(x, w, w, off.long()), lambda: ops.expert_gated_backward(g.half(), x, w, w, g, g, off)):
        with pytest.raises(TypeError):
            call()


def test_binding_refuses_what_autograd_would_have_to_record(torch, ops):
    leaf = lambda *shape: torch.zeros(*shape, requires_grad=True)
    x, w, off, g = torch.zeros(8, 64), torch.zeros(3, 32, 64), torch.zeros(4, dtype=torch.int32), torch.zeros(8, 32)
    calls = [lambda: ops.expert_gated(leaf(8, 64), w, w, off), lambda: ops.expert_gated(x, leaf(3, 32, 64), w, off),
             lambda: ops.expert_gated(x, w, leaf(3, 32, 64), off), lambda: ops.expert_gated(x, w, w, off, out=leaf(8, 32))]
    base = dict(dh=g, x=x, w_gate=w, w_up=w, gate=g, up=g)
    calls += [lambda n=n: ops.expert_gated_backward(**{**base, n: leaf(*base[n].shape)}, offsets=off) for n in base]
    for i, call in enumerate(calls):
        with pytest.raises(RuntimeError, match="autograd"):
            call()
            pytest.fail(f"call {i}")
        with torch.no_grad(), pytest.raises(ValueError, match="device tensors"):
            call()
    from torch.autograd import forward_ad as fwad
    with fwad.dual_level():
        dual = fwad.make_dual(x, torch.ones_like(x))
        for call in (lambda: ops.expert_gated(dual, w, w, off), lambda: ops.expert_gated_backward(g, dual, w, w, g, g, off)):
            with pytest.raises(RuntimeError, match="forward-mode"):
                call()
