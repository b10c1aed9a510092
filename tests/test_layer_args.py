"""The layer operators refuse what they do not take, in the binding and in the C ABI, before any
HIP call (no GPU is needed); the ABI's refusals also run on the host-sanitized copy."""
import ctypes
import os
import subprocess
import sys

import pytest

from test_hostsan import CHILD, ROOT, TESTS, asan_runtime

OK, ARG, DTYPE, SHAPE, WS = 0, -1, -2, -3, -4
F32, BF16, F16 = 0, 1, 2
P, Q, R = 0x10000, 0x8000000, 0x10000000   # addresses that are never followed


@pytest.fixture(scope="module")
def L():
    from newton_schulz_matrix_muon_amd import ops
    return ops.lib()


@pytest.fixture(scope="module")
def torch():
    import torch
    return torch


@pytest.fixture(scope="module")
def ops():
    from newton_schulz_matrix_muon_amd import ops
    return ops


def t(ptr, rows, cols, dtype=BF16, batch=1, ld=None, stride=None):
    from newton_schulz_matrix_muon_amd.ops import MnsTensor
    ld = cols if ld is None else ld
    return ctypes.byref(MnsTensor(ptr, dtype, batch, rows, cols, ld, rows * ld if stride is None else stride))


def test_layer_norm_refusals(L):
    f = L.layer_norm
    x, y = t(P, 4, 64), t(Q, 4, 64)
    assert f(None, None, None, F32, 1e-5, y, P, P, None) == ARG
    assert f(t(P, 4, 64, dtype=7), None, None, F32, 1e-5, y, R, R + 64, None) == DTYPE
    assert f(t(P, 4, 64, dtype=F16), None, None, F32, 1e-5, y, R, R + 64, None) == DTYPE
    assert f(x, None, None, F16, 1e-5, y, R, R + 64, None) == DTYPE
    assert f(x, None, None, F32, 1e-5, t(Q, 4, 63), R, R + 64, None) == SHAPE
    assert f(t(P, 4, 64, ld=63), None, None, F32, 1e-5, y, R, R + 64, None) == SHAPE
    assert f(t(P, 4, 64, batch=2, stride=200), None, None, F32, 1e-5, t(Q, 4, 64, batch=2), R, R + 64, None) == SHAPE
    assert f(t(P, 4, 0), None, None, F32, 1e-5, t(Q, 4, 0), R, R + 64, None) == SHAPE
    assert f(t(P, 1 << 25, 8), None, None, F32, 1e-5, t(Q, 1 << 25, 8), R, R + 64, None) == SHAPE
    assert f(x, None, None, F32, -1.0, y, R, R + 64, None) == ARG
    assert f(x, None, None, F32, float("nan"), y, R, R + 64, None) == ARG
    assert f(x, None, None, F32, 1e-5, y, None, R, None) == ARG
    assert f(x, None, None, F32, 1e-5, x, R, R + 64, None) == ARG            # in place
    assert f(x, None, None, F32, 1e-5, y, R, R + 4, None) == ARG             # mean and rstd overlap
    assert f(t(P + 1, 4, 64), None, None, F32, 1e-5, y, R, R + 64, None) == ARG   # not aligned to an element
    assert f(t(None, 0, 64), None, None, F32, 1e-5, t(None, 0, 64), None, None, None) == OK   # nothing to do


def test_layer_norm_backward_refusals(L):
    f = L.layer_norm_backward
    n = ctypes.c_size_t()
    assert L.mns_layer_norm_workspace_bytes(t(None, 4, 64), ctypes.byref(n)) == OK and n.value >= 4 * 2 * 64
    assert L.mns_layer_norm_workspace_bytes(None, ctypes.byref(n)) == ARG
    assert L.mns_layer_norm_workspace_bytes(t(None, -1, 64), ctypes.byref(n)) == SHAPE
    x, dy, dx = t(P, 4, 64), t(P + 4096, 4, 64), t(Q, 4, 64)
    W, DW, DB, S = R, R + 4096, R + 8192, R + 65536
    args = lambda **k: (k.get("dy", dy), k.get("x", x), k.get("mean", R + 12288), R + 16384, W, k.get("wdt", F32), k.get("dx", dx),
                        DW, k.get("db", DB), k.get("ws", S), k.get("n", n.value), None)
    assert f(*args(ws=None)) == WS
    assert f(*args(n=n.value - 1)) == WS
    assert f(*args(ws=S + 4)) == WS
    assert f(*args(dx=x)) == ARG
    assert f(*args(db=DW)) == ARG
    assert f(*args(db=S)) == ARG
    assert f(*args(mean=None)) == ARG
    assert f(*args(dy=t(P + 4096, 4, 64, dtype=F32))) == DTYPE
    assert f(*args(dy=t(P + 4096, 3, 64))) == SHAPE
    assert f(*args(wdt=F16)) == DTYPE


def test_expert_sort_refusals(L):
    n = ctypes.c_size_t()
    assert L.mns_expert_sort_workspace_bytes(16, 8, ctypes.byref(n)) == OK and n.value == 0
    assert L.mns_expert_sort_workspace_bytes(100000, 8, ctypes.byref(n)) == OK and n.value > 0
    assert L.mns_expert_sort_workspace_bytes(100000, 8, None) == ARG
    assert L.mns_expert_sort_workspace_bytes(-1, 8, ctypes.byref(n)) == SHAPE
    for e in (0, 1025, -3):
        assert L.mns_expert_sort_workspace_bytes(8, e, ctypes.byref(n)) == SHAPE
    f = L.expert_sort
    assert f(P, 2, 16, 8, Q, R, None, 0, None) == DTYPE
    assert f(None, 4, 16, 8, Q, R, None, 0, None) == ARG
    assert f(P, 4, 16, 8, None, R, None, 0, None) == ARG
    assert f(P, 4, 16, 8, Q, None, None, 0, None) == ARG
    assert f(P + 4, 8, 16, 8, Q, R, None, 0, None) == ARG
    assert f(P, 4, 16, 2000, Q, R, None, 0, None) == SHAPE
    assert f(P, 4, (1 << 24) + 1, 8, Q, R, None, 0, None) == SHAPE
    assert f(P, 4, 100000, 8, Q, R, None, 0, None) == WS
    assert f(P, 4, 16, 8, Q, P + 32, None, 0, None) == ARG                   # rank over the picks
    assert f(P, 4, 16, 8, R + 60, R, None, 0, None) == ARG                   # offsets over rank


def test_rows_refusals(L):
    x, xs, rank, off = t(P, 4, 64), t(Q, 8, 64), R, R + 4096
    f = L.expert_dispatch
    assert f(x, rank, 2, off, 8, t(Q, 9, 64), None) == SHAPE
    assert f(x, rank, 0, off, 8, xs, None) == SHAPE
    assert f(x, rank, 2, off, 0, xs, None) == SHAPE
    assert f(x, rank, 2, off, 1025, xs, None) == SHAPE
    assert f(x, None, 2, off, 8, xs, None) == ARG
    assert f(x, rank, 2, None, 8, xs, None) == ARG
    assert f(x, rank, 2, off, 8, t(Q, 8, 63), None) == SHAPE
    assert f(x, rank, 2, off, 8, t(Q, 8, 64, dtype=F16), None) == DTYPE
    assert f(x, rank, 2, off, 8, t(P + 256, 8, 64), None) == ARG
    assert f(t(P, 4, 64, batch=2), rank, 2, off, 8, xs, None) == SHAPE
    assert f(x, rank, 2, off, 8, t(R - 64, 8, 64), None) == ARG              # over rank
    assert f(t(P, 1 << 23, 8), rank, 4, off, 8, t(Q, 1 << 25, 8), None) == SHAPE
    assert f(t(None, 0, 64), None, 2, off, 8, t(None, 0, 64), None) == OK
    assert L.expert_dispatch_backward(xs, rank, 3, x, None) == SHAPE
    assert L.expert_dispatch_backward(xs, rank, 2, t(Q + 64, 4, 64), None) == ARG
    w = R + 8192
    assert L.expert_combine(xs, w, F16, rank, 2, x, None) == DTYPE
    assert L.expert_combine(xs, None, F32, rank, 2, x, None) == ARG
    assert L.expert_combine(xs, w + 2, F32, rank, 2, x, None) == ARG
    g = L.expert_combine_backward
    dys = t(Q + 65536, 8, 64)
    assert g(x, xs, w, F32, rank, 2, off, 8, xs, w + 4096, None) == ARG
    assert g(x, xs, w, F32, rank, 2, off, 8, dys, w, None) == ARG
    assert g(x, xs, w, F32, rank, 2, off, 8, dys, None, None) == ARG
    assert g(x, xs, w, F32, rank, 2, None, 8, dys, w + 4096, None) == ARG
    assert g(x, t(Q, 8, 32), w, F32, rank, 2, off, 8, dys, w + 4096, None) == SHAPE


def test_product_refusals(L):
    off = R
    x, w, y, dw = t(P, 8, 64), t(Q, 32, 64, batch=3), t(P + 65536, 8, 32), t(Q + (1 << 20), 32, 64, batch=3)
    f = L.expert_matmul
    assert f(t(P, 8, 63), w, off, y, None) == SHAPE
    assert f(x, w, off, t(P + 65536, 7, 32), None) == SHAPE
    assert f(x, w, off, t(P + 65536, 8, 31), None) == SHAPE
    assert f(x, t(Q, 32, 64, batch=1025), off, y, None) == SHAPE
    assert f(x, t(Q, 32, 64, batch=3, dtype=F16), off, y, None) == DTYPE
    assert f(x, w, None, y, None) == ARG
    assert f(x, w, off, t(P + 128, 8, 32), None) == ARG
    assert f(x, w, off + 2, y, None) == ARG
    assert f(x, t(Q, 32, 64, batch=3, stride=100), off, y, None) == SHAPE
    assert f(t(None, 0, 64), w, off, t(None, 0, 32), None) == OK
    assert L.expert_matmul_grad_input(y, w, off, t(P, 8, 63), None) == SHAPE
    assert L.expert_matmul_grad_input(y, w, off, y, None) == SHAPE
    assert L.expert_matmul_grad_weight(y, x, off, t(Q, 32, 63, batch=3), None) == SHAPE
    assert L.expert_matmul_grad_weight(y, t(P, 7, 64), off, dw, None) == SHAPE
    assert L.expert_matmul_grad_weight(y, x, off, t(P, 32, 64, batch=3), None) == ARG


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
    code = CHILD.replace("test_abi", "test_layer_args").format(root=ROOT, tests=TESTS, path=b.HOSTSAN_LIB)
    r = subprocess.run([sys.executable, "-c", code], env=env, capture_output=True, text=True, timeout=300)
    out = r.stdout + r.stderr
    assert r.returncode == 0 and "AddressSanitizer" not in out and "runtime error:" not in out, out[-4000:]
    assert "ran 5 " in r.stdout, out[-2000:]


# ------------------------------------------------------------------------------- the binding

def test_binding_refuses_shapes_types_and_host_tensors(torch, ops):
    x, w = torch.zeros(4, 64), torch.ones(64)
    with pytest.raises(ValueError, match="device tensors"):
        ops.layer_norm(x, w, w)
    with pytest.raises(ValueError, match="weight has shape"):
        ops.layer_norm(x, torch.ones(63))
    with pytest.raises(TypeError):
        ops.layer_norm(x, w.half())
    with pytest.raises(TypeError, match="bias"):
        ops.layer_norm(x.bfloat16(), w, w.bfloat16())
    with pytest.raises(TypeError):
        ops.layer_norm(x.double())
    with pytest.raises(ValueError):
        ops.layer_norm(x.t())
    with pytest.raises(ValueError, match="mean"):
        ops.layer_norm_backward(x, x, torch.zeros(3), torch.zeros(4), w)
    with pytest.raises(TypeError, match="dy"):
        ops.layer_norm_backward(x.half(), x, torch.zeros(4), torch.zeros(4), w)
    ids, rank, off = torch.zeros(4, 2, dtype=torch.int64), torch.zeros(4, 2, dtype=torch.int32), torch.zeros(4, dtype=torch.int32)
    for bad in (0, 1025):
        with pytest.raises(ValueError, match="num_experts"):
            ops.expert_sort(ids, bad)
    with pytest.raises(TypeError):
        ops.expert_sort(ids.float(), 3)
    with pytest.raises(ValueError, match="contiguous"):
        ops.expert_sort(ids.t(), 3)
    with pytest.raises(ValueError, match="tokens, k"):
        ops.expert_sort(ids[0], 3)
    with pytest.raises(ValueError, match="device tensors"):
        ops.expert_sort(ids, 3)
    with pytest.raises(TypeError, match="rank"):
        ops.expert_dispatch(x, ids, off)
    with pytest.raises(ValueError, match="rank has shape"):
        ops.expert_dispatch(x, rank[:3], off)
    with pytest.raises(ValueError, match="offsets"):
        ops.expert_dispatch(x, rank, off[:1])
    with pytest.raises(ValueError, match="device tensors"):
        ops.expert_dispatch(x, rank, off)
    with pytest.raises(ValueError, match="dxs has shape"):
        ops.expert_dispatch_backward(x, rank)
    xs, wt = torch.zeros(8, 64), torch.zeros(4, 2)
    with pytest.raises(ValueError, match="weights has shape"):
        ops.expert_combine(xs, wt[:, :1].contiguous(), rank)
    with pytest.raises(TypeError, match="weights"):
        ops.expert_combine(xs, wt.half(), rank)
    with pytest.raises(ValueError, match="dy has shape"):
        ops.expert_combine_backward(xs, xs, wt, rank, off)
    W = torch.zeros(3, 32, 64)
    with pytest.raises(ValueError, match="experts"):
        ops.expert_matmul(xs, W[:2], off)
    with pytest.raises(ValueError, match="x has shape"):
        ops.expert_matmul(xs[:, :32], W, off)
    with pytest.raises(TypeError, match="x is"):
        ops.expert_matmul(xs.half(), W, off)
    with pytest.raises(ValueError, match="out has shape"):
        ops.expert_matmul_grad_weight(torch.zeros(8, 32), xs, off, out=W[:2])
    with pytest.raises(ValueError, match="device tensors"):
        ops.expert_matmul_backward(torch.zeros(8, 32), xs, W, off)


def test_binding_refuses_what_autograd_would_have_to_record(torch, ops):
    w = torch.zeros(3, 32, 64, requires_grad=True)
    off = torch.zeros(4, dtype=torch.int32)
    with pytest.raises(RuntimeError, match="autograd"):
        ops.expert_matmul(torch.zeros(8, 64), w, off)
    with pytest.raises(RuntimeError, match="autograd"):
        ops.layer_norm(torch.zeros(8, 64, requires_grad=True))
    with torch.no_grad(), pytest.raises(ValueError, match="device tensors"):
        ops.expert_matmul(torch.zeros(8, 64), w, off)


def test_binding_refuses_forward_mode_tangents(torch, ops):
    """A dual tensor's tangent would be lost: refused, with gradients enabled or not."""
    from torch.autograd import forward_ad as fwad
    x, w, off = torch.zeros(8, 64), torch.zeros(3, 32, 64), torch.zeros(4, dtype=torch.int32)
    stat, rank, picks = torch.zeros(8), torch.zeros(8, 1, dtype=torch.int32), torch.ones(8, 1)
    with fwad.dual_level():
        dual = lambda t: fwad.make_dual(t, torch.ones_like(t))
        calls = [lambda: ops.layer_norm(dual(x)), lambda: ops.layer_norm(x, dual(torch.ones(64))),
                 lambda: ops.layer_norm_backward(dual(x), x, stat, stat), lambda: ops.expert_dispatch(dual(x), rank, off),
                 lambda: ops.expert_dispatch_backward(dual(x), rank), lambda: ops.expert_combine(x, dual(picks), rank),
                 lambda: ops.expert_combine_backward(x, dual(x), picks, rank, off), lambda: ops.expert_matmul(x, dual(w), off),
                 lambda: ops.expert_matmul_grad_input(dual(x[:, :32].contiguous()), w, off),
                 lambda: ops.expert_matmul_grad_weight(x[:, :32], dual(x), off), lambda: ops.expert_matmul_backward(x[:, :32], dual(x), w, off)]
        for call in calls:
            with pytest.raises(RuntimeError, match="forward-mode"):
                call()
            with torch.no_grad(), pytest.raises(RuntimeError, match="forward-mode"):
                call()
        # a tensor without a tangent passes this check, and so does a dual where torch itself drops tangents
        with pytest.raises(ValueError, match="device tensors"):
            ops.layer_norm(x)
        with fwad._set_fwd_grad_enabled(False), pytest.raises(ValueError, match="device tensors"):
            ops.layer_norm(dual(x))


def test_binding_refuses_results_and_statistics_that_autograd_tracks(torch, ops):
    """`out` that requires grad would be overwritten behind autograd's back, kept statistics lose their gradient."""
    leaf = lambda *shape: torch.zeros(*shape, requires_grad=True)
    x, w, off = torch.zeros(8, 64), torch.zeros(3, 32, 64), torch.zeros(4, dtype=torch.int32)
    y, stat, rank, picks = torch.zeros(8, 32), torch.zeros(8), torch.zeros(8, 1, dtype=torch.int32), torch.ones(8, 1)
    calls = [lambda: ops.layer_norm(x, out=leaf(8, 64)), lambda: ops.layer_norm_backward(x, x, stat, stat, out=leaf(8, 64)),
             lambda: ops.layer_norm_backward(x, x, leaf(8), stat), lambda: ops.layer_norm_backward(x, x, stat, leaf(8)),
             lambda: ops.expert_dispatch(x, rank, off, out=leaf(8, 64)), lambda: ops.expert_dispatch_backward(x, rank, out=leaf(8, 64)),
             lambda: ops.expert_combine(x, picks, rank, out=leaf(8, 64)),
             lambda: ops.expert_combine_backward(x, x, picks, rank, off, out=leaf(8, 64)),
             lambda: ops.expert_matmul(x, w, off, out=leaf(8, 32)), lambda: ops.expert_matmul_grad_input(y, w, off, out=leaf(8, 64)),
             lambda: ops.expert_matmul_grad_weight(y, x, off, out=leaf(3, 32, 64))]
    for i, call in enumerate(calls):
        with pytest.raises(RuntimeError, match="autograd"):
            call()
            pytest.fail(f"call {i}")
        with torch.no_grad(), pytest.raises(ValueError, match="device tensors"):
            call()
