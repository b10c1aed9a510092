"""Thin ctypes binding of libmuon_ns.so (include/muon_ns.h).

Argument marshalling only: torch tensors are described to the C ABI by pointer, dtype,
shape and strides, the workspace is a torch allocation, and the stream is torch's
current stream. Every step of the computation runs in the library's HIP kernels. If the
library is missing this module raises; there is no fallback path.
"""
from __future__ import annotations

import array
import ctypes
import os
import warnings
from typing import NamedTuple, Optional, Sequence

PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(PKG, "libmuon_ns.so")

F32, BF16, F16 = 0, 1, 2
STANDARD, GRAM = 0, 1
STATUS = {0: "MNS_OK", -1: "MNS_ERR_ARG", -2: "MNS_ERR_DTYPE", -3: "MNS_ERR_SHAPE",
          -4: "MNS_ERR_WORKSPACE", -5: "MNS_ERR_HIP", -6: "MNS_ERR_UNSUPPORTED"}

# Defaults of the guide's optimizer listing (lr, momentum, weight decay, steps, eps).
DEFAULT_STEPS = 5
DEFAULT_EPS = 1e-7
STABILIZED_RESTART_MASK = 1 << 2


class MnsTensor(ctypes.Structure):
    _fields_ = [("ptr", ctypes.c_void_p), ("dtype", ctypes.c_int32), ("batch", ctypes.c_int64),
                ("rows", ctypes.c_int64), ("cols", ctypes.c_int64), ("ld", ctypes.c_int64),
                ("stride", ctypes.c_int64)]


class MnsNsParams(ctypes.Structure):
    _fields_ = [("steps", ctypes.c_int32), ("coeffs", ctypes.POINTER(ctypes.c_float)),
                ("eps", ctypes.c_float), ("iter_dtype", ctypes.c_int32),
                ("restart_mask", ctypes.c_uint32)]


class MnsStepParams(ctypes.Structure):
    _fields_ = [("lr", ctypes.c_float), ("momentum", ctypes.c_float),
                ("weight_decay", ctypes.c_float), ("scale_coeff", ctypes.c_float),
                ("nesterov", ctypes.c_int32), ("variant", ctypes.c_int32)]


class MnsError(RuntimeError):
    def __init__(self, code: int, what: str):
        self.code = code
        super().__init__(f"{what}: {STATUS.get(code, code)} ({_lib().mns_status_string(code).decode()})"
                         + (f", hipError {_lib().mns_last_hip_error()}" if code == -5 else ""))


_LIB = None


def _lib():
    global _LIB
    if _LIB is None:
        if not os.path.exists(LIB_PATH):
            raise ImportError(f"{LIB_PATH} is missing: build it with "
                              "`python -m newton_schulz_matrix_muon_amd.build`")
        # torch carries its own HIP runtime (soname libamdhip64.so.7). Loading it first makes
        # the library bind to that same runtime; loaded the other way round, the library would
        # pull in the system runtime and the process would hold two, and the library's one
        # would not see the device torch's tensors and streams live on.
        _torch()
        _LIB = declare(ctypes.CDLL(LIB_PATH))
    return _LIB


def declare(lib):
    """Set the argument and result types of every C function on a loaded copy of the library
    (needs no GPU and does not import torch); returns the library."""
    P = ctypes.POINTER
    vp, sz = ctypes.c_void_p, ctypes.c_size_t
    lib.mns_workspace_bytes.argtypes = [ctypes.c_int, P(MnsTensor), P(MnsNsParams),
                                        ctypes.c_int64, P(sz)]
    for fn in (lib.muon_ns_batched, lib.gram_ns_batched):
        fn.argtypes = [P(MnsTensor), P(MnsTensor), P(MnsNsParams), vp, sz, vp, vp]
    lib.muon_step.argtypes = [P(MnsTensor), P(MnsTensor), P(MnsTensor), P(MnsTensor),
                              P(MnsStepParams), P(MnsNsParams), vp, sz, vp, vp]
    lib.muon_step_noalloc.argtypes = [P(MnsTensor), P(MnsTensor), P(MnsTensor), P(MnsTensor),
                                      P(MnsStepParams), P(MnsNsParams), vp, vp]
    lib.gram_ns_trace.argtypes = [P(MnsTensor), P(MnsTensor), P(MnsNsParams), vp, sz, vp, vp]
    lib.mns_workspace_bytes_grouped.argtypes = [ctypes.c_int, ctypes.c_int, P(MnsTensor),
                                                P(MnsNsParams), P(sz)]
    for fn in (lib.muon_ns_grouped, lib.gram_ns_grouped):
        fn.argtypes = [ctypes.c_int, P(MnsTensor), P(MnsTensor), P(MnsNsParams), vp, sz, vp, vp]
    lib.muon_step_grouped.argtypes = [ctypes.c_int, P(MnsTensor), P(MnsTensor), P(MnsTensor),
                                      P(MnsTensor), P(MnsStepParams), P(MnsNsParams), vp, sz,
                                      vp, vp]
    pp = P(vp)
    lib.adamw_step.argtypes = [ctypes.c_int, pp, pp, pp, pp, P(ctypes.c_int64), ctypes.c_int32,
                               P(MnsAdamwParams), vp]
    lib.adamw_step.restype = ctypes.c_int
    t, i32, i64 = P(MnsTensor), ctypes.c_int32, ctypes.c_int64
    layer = {
        "layer_norm": [t, vp, vp, i32, ctypes.c_float, t, vp, vp, vp],
        "mns_layer_norm_workspace_bytes": [t, P(sz)],
        "layer_norm_backward": [t, t, vp, vp, vp, i32, t, vp, vp, vp, sz, vp],
        "mns_expert_sort_workspace_bytes": [i64, i32, P(sz)],
        "expert_sort": [vp, i32, i64, i32, vp, vp, vp, sz, vp],
        "expert_dispatch": [t, vp, i32, vp, i32, t, vp],
        "expert_dispatch_backward": [t, vp, i32, t, vp],
        "expert_combine": [t, vp, i32, vp, i32, t, vp],
        "expert_combine_backward": [t, t, vp, i32, vp, i32, vp, i32, t, vp, vp],
        "expert_matmul": [t, t, vp, t, vp],
        "expert_matmul_grad_input": [t, t, vp, t, vp],
        "expert_matmul_grad_weight": [t, t, vp, t, vp],
        "rms_norm": [t, t, vp, i32, ctypes.c_float, t, t, vp, vp],
        "rms_norm_mx8": [t, t, vp, i32, ctypes.c_float, vp, vp, t, vp, vp],
        "mns_rms_norm_workspace_bytes": [t, P(sz)],
        "rms_norm_backward": [t, t, vp, vp, i32, t, t, vp, vp, sz, vp],
        "embed": [vp, i32, t, ctypes.c_float, t, vp],
        "mns_embed_workspace_bytes": [i64, i64, i64, P(sz)],
        "embed_backward": [t, vp, i32, ctypes.c_float, t, vp, sz, vp],
        "expert_gated": [t, t, t, vp, i32, t, t, t, vp, sz, vp],
        "mns_expert_gated_workspace_bytes": [i64, i64, i32, i32, P(sz), P(sz)],
        "mns_expert_gated_dense_workspace_bytes": [i64, i64, i64, i32, P(sz), P(sz)],
        "expert_gated_backward": [t, t, t, t, t, t, vp, i32, t, t, t, vp, sz, vp],
        "adamw8_step": [ctypes.c_int, pp, pp, pp, pp, pp, pp, P(i64), i32, P(MnsAdamw8Params), vp],
    }
    for name, argtypes in layer.items():
        fn = getattr(lib, name)
        fn.argtypes = argtypes
        fn.restype = ctypes.c_int
    lib.mns_status_string.argtypes = [ctypes.c_int]
    lib.mns_status_string.restype = ctypes.c_char_p
    lib.mns_last_hip_error.argtypes = []
    lib.mns_version.argtypes = []
    lib.mns_timing_enable.argtypes = [ctypes.c_int]
    lib.mns_timing_reset.argtypes = []
    lib.mns_timing_query.argtypes = [ctypes.c_int, P(ctypes.c_double), P(ctypes.c_int64)]
    lib.mns_timing_kinds.argtypes = []
    lib.mns_kernel_kind_name.argtypes = [ctypes.c_int]
    lib.mns_kernel_kind_name.restype = ctypes.c_char_p
    for f in (lib.mns_workspace_bytes, lib.muon_ns_batched, lib.gram_ns_batched, lib.gram_ns_trace,
              lib.mns_workspace_bytes_grouped, lib.muon_ns_grouped, lib.gram_ns_grouped,
              lib.muon_step_grouped,
              lib.muon_step, lib.muon_step_noalloc, lib.mns_last_hip_error, lib.mns_version, lib.mns_timing_enable,
              lib.mns_timing_reset, lib.mns_timing_query, lib.mns_timing_kinds):
        f.restype = ctypes.c_int
    return lib


def lib():
    """The loaded ctypes library (raises ImportError if it has not been built)."""
    return _lib()


def _check(code: int, what: str):
    if code != 0:
        raise MnsError(code, what)


_TORCH = None


def _torch():
    global _TORCH
    if _TORCH is None:
        import torch
        _TORCH = torch
    return _TORCH


_DTYPE_CODES = {}


def dtype_code(t) -> int:
    if not _DTYPE_CODES:
        torch = _torch()
        _DTYPE_CODES.update({torch.float32: F32, torch.bfloat16: BF16, torch.float16: F16})
    code = _DTYPE_CODES.get(t.dtype)
    if code is None:
        raise TypeError(f"unsupported dtype {t.dtype}")
    return code


def describe(t) -> MnsTensor:
    """mns_tensor for a 2-D (one matrix) or 3-D (batch) tensor with unit column stride."""
    shape, strides = t.shape, t.stride()
    if len(shape) == 2:
        b, (r, c) = 1, shape
    elif len(shape) == 3:
        b, r, c = shape
    else:
        raise ValueError("expected a 2-D matrix or a 3-D batch")
    if strides[-1] != 1:
        raise ValueError("rows must be contiguous (stride(-1) == 1)")
    ld = strides[-2] if r > 1 else c
    return MnsTensor(t.data_ptr(), dtype_code(t), b, r, c, ld, strides[0] if b > 1 else r * ld)


# ------------------------------------------------------------------ argument checks
# The C ABI takes bare device pointers; these checks run before any library call so that a
# host tensor, a mismatched dtype or a short buffer raises here instead of reaching a kernel.
# Dtype, shape and size checks come first and device checks last.

def _batch(t) -> int:
    return t.shape[0] if t.dim() == 3 else 1


def _check_same_shape(what, ref, **named):
    for name, t in named.items():
        if t is not None and tuple(t.shape) != tuple(ref.shape):
            raise ValueError(f"{what}: {name} has shape {tuple(t.shape)}, expected {tuple(ref.shape)}")


def _check_flags(what, flags, total):
    if flags is None:
        return
    torch = _torch()
    if flags.dtype != torch.int32:
        raise TypeError(f"{what}: flags must be int32, got {flags.dtype}")
    if not flags.is_contiguous():
        raise ValueError(f"{what}: flags must be contiguous")
    if flags.numel() < total:
        raise ValueError(f"{what}: flags holds {flags.numel()} entries, the call needs {total}")


def _check_workspace(what, ws):
    if ws is not None and not ws.is_contiguous():
        raise ValueError(f"{what}: workspace must be contiguous")


def _check_device(what, ref, **named):
    """Every named tensor (None skipped) is a device tensor on ref's device."""
    if not ref.is_cuda:
        raise ValueError(f"{what}: tensors must be device tensors (got {ref.device})")
    device = ref.device
    for name, t in named.items():
        if t is not None and t.device != device:
            raise ValueError(f"{what}: {name} is on {t.device}, expected {ref.device}")


def _ws_bytes(ws) -> int:
    return ws.numel() * ws.element_size()


def ns_params(steps: int = DEFAULT_STEPS, coeffs: Optional[Sequence] = None,
              eps: float = DEFAULT_EPS, iter_dtype: Optional[int] = None, io_dtype: int = BF16,
              restart_mask: int = STABILIZED_RESTART_MASK):
    keep = None
    cptr = None
    if coeffs is not None:
        flat = []
        for row in coeffs:
            flat.extend(float(v) for v in row)
        if len(flat) != 3 * steps:
            raise ValueError("coeffs must hold one (a, b, c) triple per step")
        keep = (ctypes.c_float * len(flat))(*flat)
        cptr = ctypes.cast(keep, ctypes.POINTER(ctypes.c_float))
    if iter_dtype is None:
        iter_dtype = F32 if io_dtype == F32 else F16
    p = MnsNsParams(steps, cptr, eps, iter_dtype, restart_mask)
    p._keep = keep  # keep the coefficient array alive with the struct
    return p


def _stream_ptr(t):
    torch = _torch()
    return ctypes.c_void_p(torch.cuda.current_stream(t.device).cuda_stream)


def workspace_bytes(variant: int, G, params: MnsNsParams, max_batch_chunk: int = 0) -> int:
    out = ctypes.c_size_t(0)
    _check(_lib().mns_workspace_bytes(variant, ctypes.byref(describe(G)), ctypes.byref(params),
                                      max_batch_chunk, ctypes.byref(out)), "mns_workspace_bytes")
    return out.value


def _workspace(variant, G, params, workspace):
    torch = _torch()
    if workspace is None:
        workspace = torch.empty(workspace_bytes(variant, G, params), dtype=torch.uint8,
                                device=G.device)
    return workspace


def _ns(variant, G, out, params, workspace, flags):
    torch = _torch()
    what = "muon_ns_batched" if variant == STANDARD else "gram_ns_batched"
    if out is not None:
        _check_same_shape(what, G, out=out)
        if out.dtype != G.dtype:
            raise TypeError(f"{what}: out must have G's dtype {G.dtype}, got {out.dtype}")
    _check_flags(what, flags, _batch(G))
    _check_workspace(what, workspace)
    _check_device(what, G, out=out, flags=flags, workspace=workspace)
    out = torch.empty_like(G) if out is None else out
    ws = _workspace(variant, G, params, workspace)
    fn = _lib().muon_ns_batched if variant == STANDARD else _lib().gram_ns_batched
    fptr = ctypes.c_void_p(flags.data_ptr()) if flags is not None else None
    _check(fn(ctypes.byref(describe(G)), ctypes.byref(describe(out)), ctypes.byref(params),
              ctypes.c_void_p(ws.data_ptr()), _ws_bytes(ws), fptr, _stream_ptr(G)), what)
    return out


def muon_ns(G, *, steps: int = DEFAULT_STEPS, coeffs=None, eps: float = DEFAULT_EPS,
            iter_dtype: Optional[int] = None, out=None, workspace=None, flags=None):
    """Standard Newton-Schulz of a matrix or batch (C ABI ``muon_ns_batched``)."""
    p = ns_params(steps, coeffs, eps, iter_dtype, dtype_code(G), 0)
    return _ns(STANDARD, G, out, p, workspace, flags)


def gram_ns(G, *, steps: int = DEFAULT_STEPS, coeffs=None, eps: float = DEFAULT_EPS,
            iter_dtype: Optional[int] = None, restart_mask: int = STABILIZED_RESTART_MASK,
            out=None, workspace=None, flags=None):
    """Gram Newton-Schulz (C ABI ``gram_ns_batched``); restart_mask=0 is the naive variant."""
    p = ns_params(steps, coeffs, eps, iter_dtype, dtype_code(G), restart_mask)
    return _ns(GRAM, G, out, p, workspace, flags)


def muon_step(W, G, M, *, lr: float, momentum: float, weight_decay: float,
              scale_coeff: float = 0.2, nesterov: bool = False, variant: int = GRAM,
              steps: int = DEFAULT_STEPS, coeffs=None, eps: float = DEFAULT_EPS,
              iter_dtype: Optional[int] = None, restart_mask: int = STABILIZED_RESTART_MASK,
              U_out=None, workspace=None, flags=None):
    """One fused Muon step (C ABI ``muon_step``); W and M are updated in place."""
    torch = _torch()
    what = "muon_step"
    _check_same_shape(what, G, W=W, M=M, U_out=U_out)
    if M.dtype != torch.float32:
        raise TypeError(f"{what}: the momentum buffer M must be float32, got {M.dtype}")
    _check_flags(what, flags, _batch(G))
    _check_workspace(what, workspace)
    _check_device(what, G, W=W, M=M, U_out=U_out, flags=flags, workspace=workspace)
    p = ns_params(steps, coeffs, eps, iter_dtype, dtype_code(G),
                  restart_mask if variant == GRAM else 0)
    sp = MnsStepParams(lr, momentum, weight_decay, scale_coeff, 1 if nesterov else 0, variant)
    ws = _workspace(variant, G, p, workspace)
    fptr = ctypes.c_void_p(flags.data_ptr()) if flags is not None else None
    u = ctypes.byref(describe(U_out)) if U_out is not None else None
    _check(_lib().muon_step(ctypes.byref(describe(W)), ctypes.byref(describe(G)),
                            ctypes.byref(describe(M)), u, ctypes.byref(sp), ctypes.byref(p),
                            ctypes.c_void_p(ws.data_ptr()), _ws_bytes(ws), fptr, _stream_ptr(G)),
           what)
    return W


# Size of the static device scratch behind muon_step_noalloc (MNS_NOALLOC_SCRATCH_BYTES).
NOALLOC_SCRATCH_BYTES = 256 << 20


def muon_step_noalloc(W, G, M, *, lr: float, momentum: float, weight_decay: float,
                      scale_coeff: float = 0.2, nesterov: bool = False, variant: int = GRAM,
                      steps: int = DEFAULT_STEPS, coeffs=None, eps: float = DEFAULT_EPS,
                      iter_dtype: Optional[int] = None, restart_mask: int = STABILIZED_RESTART_MASK,
                      U_out=None, flags=None):
    """One fused Muon step without a workspace (C ABI ``muon_step_noalloc``: the library's
    static device scratch); W and M are updated in place."""
    torch = _torch()
    what = "muon_step_noalloc"
    _check_same_shape(what, G, W=W, M=M, U_out=U_out)
    if M.dtype != torch.float32:
        raise TypeError(f"{what}: the momentum buffer M must be float32, got {M.dtype}")
    _check_flags(what, flags, _batch(G))
    _check_device(what, G, W=W, M=M, U_out=U_out, flags=flags)
    p = ns_params(steps, coeffs, eps, iter_dtype, dtype_code(G),
                  restart_mask if variant == GRAM else 0)
    sp = MnsStepParams(lr, momentum, weight_decay, scale_coeff, 1 if nesterov else 0, variant)
    fptr = ctypes.c_void_p(flags.data_ptr()) if flags is not None else None
    u = ctypes.byref(describe(U_out)) if U_out is not None else None
    _check(_lib().muon_step_noalloc(ctypes.byref(describe(W)), ctypes.byref(describe(G)),
                                    ctypes.byref(describe(M)), u, ctypes.byref(sp), ctypes.byref(p),
                                    fptr, _stream_ptr(G)), what)
    return W


# ------------------------------------------------------------------ grouped calls
MAX_GROUPS = 4


def _tensor_array(ts):
    arr = (MnsTensor * len(ts))()
    for i, t in enumerate(ts):
        arr[i] = t if isinstance(t, MnsTensor) else describe(t)
    return arr


def workspace_bytes_grouped(variant: int, Gs, params: MnsNsParams) -> int:
    """Workspace that lets a grouped call process every group side by side."""
    n = ctypes.c_size_t()
    _check(_lib().mns_workspace_bytes_grouped(variant, len(Gs), _tensor_array(Gs), ctypes.byref(params),
                                              ctypes.byref(n)), "mns_workspace_bytes_grouped")
    return n.value


def _check_groups(what, Gs, flags, workspace, **lists):
    """Group lists of equal length (1 .. MAX_GROUPS), flags covering every matrix of every
    group, everything on the first G's device."""
    n = len(Gs)
    if not 1 <= n <= MAX_GROUPS:
        raise ValueError(f"{what}: between 1 and {MAX_GROUPS} groups, got {n}")
    for name, ts in lists.items():
        if ts is not None and len(ts) != n:
            raise ValueError(f"{what}: {name} has {len(ts)} entries for {n} groups")
    _check_flags(what, flags, sum(_batch(G) for G in Gs))
    _check_workspace(what, workspace)
    named = {"flags": flags, "workspace": workspace}
    for i, G in enumerate(Gs):
        named[f"G[{i}]"] = G
        for name, ts in lists.items():
            if ts is not None:
                named[f"{name}[{i}]"] = ts[i]
    _check_device(what, Gs[0], **named)


def _ns_grouped(variant, Gs, outs, params, workspace, flags):
    torch = _torch()
    what = "muon_ns_grouped" if variant == STANDARD else "gram_ns_grouped"
    if outs is not None:
        if len(outs) != len(Gs):
            raise ValueError(f"{what}: outs has {len(outs)} entries for {len(Gs)} groups")
        for i, (G, O) in enumerate(zip(Gs, outs)):
            _check_same_shape(what, G, **{f"outs[{i}]": O})
            if O.dtype != G.dtype:
                raise TypeError(f"{what}: outs[{i}] must have dtype {G.dtype}, got {O.dtype}")
    _check_groups(what, Gs, flags, workspace, outs=outs)
    outs = [torch.empty_like(G) for G in Gs] if outs is None else list(outs)
    if workspace is None:
        workspace = torch.empty(workspace_bytes_grouped(variant, Gs, params), dtype=torch.uint8,
                                device=Gs[0].device)
    fn = _lib().muon_ns_grouped if variant == STANDARD else _lib().gram_ns_grouped
    fptr = ctypes.c_void_p(flags.data_ptr()) if flags is not None else None
    _check(fn(len(Gs), _tensor_array(Gs), _tensor_array(outs), ctypes.byref(params),
              ctypes.c_void_p(workspace.data_ptr()), _ws_bytes(workspace), fptr, _stream_ptr(Gs[0])),
           what)
    return outs


def muon_ns_grouped(Gs, *, steps: int = DEFAULT_STEPS, coeffs=None, eps: float = DEFAULT_EPS,
                    iter_dtype: Optional[int] = None, outs=None, workspace=None, flags=None):
    """Standard Newton-Schulz of several batches of different shapes (C ABI ``muon_ns_grouped``)."""
    p = ns_params(steps, coeffs, eps, iter_dtype, dtype_code(Gs[0]), 0)
    return _ns_grouped(STANDARD, Gs, outs, p, workspace, flags)


def gram_ns_grouped(Gs, *, steps: int = DEFAULT_STEPS, coeffs=None, eps: float = DEFAULT_EPS,
                    iter_dtype: Optional[int] = None, restart_mask: int = STABILIZED_RESTART_MASK,
                    outs=None, workspace=None, flags=None):
    """Gram Newton-Schulz of several batches of different shapes (C ABI ``gram_ns_grouped``)."""
    p = ns_params(steps, coeffs, eps, iter_dtype, dtype_code(Gs[0]), restart_mask)
    return _ns_grouped(GRAM, Gs, outs, p, workspace, flags)


def muon_step_grouped(Ws, Gs, Ms, *, lr: float, momentum: float, weight_decay: float,
                      scale_coeff: float = 0.2, nesterov: bool = False, variant: int = GRAM,
                      steps: int = DEFAULT_STEPS, coeffs=None, eps: float = DEFAULT_EPS,
                      iter_dtype: Optional[int] = None, restart_mask: int = STABILIZED_RESTART_MASK,
                      U_outs=None, workspace=None, flags=None):
    """One fused Muon step over several batches of different shapes (C ABI
    ``muon_step_grouped``); every W and M is updated in place."""
    torch = _torch()
    what = "muon_step_grouped"
    for name, ts in (("Ws", Ws), ("Ms", Ms), ("U_outs", U_outs)):
        if ts is not None and len(ts) != len(Gs):
            raise ValueError(f"{what}: {name} has {len(ts)} entries for {len(Gs)} groups")
    for i, G in enumerate(Gs):
        _check_same_shape(what, G, **{f"Ws[{i}]": Ws[i], f"Ms[{i}]": Ms[i],
                                      f"U_outs[{i}]": U_outs[i] if U_outs is not None else None})
        if Ms[i].dtype != torch.float32:
            raise TypeError(f"{what}: Ms[{i}] must be float32, got {Ms[i].dtype}")
    _check_groups(what, Gs, flags, workspace, Ws=Ws, Ms=Ms, U_outs=U_outs)
    p = ns_params(steps, coeffs, eps, iter_dtype, dtype_code(Gs[0]),
                  restart_mask if variant == GRAM else 0)
    sp = MnsStepParams(lr, momentum, weight_decay, scale_coeff, 1 if nesterov else 0, variant)
    if workspace is None:
        workspace = torch.empty(workspace_bytes_grouped(variant, Gs, p), dtype=torch.uint8,
                                device=Gs[0].device)
    fptr = ctypes.c_void_p(flags.data_ptr()) if flags is not None else None
    u = _tensor_array(U_outs) if U_outs is not None else None
    _check(_lib().muon_step_grouped(len(Gs), _tensor_array(Ws), _tensor_array(Gs), _tensor_array(Ms),
                                    u, ctypes.byref(sp), ctypes.byref(p),
                                    ctypes.c_void_p(workspace.data_ptr()), _ws_bytes(workspace), fptr,
                                    _stream_ptr(Gs[0])), what)
    return Ws


# ------------------------------------------------------------------ AdamW (hybrid optimizer)
class MnsAdamwParams(ctypes.Structure):
    _fields_ = [("lr", ctypes.c_float), ("beta1", ctypes.c_float), ("beta2", ctypes.c_float),
                ("eps", ctypes.c_float), ("weight_decay", ctypes.c_float), ("step", ctypes.c_int32),
                ("bias_correction", ctypes.c_int32)]


def adamw_step(params, grads, exp_avgs, exp_avg_sqs, *, lr: float, beta1: float = 0.9,
               beta2: float = 0.95, eps: float = 1e-8, weight_decay: float = 0.1, step: int = 1,
               bias_correction: bool = False):
    """One AdamW step over lists of contiguous tensors (C ABI ``adamw_step``); params and both
    fp32 moments are updated in place."""
    torch = _torch()
    n = len(params)
    if not (len(grads) == len(exp_avgs) == len(exp_avg_sqs) == n) or n == 0:
        raise ValueError("params, grads and moments must be non-empty lists of equal length")
    pdt = params[0].dtype
    for i, (p_, g_, m_, v_) in enumerate(zip(params, grads, exp_avgs, exp_avg_sqs)):
        if p_.dtype != pdt:
            raise TypeError(f"adamw_step: params[{i}] is {p_.dtype}; every parameter must be {pdt}")
        if g_.dtype != pdt:
            raise TypeError(f"adamw_step: grads[{i}] is {g_.dtype}, its parameter is {pdt}")
        if m_.dtype != torch.float32 or v_.dtype != torch.float32:
            raise TypeError(f"adamw_step: the moments of tensor {i} must be float32")
        if not (p_.numel() == g_.numel() == m_.numel() == v_.numel()):
            raise ValueError("each parameter, gradient and moment pair must have equal sizes")
    for group in (params, grads, exp_avgs, exp_avg_sqs):
        for t in group:
            if not t.is_contiguous():
                raise ValueError("AdamW tensors must be contiguous")
    named = {}
    for i in range(n):
        named.update({f"params[{i}]": params[i], f"grads[{i}]": grads[i],
                      f"exp_avgs[{i}]": exp_avgs[i], f"exp_avg_sqs[{i}]": exp_avg_sqs[i]})
    _check_device("adamw_step", params[0], **named)
    arr = lambda ts: (ctypes.c_void_p * n)(*[t.data_ptr() for t in ts])
    numels = (ctypes.c_int64 * n)(*[t.numel() for t in params])
    ap = MnsAdamwParams(lr, beta1, beta2, eps, weight_decay, step, 1 if bias_correction else 0)
    _check(_lib().adamw_step(n, arr(params), arr(grads), arr(exp_avgs), arr(exp_avg_sqs), numels,
                             dtype_code(params[0]), ctypes.byref(ap), _stream_ptr(params[0])),
           "adamw_step")
    return params


class MnsAdamw8Params(ctypes.Structure):
    _fields_ = [("lr", ctypes.c_double), ("beta1", ctypes.c_double), ("beta2", ctypes.c_double),
                ("eps", ctypes.c_double), ("weight_decay", ctypes.c_double), ("step", ctypes.c_int32),
                ("bias_correction", ctypes.c_int32), ("seed", ctypes.c_uint64), ("device_step", ctypes.c_void_p)]


MX_BLOCK = 32   # elements that share a power of two in 8-bit values


class Adamw8State(NamedTuple):
    """Moments of one parameter in 8 bits: m and r = sqrt(v) as float8_e4m3fn codes (flat, one per element)
    with float8_e8m0fnu powers of two (one per 32 elements); a value is code * power."""
    exp_avg: object
    exp_avg_scale: object
    root: object
    root_scale: object


def adamw8_state(param) -> Adamw8State:
    """The state of a parameter before its first step (all zero)."""
    torch = _torch()
    n = param.numel()
    zeros = lambda count, dtype: torch.zeros(count, dtype=torch.uint8, device=param.device).view(dtype)
    blocks = (n + MX_BLOCK - 1) // MX_BLOCK
    return Adamw8State(zeros(n, torch.float8_e4m3fn), zeros(blocks, torch.float8_e8m0fnu),
                       zeros(n, torch.float8_e4m3fn), zeros(blocks, torch.float8_e8m0fnu))


def adamw8_step(params, grads, states, *, lr: float, step, beta1: float = 0.9, beta2: float = 0.95, eps: float = 1e-8,
                weight_decay: float = 0.1, bias_correction: bool = False, seed: int = 0):
    """One AdamW step over lists of contiguous tensors with their moments in 8 bits (C ABI ``adamw8_step``);
    params and states (adamw8_state's, or tuples like it) are updated in place. The states are rounded at
    random: the numbers depend on seed, step (count it up), a tensor's place in the list and the element's.
    step: an int, or a device tensor of one int64 that is read when the kernels run. A call captured into a graph
    needs the tensor, advanced in the graph or before each replay (``step.add_(1)``): replays of a captured int round
    with the same numbers every time, and moments whose change is below a code's step stand still."""
    torch = _torch()
    what = "adamw8_step"
    n = len(params)
    if not (len(grads) == len(states) == n) or n == 0:
        raise ValueError(f"{what}: params, grads and states must be non-empty lists of equal length")
    device_step = step if isinstance(step, torch.Tensor) else None
    if device_step is not None:
        _check_flat(what, params[0], (torch.int64,), step=device_step)
        if device_step.numel() != 1:
            raise ValueError(f"{what}: a step on the device must be one number, got {device_step.numel()}")
    elif not 1 <= step < 2 ** 31:
        raise ValueError(f"{what}: step must count from 1, got {step}")
    if not 0 <= seed < 2 ** 64:
        raise ValueError(f"{what}: seed must fit 64 bits, got {seed}")
    code = dtype_code(params[0])
    if set(map(len, states)) != {4}:
        i = next(i for i, s in enumerate(states) if len(s) != 4)
        raise ValueError(f"{what}: states[{i}] must hold four tensors, got {len(states[i])}")
    # column by column: a list of some hundred tensors costs more in these checks than in its kernels
    Tensor = torch.Tensor
    numels = list(map(Tensor.numel, params))
    blocks = [(count + MX_BLOCK - 1) // MX_BLOCK for count in numels]
    codes, scales = (torch.float8_e4m3fn, torch.uint8), (torch.float8_e8m0fnu, torch.uint8)
    columns = (list(params), list(grads), *map(list, zip(*states)))
    names = ("params", "grads", *Adamw8State._fields)
    own = (params[0].dtype,)
    for name, column, allowed, sizes in zip(names, columns, (own, own, codes, scales, codes, scales), (numels, numels, numels, blocks, numels, blocks)):
        if not {t.dtype for t in column}.issubset(allowed):
            i = next(i for i, t in enumerate(column) if t.dtype not in allowed)
            raise TypeError(f"{what}: {name}[{i}] is {column[i].dtype}, expected {allowed[0]}")
        if list(map(Tensor.numel, column)) != sizes:
            i = next(i for i, t in enumerate(column) if t.numel() != sizes[i])
            raise ValueError(f"{what}: {name}[{i}] has {column[i].numel()} elements, expected {sizes[i]}")
        if not all(map(Tensor.is_contiguous, column)):
            i = next(i for i, t in enumerate(column) if not t.is_contiguous())
            raise ValueError(f"{what}: {name}[{i}] must be contiguous")
    device = params[0].device
    if not params[0].is_cuda:
        raise ValueError(f"{what}: tensors must be device tensors (got {device})")
    index = params[0].get_device()
    for name, column in zip(names, columns):
        if set(map(Tensor.get_device, column)) != {index}:
            i = next(i for i, t in enumerate(column) if t.get_device() != index)
            raise ValueError(f"{what}: {name}[{i}] is on {column[i].device}, expected {device}")
    if device_step is not None and device_step.get_device() != index:
        raise ValueError(f"{what}: step is on {device_step.device}, expected {device}")
    if device_step is None and torch.cuda.is_current_stream_capturing():
        warnings.warn(f"{what}: captured with a step from the host, whose random numbers every replay uses again; give step as a "
                      "device tensor", stacklevel=2)
    pointers = ctypes.c_void_p * n
    lists = [pointers.from_buffer(array.array("Q", map(Tensor.data_ptr, column))) for column in columns]
    sizes = (ctypes.c_int64 * n).from_buffer(array.array("q", numels))
    ap = MnsAdamw8Params(lr, beta1, beta2, eps, weight_decay, 1 if device_step is not None else step, 1 if bias_correction else 0, seed,
                         _ptr(device_step))
    _launch(what, params[0], n, *lists, sizes, code, ctypes.byref(ap))
    return params


def hybrid_step(matrix_groups, vector_params, *, muon: dict, adamw: dict, seed: int = 0):
    """The hybrid optimizer step: Muon for the 2-D matrices (``matrix_groups``: list of
    (W, G, M) batches, one grouped call) and AdamW for everything else (``vector_params``:
    list of (param, grad, exp_avg, exp_avg_sq), or (param, grad, adamw8_state(param)) where the
    moments are held in 8 bits; those need ``step`` in ``adamw`` and take ``seed``), enqueued on the
    current stream. A step on the device (adamw8_step) goes with moments in 32 bits only without their
    bias correction, which adamw_step works out on the host."""
    entries = [tuple(v) for v in vector_params or ()]   # may be iterators, which are gone through once
    for i, v in enumerate(entries):
        if len(v) not in (3, 4):
            raise ValueError(f"hybrid_step: entry {i} of vector_params holds {len(v)} things, expected 3 or 4")
    in32 = [v for v in entries if len(v) == 4]
    in8 = [v for v in entries if len(v) == 3]
    if in8 and "step" not in adamw:
        raise TypeError("hybrid_step: moments in 8 bits need step in adamw")
    adamw32 = adamw
    if entries and isinstance(adamw.get("step"), _torch().Tensor):
        if adamw.get("bias_correction") and in32:
            raise ValueError("hybrid_step: adamw_step corrects its bias by a step on the host, got one on the device")
        adamw32 = {k: v for k, v in adamw.items() if k != "step"}
    if matrix_groups:
        Ws, Gs, Ms = (list(x) for x in zip(*matrix_groups))
        muon_step_grouped(Ws, Gs, Ms, **muon)
    if in32:
        ps, gs, ms, vs = (list(x) for x in zip(*in32))
        adamw_step(ps, gs, ms, vs, **adamw32)
    if in8:
        ps, gs, ss = (list(x) for x in zip(*in8))
        adamw8_step(ps, gs, ss, seed=seed, **adamw)


# ------------------------------------------------------------------ the layer around the experts
# Layer norm and a mixture of experts, forward and backward, next to the optimizer that takes
# their gradients: expert_matmul_backward's dW is muon_step's G, the norm's are adamw_step's.
# Gradients are explicit calls; a call that autograd would have to record, or whose forward-mode
# tangent would be lost, is refused.

MAX_EXPERTS = 1024


def _check_recorded(what, *ts):
    torch = _torch()
    for t in ts:
        if t is not None and t.requires_grad and torch.is_grad_enabled():
            raise RuntimeError(f"{what}: not recorded by autograd; call it under torch.no_grad() (or in an "
                               "autograd.Function) and its gradient explicitly")
    # a dual tensor does not require grad; duals exist inside a dual level only (0.3 us a tensor to ask)
    fwad = torch.autograd.forward_ad
    if getattr(fwad, "_current_level", 0) >= 0:
        for t in ts:
            if t is not None and fwad.unpack_dual(t).tangent is not None:
                raise RuntimeError(f"{what}: no forward-mode derivative; pass the primal (forward_ad.unpack_dual) and take "
                                   "the tangent through the explicit formulas")


def _check_rows(what, ref, **named):
    """Row buffers: 2-D tensors of ref's dtype."""
    for name, t in named.items():
        if t is None:
            continue
        if t.dim() != 2:
            raise ValueError(f"{what}: {name} must be 2-D, got {t.dim()}-D")
        if t.dtype != ref.dtype:
            raise TypeError(f"{what}: {name} is {t.dtype}, expected {ref.dtype}")


def _check_shape(what, name, t, shape):
    if t.shape != shape:   # a torch.Size compares with a tuple
        raise ValueError(f"{what}: {name} has shape {tuple(t.shape)}, expected {tuple(shape)}")


def _check_flat(what, ref, dtypes, **named):
    """Contiguous buffers of one of the dtypes."""
    for name, t in named.items():
        if t is None:
            continue
        if t.dtype not in dtypes:
            raise TypeError(f"{what}: {name} is {t.dtype}, expected " + " or ".join(str(d) for d in dtypes))
        if not t.is_contiguous():
            raise ValueError(f"{what}: {name} must be contiguous")


def _check_rank(what, rank, offsets=None):
    torch = _torch()
    if rank.dim() != 2:
        raise ValueError(f"{what}: rank must be [tokens, k], got {rank.dim()}-D")
    _check_flat(what, rank, (torch.int32,), rank=rank, offsets=offsets)
    if offsets is not None:
        _check_offsets(what, offsets)


def _check_offsets(what, offsets):
    torch = _torch()
    _check_flat(what, offsets, (torch.int32,), offsets=offsets)
    if offsets.dim() != 1 or not 2 <= offsets.numel() <= MAX_EXPERTS + 1:
        raise ValueError(f"{what}: offsets must be [experts + 1] with 1 to {MAX_EXPERTS} experts, got {tuple(offsets.shape)}")


def _ptr(t):
    return None if t is None else t.data_ptr()


def _raw_stream(index):
    """The current stream's handle (torch.cuda.current_stream builds an object for it, 1.5 us)."""
    torch = _torch()
    get = getattr(torch._C, "_cuda_getCurrentRawStream", None)
    return get(index) if get else torch.cuda.current_stream(index).cuda_stream


def _launch(what, ref, *args):
    """Call the C function `what` on ref's device and its current stream there."""
    index = ref.device.index
    fn = getattr(_lib(), what)
    if index == _torch().cuda.current_device():
        code = fn(*args, _raw_stream(index))
    else:
        with _torch().cuda.device(index):
            code = fn(*args, _raw_stream(index))
    if code:
        raise MnsError(code, what)


def layer_norm(x, weight=None, bias=None, *, eps: float = 1e-5, out=None):
    """(y, mean, rstd): layer norm over the columns of x ([rows, cols] or [batch, rows, cols]; C ABI
    ``layer_norm``). weight and bias: [cols] of x's dtype or float32. mean and rstd: float32, one per
    row, for the backward pass."""
    torch = _torch()
    what = "layer_norm"
    _check_recorded(what, x, weight, bias, out)
    xd = describe(x)
    _check_flat(what, x, (x.dtype, torch.float32), weight=weight, bias=bias)
    lead, cols = x.shape[:-1], x.shape[-1:]
    wcode = F32
    for name, t in (("weight", weight), ("bias", bias)):
        if t is not None:
            if t.shape != cols:
                _check_shape(what, name, t, cols)
            wcode = dtype_code(t)
    if weight is not None and bias is not None and weight.dtype != bias.dtype:
        raise TypeError(f"{what}: weight is {weight.dtype}, bias is {bias.dtype}")
    if out is not None:
        _check_same_shape(what, x, out=out)
        if out.dtype != x.dtype:
            raise TypeError(f"{what}: out must have x's dtype {x.dtype}, got {out.dtype}")
    _check_device(what, x, weight=weight, bias=bias, out=out)
    y = x.new_empty(x.shape) if out is None else out
    mean = torch.empty(lead, dtype=torch.float32, device=x.device)
    rstd = torch.empty(lead, dtype=torch.float32, device=x.device)
    _launch(what, x, xd, _ptr(weight), _ptr(bias), wcode, eps, describe(y),
            _ptr(mean), _ptr(rstd))
    return y, mean, rstd


def layer_norm_workspace_bytes(x) -> int:
    n = ctypes.c_size_t()
    _check(_lib().mns_layer_norm_workspace_bytes(ctypes.byref(describe(x)), ctypes.byref(n)), "mns_layer_norm_workspace_bytes")
    return n.value


def layer_norm_backward(dy, x, mean, rstd, weight=None, *, param_grads: bool = True, out=None, workspace=None):
    """(dx, dweight, dbias) of layer_norm (C ABI ``layer_norm_backward``). dweight and dbias have
    weight's dtype; they are None without weight or with param_grads=False."""
    torch = _torch()
    what = "layer_norm_backward"
    _check_recorded(what, dy, x, mean, rstd, weight, out)
    _check_same_shape(what, x, dy=dy, out=out)
    for name, t in (("dy", dy), ("out", out)):
        if t is not None and t.dtype != x.dtype:
            raise TypeError(f"{what}: {name} is {t.dtype}, expected {x.dtype}")
    _check_flat(what, x, (torch.float32,), mean=mean, rstd=rstd)
    _check_flat(what, x, (x.dtype, torch.float32), weight=weight)
    for name, t, shape in (("mean", mean, x.shape[:-1]), ("rstd", rstd, x.shape[:-1]), ("weight", weight, x.shape[-1:])):
        if t is not None:
            _check_shape(what, name, t, shape)
    _check_workspace(what, workspace)
    _check_device(what, x, dy=dy, mean=mean, rstd=rstd, weight=weight, out=out, workspace=workspace)
    dx = x.new_empty(x.shape) if out is None else out
    dw = db = None
    if weight is not None and param_grads:
        dw, db = torch.empty_like(weight), torch.empty_like(weight)
        if workspace is None:
            workspace = torch.empty(layer_norm_workspace_bytes(x), dtype=torch.uint8, device=x.device)
    _launch(what, x, describe(dy), describe(x), _ptr(mean), _ptr(rstd), _ptr(weight),
            dtype_code(weight) if weight is not None else F32, describe(dx), _ptr(dw), _ptr(db), _ptr(workspace),
            0 if workspace is None else _ws_bytes(workspace))
    return dx, dw, db


def expert_sort_workspace_bytes(slots: int, num_experts: int) -> int:
    n = ctypes.c_size_t()
    _check(_lib().mns_expert_sort_workspace_bytes(slots, num_experts, ctypes.byref(n)), "mns_expert_sort_workspace_bytes")
    return n.value


def expert_sort(experts, num_experts: int, *, workspace=None):
    """(offsets, rank) of the picks experts ([tokens, k] int32 or int64; C ABI ``expert_sort``): expert
    e's sorted rows are offsets[e] .. offsets[e + 1] - 1 (int32 [num_experts + 1]), rank[t, j] is the
    row of token t's j-th pick (int32 [tokens, k]), -1 for a pick outside 0 .. num_experts - 1."""
    torch = _torch()
    what = "expert_sort"
    if experts.dim() != 2 or experts.shape[1] < 1:
        raise ValueError(f"{what}: experts must be [tokens, k], got {tuple(experts.shape)}")
    if not 1 <= num_experts <= MAX_EXPERTS:
        raise ValueError(f"{what}: num_experts must be 1 to {MAX_EXPERTS}, got {num_experts}")
    _check_flat(what, experts, (torch.int32, torch.int64), experts=experts)
    _check_workspace(what, workspace)
    _check_device(what, experts, workspace=workspace)
    slots = experts.numel()
    offsets = experts.new_empty(num_experts + 1, dtype=torch.int32)
    rank = experts.new_empty(experts.shape, dtype=torch.int32)
    if workspace is None:
        n = expert_sort_workspace_bytes(slots, num_experts)
        workspace = torch.empty(n, dtype=torch.uint8, device=experts.device) if n else None
    _launch(what, experts, _ptr(experts), experts.element_size(), slots, num_experts, offsets.data_ptr(), _ptr(rank),
            _ptr(workspace), 0 if workspace is None else _ws_bytes(workspace))
    return offsets, rank


def expert_dispatch(x, rank, offsets, *, out=None):
    """The tokens' rows sorted by expert: out[rank[t, j]] = x[t], the rows of no expert zero
    ([tokens * k, dim]; C ABI ``expert_dispatch``)."""
    torch = _torch()
    what = "expert_dispatch"
    _check_recorded(what, x, out)
    _check_rank(what, rank, offsets)
    _check_rows(what, x, x=x, out=out)
    _check_shape(what, "rank", rank, (x.shape[0], rank.shape[1]))
    if out is not None:
        _check_shape(what, "out", out, (rank.numel(), x.shape[1]))
    _check_device(what, x, rank=rank, offsets=offsets, out=out)
    xs = x.new_empty((rank.numel(), x.shape[1])) if out is None else out
    _launch(what, x, describe(x), _ptr(rank), rank.shape[1], offsets.data_ptr(), offsets.numel() - 1, describe(xs))
    return xs


def expert_dispatch_backward(dxs, rank, *, out=None):
    """dx[t] = sum_j dxs[rank[t, j]] (C ABI ``expert_dispatch_backward``)."""
    torch = _torch()
    what = "expert_dispatch_backward"
    _check_recorded(what, dxs, out)
    _check_rank(what, rank)
    _check_rows(what, dxs, dxs=dxs, out=out)
    _check_shape(what, "dxs", dxs, (rank.numel(), dxs.shape[1]))
    if out is not None:
        _check_shape(what, "out", out, (rank.shape[0], dxs.shape[1]))
    _check_device(what, dxs, rank=rank, out=out)
    dx = dxs.new_empty((rank.shape[0], dxs.shape[1])) if out is None else out
    _launch(what, dxs, describe(dxs), _ptr(rank), rank.shape[1], describe(dx))
    return dx


def expert_combine(ys, weights, rank, *, out=None):
    """y[t] = sum_j weights[t, j] ys[rank[t, j]] (C ABI ``expert_combine``). weights: [tokens, k] of ys's
    dtype or float32; a slot without a row adds nothing, whatever its weight."""
    torch = _torch()
    what = "expert_combine"
    _check_recorded(what, ys, weights, out)
    _check_rank(what, rank)
    _check_rows(what, ys, ys=ys, out=out)
    _check_flat(what, ys, (ys.dtype, torch.float32), weights=weights)
    _check_shape(what, "weights", weights, rank.shape)
    _check_shape(what, "ys", ys, (rank.numel(), ys.shape[1]))
    if out is not None:
        _check_shape(what, "out", out, (rank.shape[0], ys.shape[1]))
    _check_device(what, ys, weights=weights, rank=rank, out=out)
    y = ys.new_empty((rank.shape[0], ys.shape[1])) if out is None else out
    _launch(what, ys, describe(ys), _ptr(weights), dtype_code(weights), _ptr(rank), rank.shape[1], describe(y))
    return y


def expert_combine_backward(dy, ys, weights, rank, offsets, *, out=None):
    """(dys, dweights) of expert_combine (C ABI ``expert_combine_backward``); dweights has weights'
    dtype, 0 for a slot without a row."""
    torch = _torch()
    what = "expert_combine_backward"
    _check_recorded(what, dy, ys, weights, out)
    _check_rank(what, rank, offsets)
    _check_rows(what, ys, dy=dy, ys=ys, out=out)
    _check_flat(what, ys, (ys.dtype, torch.float32), weights=weights)
    _check_shape(what, "weights", weights, rank.shape)
    _check_shape(what, "ys", ys, (rank.numel(), ys.shape[1]))
    _check_shape(what, "dy", dy, (rank.shape[0], ys.shape[1]))
    if out is not None:
        _check_shape(what, "out", out, ys.shape)
    _check_device(what, ys, dy=dy, weights=weights, rank=rank, offsets=offsets, out=out)
    dys = ys.new_empty(ys.shape) if out is None else out
    dw = torch.empty_like(weights)
    _launch(what, ys, describe(dy), describe(ys), _ptr(weights), dtype_code(weights), _ptr(rank), rank.shape[1],
            offsets.data_ptr(), offsets.numel() - 1, describe(dys), _ptr(dw))
    return dys, dw


def _check_product(what, w, offsets, **rows):
    _check_recorded(what, w, *rows.values())
    _check_offsets(what, offsets)
    if w.dim() != 3:
        raise ValueError(f"{what}: w must be [experts, rows, cols], got {w.dim()}-D")
    if w.shape[0] != offsets.numel() - 1:
        raise ValueError(f"{what}: w holds {w.shape[0]} experts, offsets {offsets.numel() - 1}")
    _check_rows(what, w, **rows)


def expert_matmul(x, w, offsets, *, out=None):
    """y[s] = w[e] x[s] for the rows s of expert e, the rows of no expert zero (C ABI ``expert_matmul``).
    x: [rows, K] sorted by expert, w: [experts, N, K], offsets as expert_sort gives them."""
    torch = _torch()
    what = "expert_matmul"
    _check_product(what, w, offsets, x=x, out=out)
    _check_shape(what, "x", x, (x.shape[0], w.shape[2]))
    if out is not None:
        _check_shape(what, "out", out, (x.shape[0], w.shape[1]))
    _check_device(what, x, w=w, offsets=offsets, out=out)
    y = x.new_empty((x.shape[0], w.shape[1])) if out is None else out
    _launch(what, x, describe(x), describe(w), offsets.data_ptr(), describe(y))
    return y


def expert_matmul_grad_input(dy, w, offsets, *, out=None):
    """dx[s] = w[e]^T dy[s] for the rows s of expert e (C ABI ``expert_matmul_grad_input``)."""
    torch = _torch()
    what = "expert_matmul_grad_input"
    _check_product(what, w, offsets, dy=dy, out=out)
    _check_shape(what, "dy", dy, (dy.shape[0], w.shape[1]))
    if out is not None:
        _check_shape(what, "out", out, (dy.shape[0], w.shape[2]))
    _check_device(what, dy, w=w, offsets=offsets, out=out)
    dx = dy.new_empty((dy.shape[0], w.shape[2])) if out is None else out
    _launch(what, dy, describe(dy), describe(w), offsets.data_ptr(), describe(dx))
    return dx


def expert_matmul_grad_weight(dy, x, offsets, *, out=None):
    """dw[e] = sum over expert e's rows of dy[s] x[s]^T, zero for an expert without rows (C ABI
    ``expert_matmul_grad_weight``): [experts, N, K], the gradient batch that muon_step takes."""
    torch = _torch()
    what = "expert_matmul_grad_weight"
    _check_recorded(what, dy, x, out)
    _check_offsets(what, offsets)
    _check_rows(what, x, dy=dy, x=x)
    _check_shape(what, "dy", dy, (x.shape[0], dy.shape[1]))
    shape = (offsets.numel() - 1, dy.shape[1], x.shape[1])
    if out is not None:
        _check_shape(what, "out", out, shape)
        if out.dtype != x.dtype:
            raise TypeError(f"{what}: out is {out.dtype}, expected {x.dtype}")
    _check_device(what, x, dy=dy, offsets=offsets, out=out)
    dw = x.new_empty(shape) if out is None else out
    _launch(what, x, describe(dy), describe(x), offsets.data_ptr(), describe(dw))
    return dw


def expert_matmul_backward(dy, x, w, offsets):
    """(dx, dw) of expert_matmul: expert_matmul_grad_input and expert_matmul_grad_weight."""
    what = "expert_matmul_backward"
    _check_product(what, w, offsets, dy=dy, x=x)
    _check_shape(what, "x", x, (x.shape[0], w.shape[2]))
    _check_shape(what, "dy", dy, (x.shape[0], w.shape[1]))
    _check_device(what, dy, x=x, w=w, offsets=offsets)
    dyd, xd, at = describe(dy), describe(x), offsets.data_ptr()
    dx, dw = x.new_empty(x.shape), w.new_empty(w.shape)
    _launch("expert_matmul_grad_input", dy, dyd, describe(w), at, describe(dx))
    _launch("expert_matmul_grad_weight", dy, dyd, xd, at, describe(dw))
    return dx, dw


ACTIVATIONS = {"silu": 0, "gelu": 1, "relu": 2}


def _check_gated(what, x, w_gate, w_up, offsets, act, **inner):
    """Both matrices of every expert, or of a dense layer (2-D, no offsets); inner: buffers of [rows, N]."""
    _check_recorded(what, x, w_gate, w_up, *inner.values())
    if act not in ACTIVATIONS:
        raise ValueError(f"{what}: act must be one of {', '.join(ACTIVATIONS)}, got {act!r}")
    if w_gate.dim() not in (2, 3):
        raise ValueError(f"{what}: w_gate must be [experts, rows, cols] or [rows, cols], got {w_gate.dim()}-D")
    _check_like(what, w_gate, w_up=w_up)
    if offsets is not None:
        _check_offsets(what, offsets)
    if offsets is None and _batch(w_gate) != 1:
        raise ValueError(f"{what}: {_batch(w_gate)} experts need offsets")
    if offsets is not None and _batch(w_gate) != offsets.numel() - 1:
        raise ValueError(f"{what}: w_gate holds {_batch(w_gate)} experts, offsets {offsets.numel() - 1}")
    _check_rows(what, w_gate, x=x, **inner)
    _check_shape(what, "x", x, (x.shape[0], w_gate.shape[-1]))
    for name, t in inner.items():
        if t is not None:
            _check_shape(what, name, t, (x.shape[0], w_gate.shape[-2]))
    return ACTIVATIONS[act]


def expert_gated(x, w_gate, w_up, offsets=None, *, act: str = "silu", keep: bool = False, out=None, workspace=None):
    """act(x w_gate[e]^T) * (x w_up[e]^T) for the rows of expert e, the rows of no expert zero, in one kernel
    (C ABI ``expert_gated``). x: [rows, K] sorted by expert, w_gate and w_up: [experts, N, K] with offsets as
    expert_sort gives them, or [N, K] without offsets: a dense layer. act: silu, gelu (with erf) or relu.
    keep=True: (h, gate, up) with both projections, for expert_gated_backward."""
    torch = _torch()
    what = "expert_gated"
    code = _check_gated(what, x, w_gate, w_up, offsets, act, out=out)
    _check_workspace(what, workspace)
    _check_device(what, x, w_gate=w_gate, w_up=w_up, offsets=offsets, out=out, workspace=workspace)
    shape = (x.shape[0], w_gate.shape[-2])
    h = x.new_empty(shape) if out is None else out
    gate, up = (x.new_empty(shape), x.new_empty(shape)) if keep else (None, None)
    if workspace is None and offsets is None:
        n = expert_gated_workspace_bytes(*shape, x, dense=True, cols=x.shape[1])[0]
        workspace = torch.empty(n, dtype=torch.uint8, device=x.device) if n else None
    _launch(what, x, describe(x), describe(w_gate), describe(w_up), _ptr(offsets), code, describe(h), describe(gate) if keep else None,
            describe(up) if keep else None, _ptr(workspace), 0 if workspace is None else _ws_bytes(workspace))
    return (h, gate, up) if keep else h


def expert_gated_workspace_bytes(rows: int, inner: int, like, *, dense: bool = False, cols: Optional[int] = None) -> tuple:
    """(expert_gated's, expert_gated_backward's); like: a tensor of the rows' dtype; dense: without offsets, of which calls
    that cut no round need less: cols (K) tells them apart."""
    forward, backward = ctypes.c_size_t(), ctypes.c_size_t()
    if dense and cols is not None:
        _check(_lib().mns_expert_gated_dense_workspace_bytes(rows, inner, cols, dtype_code(like), ctypes.byref(forward), ctypes.byref(backward)),
               "mns_expert_gated_dense_workspace_bytes")
        return forward.value, backward.value
    _check(_lib().mns_expert_gated_workspace_bytes(rows, inner, 0 if dense else 1, dtype_code(like), ctypes.byref(forward), ctypes.byref(backward)),
           "mns_expert_gated_workspace_bytes")
    return forward.value, backward.value


def expert_gated_backward(dh, x, w_gate, w_up, gate, up, offsets=None, *, act: str = "silu", need_input: bool = True,
                          need_weights: bool = True, workspace=None):
    """(dx, dw_gate, dw_up) of expert_gated from gate and up as it kept them (C ABI ``expert_gated_backward``):
    the weights' gradients as the batches that muon_step takes. need_input, need_weights: what is not
    wanted is None."""
    torch = _torch()
    what = "expert_gated_backward"
    code = _check_gated(what, x, w_gate, w_up, offsets, act, dh=dh, gate=gate, up=up)
    if not need_input and not need_weights:
        raise ValueError(f"{what}: nothing wanted")
    _check_workspace(what, workspace)
    _check_device(what, x, dh=dh, w_gate=w_gate, w_up=w_up, gate=gate, up=up, offsets=offsets, workspace=workspace)
    if workspace is None:
        n = expert_gated_workspace_bytes(x.shape[0], w_gate.shape[-2], x, dense=offsets is None and need_input, cols=x.shape[1])[1]
        workspace = torch.empty(n, dtype=torch.uint8, device=x.device)
    dx = x.new_empty(x.shape) if need_input else None
    dwg, dwu = (w_gate.new_empty(w_gate.shape), w_gate.new_empty(w_gate.shape)) if need_weights else (None, None)
    opt = lambda t: None if t is None else describe(t)
    _launch(what, x, describe(dh), describe(x), describe(w_gate), describe(w_up), describe(gate), describe(up), _ptr(offsets), code, opt(dx),
            opt(dwg), opt(dwu), _ptr(workspace), _ws_bytes(workspace))
    return dx, dwg, dwu


# ------------------------------------------------------------------ around the layer
# The norm and the embeddings of the model that the layer belongs to; the conventions are the layer's.

def _check_scale_vector(what, x, weight):
    if weight is None:
        return F32
    if weight.dtype != x.dtype and weight.dtype != _torch().float32 or not weight.is_contiguous():
        _check_flat(what, x, (x.dtype, _torch().float32), weight=weight)
    _check_shape(what, "weight", weight, x.shape[-1:])
    return dtype_code(weight)


def _check_like(what, x, **named):
    """Buffers of x's shape and dtype."""
    _check_same_shape(what, x, **named)
    for name, t in named.items():
        if t is not None and t.dtype != x.dtype:
            raise TypeError(f"{what}: {name} is {t.dtype}, expected {x.dtype}")


def _rms_forward(what, x, weight, residual, residual_out, **more):
    _check_recorded(what, x, weight, residual, residual_out, *more.values())
    xd = describe(x)
    code = _check_scale_vector(what, x, weight)
    if residual is None and residual_out is not None:
        raise ValueError(f"{what}: residual_out without residual")
    _check_like(what, x, residual=residual, residual_out=residual_out, out=more.get("out"))
    _check_device(what, x, weight=weight, residual=residual, residual_out=residual_out, **more)
    h = x if residual is None else _rows_like(x) if residual_out is None else residual_out
    rstd = x.new_empty(x.shape[:-1], dtype=_torch().float32)
    return xd, code, h, rstd


def _rows_like(x):
    """An uninitialised buffer of x's shape with whole rows (empty_like costs 0.6 us less, and may take over strides)."""
    return _torch().empty_like(x) if x.is_contiguous() else x.new_empty(x.shape)


def rms_norm(x, weight=None, *, residual=None, eps: float = 1e-6, out=None, residual_out=None):
    """(y, h, rstd): h = x + residual in x's dtype (h is x without a residual) and its root-mean-square
    norm over the columns, y = h * rstd * weight (C ABI ``rms_norm``). x: [rows, cols] or [batch, rows,
    cols]; weight: [cols] of x's dtype or float32; rstd: float32, one per row. residual_out may be
    residual itself: the stream is then updated in place."""
    what = "rms_norm"
    xd, code, h, rstd = _rms_forward(what, x, weight, residual, residual_out, out=out)
    y = _rows_like(x) if out is None else out
    kept = residual is not None
    _launch(what, x, xd, describe(residual) if kept else None, _ptr(weight), code, eps, describe(y), describe(h) if kept else None, _ptr(rstd))
    return y, h, rstd


def rms_norm_mx8(x, weight=None, *, residual=None, eps: float = 1e-6, residual_out=None):
    """(q, scales, h, rstd): rms_norm with its output in 8 bits (C ABI ``rms_norm_mx8``): q float8_e4m3fn of
    x's shape, scales float8_e8m0fnu, one power of two per 32 columns; y = q * scales."""
    torch = _torch()
    what = "rms_norm_mx8"
    xd, code, h, rstd = _rms_forward(what, x, weight, residual, residual_out)
    q = x.new_empty(x.shape, dtype=torch.float8_e4m3fn)
    scales = x.new_empty((*x.shape[:-1], (x.shape[-1] + MX_BLOCK - 1) // MX_BLOCK), dtype=torch.float8_e8m0fnu)
    kept = residual is not None
    _launch(what, x, xd, describe(residual) if kept else None, _ptr(weight), code, eps, _ptr(q), _ptr(scales),
            describe(h) if kept else None, _ptr(rstd))
    return q, scales, h, rstd


def rms_norm_workspace_bytes(x) -> int:
    n = ctypes.c_size_t()
    _check(_lib().mns_rms_norm_workspace_bytes(ctypes.byref(describe(x)), ctypes.byref(n)), "mns_rms_norm_workspace_bytes")
    return n.value


def rms_norm_backward(dy, h, rstd, weight=None, *, dh=None, param_grads: bool = True, out=None, workspace=None):
    """(dx, dweight) of rms_norm (C ABI ``rms_norm_backward``): dx is the gradient of x and of residual, dh
    (the gradient that reaches h along the stream) included. out may be dh itself. dweight has weight's
    dtype; it is None without weight or with param_grads=False."""
    torch = _torch()
    what = "rms_norm_backward"
    _check_recorded(what, dy, h, rstd, weight, dh, out)
    hd = describe(h)
    _check_like(what, h, dy=dy, dh=dh, out=out)
    _check_flat(what, h, (torch.float32,), rstd=rstd)
    _check_shape(what, "rstd", rstd, h.shape[:-1])
    code = _check_scale_vector(what, h, weight)
    _check_workspace(what, workspace)
    _check_device(what, h, dy=dy, rstd=rstd, weight=weight, dh=dh, out=out, workspace=workspace)
    dx = h.new_empty(h.shape) if out is None else out
    dw = None
    if weight is not None and param_grads:
        dw = torch.empty_like(weight)
        if workspace is None:
            workspace = torch.empty(rms_norm_workspace_bytes(h), dtype=torch.uint8, device=h.device)
    _launch(what, h, describe(dy), hd, _ptr(rstd), _ptr(weight), code, None if dh is None else describe(dh), describe(dx), _ptr(dw),
            _ptr(workspace), 0 if workspace is None else _ws_bytes(workspace))
    return dx, dw


def _check_tokens(what, tokens):
    torch = _torch()
    _check_flat(what, tokens, (torch.int32, torch.int64), tokens=tokens)


def embed(tokens, table, *, scale: float = 1.0, out=None):
    """scale * table[tokens], a row of zeros for a token outside 0 .. rows - 1 (C ABI ``embed``). tokens: int32
    or int64, any shape; table: [rows, cols]; the result: [*tokens.shape, cols] (out: [tokens, cols])."""
    what = "embed"
    _check_recorded(what, table, out)
    _check_tokens(what, tokens)
    _check_rows(what, table, table=table, out=out)
    if table.shape[0] < 1:
        raise ValueError(f"{what}: table has no rows")
    if out is not None:
        _check_shape(what, "out", out, (tokens.numel(), table.shape[1]))
    _check_device(what, table, tokens=tokens, out=out)
    y = table.new_empty((tokens.numel(), table.shape[1])) if out is None else out
    _launch(what, table, _ptr(tokens), tokens.element_size(), describe(table), scale, describe(y))
    return y.view(*tokens.shape, table.shape[1]) if out is None else y


def embed_workspace_bytes(tokens: int, rows: int, cols: int) -> int:
    n = ctypes.c_size_t()
    _check(_lib().mns_embed_workspace_bytes(tokens, rows, cols, ctypes.byref(n)), "mns_embed_workspace_bytes")
    return n.value


def embed_backward(dy, tokens, rows: int, *, scale: float = 1.0, out=None, workspace=None):
    """The dense gradient of embed's table, [rows, cols] of dy's dtype: scale times the sum of dy's rows of each
    token, zero for a token that does not occur (C ABI ``embed_backward``). dy: [tokens, cols], or
    contiguous [*tokens.shape, cols]."""
    torch = _torch()
    what = "embed_backward"
    _check_recorded(what, dy, out)
    _check_tokens(what, tokens)
    if dy.dim() != 2 and dy.shape[:-1] == tokens.shape:
        if not dy.is_contiguous():
            raise ValueError(f"{what}: dy of more than two dimensions must be contiguous")
        dy = dy.view(tokens.numel(), dy.shape[-1])
    _check_rows(what, dy, dy=dy, out=out)
    _check_shape(what, "dy", dy, (tokens.numel(), dy.shape[1]))
    if rows < 1:
        raise ValueError(f"{what}: rows must be at least 1, got {rows}")
    if out is not None:
        _check_shape(what, "out", out, (rows, dy.shape[1]))
    _check_workspace(what, workspace)
    _check_device(what, dy, tokens=tokens, out=out, workspace=workspace)
    need = embed_workspace_bytes(tokens.numel(), rows, dy.shape[1])
    dt = dy.new_empty((rows, dy.shape[1])) if out is None else out
    if workspace is None:
        workspace = torch.empty(need, dtype=torch.uint8, device=dy.device)
    _launch(what, dy, describe(dy), _ptr(tokens), tokens.element_size(), scale, describe(dt), _ptr(workspace), _ws_bytes(workspace))
    return dt


def gram_trace(G, *, steps: int = DEFAULT_STEPS, coeffs=None, eps: float = DEFAULT_EPS,
               iter_dtype: Optional[int] = None, restart_mask: int = STABILIZED_RESTART_MASK):
    """(O, trace) for the first matrix of G: the Gram iterate after each step 1 .. K-1 as a
    [K-1, n, n] fp32 tensor (C ABI ``gram_ns_trace``)."""
    torch = _torch()
    _check_device("gram_ns_trace", G)
    G1 = G[0] if G.dim() == 3 else G
    p = ns_params(steps, coeffs, eps, iter_dtype, dtype_code(G1), restart_mask)
    n = min(G1.shape)
    out = torch.empty_like(G1)
    trace = torch.empty(steps - 1, n, n, dtype=torch.float32, device=G1.device)
    ws = _workspace(GRAM, G1, p, None)
    _check(_lib().gram_ns_trace(ctypes.byref(describe(G1)), ctypes.byref(describe(out)),
                                 ctypes.byref(p), ctypes.c_void_p(ws.data_ptr()), _ws_bytes(ws),
                                 ctypes.c_void_p(trace.data_ptr()), _stream_ptr(G1)),
           "gram_ns_trace")
    return out, trace


# ------------------------------------------------------------------ launch timing

def timing_enable(on: bool = True):
    _check(_lib().mns_timing_enable(1 if on else 0), "mns_timing_enable")


def timing_reset():
    _check(_lib().mns_timing_reset(), "mns_timing_reset")


def timing_query() -> dict:
    """{kind_name: (total_ms, launches)} over the events recorded since the last reset."""
    L = _lib()
    out = {}
    for k in range(L.mns_timing_kinds()):
        ms, n = ctypes.c_double(0.0), ctypes.c_int64(0)
        _check(L.mns_timing_query(k, ctypes.byref(ms), ctypes.byref(n)), "mns_timing_query")
        out[L.mns_kernel_kind_name(k).decode()] = (ms.value, n.value)
    return out
