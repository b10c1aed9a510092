"""AdamW in 8 bits with its step on the device: what the binding and the C ABI refuse, before any HIP call (no GPU is needed)."""
import ctypes

import pytest

from test_block_args import P, Q, R, S, U
from test_layer_args import ARG, BF16, L, OK, ops, torch  # noqa: F401 (fixtures)


def test_abi_refusals_of_a_step_on_the_device(L):
    from newton_schulz_matrix_muon_amd.ops import MnsAdamw8Params
    arr = lambda v: (ctypes.c_void_p * 1)(v)

    def call(step, at, numel=100):
        lists = [arr(v) for v in ((P, Q, R, R + 4096, S, S + 4096) if numel else (None,) * 6)]
        return L.adamw8_step(1, *lists, (ctypes.c_int64 * 1)(numel), BF16, ctypes.byref(MnsAdamw8Params(1e-3, 0.9, 0.95, 1e-8, 0.1, step, 1, 0, at)), None)
    assert call(0, None) == ARG and call(1, U + 4) == ARG
    assert call(0, U, numel=0) == OK                                         # `step` is not read then
    for buf in (P, P + 192, Q, Q + 192, R + 96, R + 4096, S, S + 4096):      # over a parameter, a gradient, codes, powers
        assert call(1, buf) == ARG, hex(buf)


def test_binding_refuses_steps_on_the_device(torch, ops):
    p = torch.zeros(100)
    call = lambda step: ops.adamw8_step([p], [p.clone()], [ops.adamw8_state(p)], lr=1e-3, step=step)
    for step in (torch.tensor(1.0), torch.tensor(1, dtype=torch.int32), torch.tensor(True)):
        with pytest.raises(TypeError, match="step"):
            call(step)
    for step in (torch.zeros(2, dtype=torch.int64), torch.zeros(0, dtype=torch.int64)):
        with pytest.raises(ValueError, match="one number"):
            call(step)
    with pytest.raises(ValueError, match="device tensors"):
        call(torch.tensor(1))


def test_hybrid_refuses_a_step_on_the_device_where_the_host_needs_it(torch, ops, monkeypatch):
    seen = []
    for name in ("muon_step_grouped", "adamw_step", "adamw8_step"):
        monkeypatch.setattr(ops, name, lambda *a, _n=name, **k: seen.append((_n, k)))
    p, step = torch.zeros(4), torch.tensor(1)
    both = [(p, p, p, p), (p, p, ops.adamw8_state(p))]
    with pytest.raises(ValueError, match="on the host"):
        ops.hybrid_step([(p, p, p)], both, muon={}, adamw=dict(lr=1e-3, step=step, bias_correction=True))
    assert not seen                                                          # nothing was enqueued
    ops.hybrid_step([(p, p, p)], both, muon={}, adamw=dict(lr=1e-3, step=step), seed=3)
    assert seen == [("muon_step_grouped", {}), ("adamw_step", dict(lr=1e-3)), ("adamw8_step", dict(lr=1e-3, step=step, seed=3))]
