"""The workspace of the gated block's dense calls: the split's part only where a round is cut (no GPU is needed)."""
import ctypes

import pytest

from test_layer_args import ARG, BF16, DTYPE, F16, F32, L, SHAPE, ops, torch  # noqa: F401 (fixtures)


def sizes(L, rows, inner, cols, dtype=BF16):
    a, b = ctypes.c_size_t(), ctypes.c_size_t()
    assert L.mns_expert_gated_dense_workspace_bytes(rows, inner, cols, dtype, ctypes.byref(a), ctypes.byref(b)) == 0
    c, d = ctypes.c_size_t(), ctypes.c_size_t()
    assert L.mns_expert_gated_workspace_bytes(rows, inner, 0, dtype, ctypes.byref(c), ctypes.byref(d)) == 0
    split = c.value
    assert a.value in (0, split) and b.value in (d.value, d.value - split)
    return a.value > 0, b.value == d.value


@pytest.mark.parametrize("dtype", [BF16, F16])
def test_the_split_has_room_where_a_round_is_cut(L, dtype):
    # (forward, input gradient): few rows, too few tiles, one whole round, widths of no whole chunk; then cut rounds of either
    for shape in ((1, 18432, 7168), (1, 4096, 3000), (4, 18432, 7168), (16, 4096, 3000), (300, 1024, 4096), (1024, 8192, 4096), (0, 18432, 7168), (600, 64, 4096)):
        assert not sizes(L, *shape, dtype)[0], shape
    # 2 x 144 tiles of 256 x 128 and, of 256 x 256, 2 x 28; 8 x 16, half of the CUs
    assert sizes(L, 509, 18432, 7168, dtype) == (True, True) and sizes(L, 2048, 2048, 4096, dtype)[0]
    assert sizes(L, 600, 2064, 2568, dtype)[0] and sizes(L, 1290, 2047, 2056, dtype) == (False, True)
    assert not sizes(L, 1, 18432, 7168, dtype)[1] and not sizes(L, 600, 1152, 4096, dtype)[1]


def test_what_the_call_refuses(L):
    a, b = ctypes.c_size_t(), ctypes.c_size_t()
    f = lambda rows, inner, cols, dtype=BF16, p=a, q=b: L.mns_expert_gated_dense_workspace_bytes(rows, inner, cols, dtype, p and ctypes.byref(p), q and ctypes.byref(q))
    assert f(8, 32, 64, p=None) == ARG and f(8, 32, 64, q=None) == ARG and f(8, 32, 64, 5) == DTYPE
    for bad in ((-1, 32, 64), (8, 0, 64), (8, 32, 0), (8, 32, (1 << 20) + 1), (8, (1 << 20) + 1, 64), ((1 << 24) + 1, 32, 64)):
        assert f(*bad) == SHAPE, bad
    assert f(8, 32, 64, F32) == 0 and (a.value, b.value) == (0, 2 * 8 * 32 * 4)
    assert f(1 << 24, 1 << 20, 1 << 20) == 0


def test_the_binding_asks_with_its_own_shape(torch, ops):
    x = torch.zeros(1, dtype=torch.bfloat16)
    assert ops.expert_gated_workspace_bytes(1, 18432, x, dense=True, cols=7168) == (0, 2 * 18432 * 2)
    assert ops.expert_gated_workspace_bytes(1, 18432, x, dense=True)[0] > 0
    assert ops.expert_gated_workspace_bytes(1, 18432, x, cols=7168) == (0, 2 * 18432 * 2)
