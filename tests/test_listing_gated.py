"""test_listing.py's rule on the scalars that the DMA reads, for the 256 x 256 tiles of two matrices: the gated block's
forward product, its input gradient and its weights' gradients, and those whose last round is cut."""
import pytest

from test_listing import instructions, listing, pytestmark, registers, states_before_read  # noqa: F401 (pytestmark applies here too)


@pytest.mark.parametrize("dtype", ["__bf16", "_Float16"])
@pytest.mark.parametrize("kernel", ["EX_GATE, {}", "EX_DX2, {}", "EX_DW2, {}", "EX_GATE, {}, true", "EX_DX2, {}, true"])
def test_the_dma_waits_for_the_scalars_it_reads(tmp_path, kernel, dtype):
    ins, follow = instructions(listing(tmp_path, "layer/expert_pingpong.hpp", f"expert_gemm_pp<{kernel.format(dtype)}>(GatedArgs)")[0])
    assert sum(name.startswith("buffer_load") and ops[-1] == "0" for name, ops in ins) >= 16
    reads = lambda name, ops: set().union(*(registers("s", o) for o in ops)) if name.startswith("buffer_") else set()
    writes = lambda name, ops: registers("s", ops[0]) if name.startswith("s_") else set()
    waits = [i for i, (name, ops) in enumerate(ins) if name == "s_nop" and int(ops[0], 0) == 4]
    assert len(waits) >= 2                                     # one in each place that moves on by a stage
    for i, (name, ops) in enumerate(ins):
        if name.startswith(("v_readfirstlane", "v_readlane")):
            assert states_before_read(ins, follow, i, registers("s", ops[0]), reads, writes, 5) >= 5, (name, ops)
    # the statement sets m0 without the compiler's knowledge, so nothing else may live in it
    assert not [(name, ops) for name, ops in ins if "m0" in ops and not (name == "s_mov_b32" and ops[0] == "m0")]
    # nothing in scratch: its loads and stores would stand between the queue's counts
    assert not [name for name, _ in ins if name.startswith("scratch_")]
