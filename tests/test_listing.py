"""Rules that the compiler cannot keep for the kernels, checked on the listings it makes of them (gfx950, no GPU needed)."""
import os
import re
import shutil
import subprocess

import pytest

from newton_schulz_matrix_muon_amd import build as b

pytestmark = pytest.mark.skipif(not os.path.exists("/opt/rocm/bin/hipcc"), reason="no compiler")


def listing(tmp_path, include, kernel, csrc=b.CSRC, flags=()):
    """The gfx950 assembly of one kernel's instantiation, and what the compiler said."""
    src, out = tmp_path / "one.hip", tmp_path / "one.s"
    src.write_text(f'#include <hip/hip_runtime.h>\n#include "{include}"\nnamespace mns {{ template __global__ void {kernel}; }}\n')
    flags = [f for f in b.HIPCC_FLAGS if f != "-shared"] + list(flags)
    r = subprocess.run([b.hipcc(), *flags, "--cuda-device-only", "-S", "-I", os.path.join(b.ROOT, "include"), "-I", csrc,
                        str(src), "-o", str(out)], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-3000:]
    return out.read_text(), r.stderr


def instructions(text):
    """(name, operands) of a kernel's instructions and, for each, the indexes of those that can follow it."""
    body = text[re.search(r"^_Z\w+:", text, re.M).end():text.index(".Lfunc_end")]
    ins, labels = [], {}
    for line in body.splitlines():
        line = line.split(";")[0].strip()
        if m := re.match(r"(\.\w+):", line):
            labels[m[1]] = len(ins)
        elif line and not line.startswith("."):
            name, _, rest = line.replace("\t", " ").partition(" ")
            ins.append((name, [o.strip().split(" ")[0] for o in re.split(r",(?![^\[]*\])", rest)]))
    follow = []
    for i, (name, ops) in enumerate(ins):
        to = [] if name in ("s_endpgm", "s_branch") else [i + 1]
        follow.append(to + ([labels[ops[0]]] if "branch" in name else []))
    return ins, follow


def registers(kind, operand):
    """Numbers of the registers of a kind (s, v or a) that an operand names."""
    m = re.fullmatch(kind + r"(?:(\d+)|\[(\d+):(\d+)\])", operand)
    return set() if not m else {int(m[1])} if m[1] else set(range(int(m[2]), int(m[3]) + 1))


def states_before_read(ins, follow, at, written, reads, forgets, most):
    """Fewest wait states between instruction `at` and one that reads what it wrote, over all paths (most: none within)."""
    best, seen, stack = most, {}, [(j, 0, frozenset(written)) for j in follow[at]]
    while stack:
        j, n, live = stack.pop()
        if n >= best or not live or seen.get((j, live), most) <= n:
            continue
        seen[j, live] = n
        name, ops = ins[j]
        if reads(name, ops) & live:
            best = n
            continue
        live = live - forgets(name, ops)
        n += int(ops[0], 0) + 1 if name == "s_nop" else 1
        stack += [(k, n, live) for k in follow[j]]
    return best


@pytest.mark.parametrize("dtype", ["__bf16", "_Float16"])
@pytest.mark.parametrize("mode", ["EX_FWD", "EX_DX", "EX_DW"])
def test_the_dma_waits_for_the_scalars_it_reads(tmp_path, mode, dtype):
    """A vector memory instruction may read a scalar register five wait states after a vector instruction wrote it,
    at the earliest. The compiler does not look into the asm statement that issues the DMA: a wait has to follow
    the last of the scalars' writes (and the compiler must not write them again on the way)."""
    ins, follow = instructions(listing(tmp_path, "layer/expert_pingpong.hpp", f"expert_gemm_pp<{mode}, {dtype}>(ExpertArgs)")[0])
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


@pytest.mark.parametrize("dtype", ["float", "__bf16", "_Float16"])
def test_sums_in_accumulation_registers_are_refused(tmp_path, dtype):
    """The few rows' kernel as it is passes the build's check; built for one wave a SIMD, where the compiler puts its sums
    into accumulation registers, it does not."""
    kernel = f"expert_few_fwd<{dtype}, CHUNK_ALIGNED>(ExpertArgs)"
    assert b.check_registers(listing(tmp_path, "layer/expert_few.hpp", kernel, flags=[b.RESOURCES])[1]) == 1
    one = tmp_path / "csrc"
    shutil.copytree(b.CSRC, one)
    path = one / "layer" / "expert_few.hpp"
    text = path.read_text()
    assert text.count("__launch_bounds__(256, 2) expert_few_fwd") == 1
    path.write_text(text.replace("__launch_bounds__(256, 2) expert_few_fwd", "__launch_bounds__(256) expert_few_fwd"))
    asm, said = listing(tmp_path, "layer/expert_few.hpp", kernel, csrc=str(one), flags=[b.RESOURCES])
    assert "v_accvgpr_read" in asm
    with pytest.raises(RuntimeError, match="expert_few_fwd"):
        b.check_registers(said)
