"""Build libmuon_ns.so in-tree with hipcc for gfx950 (no JIT cache, no torch extension).

Usage: python -m newton_schulz_matrix_muon_amd.build [-v] [--hostsan]
"""
from __future__ import annotations

import os
import re
import subprocess
import sys

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
LIB = os.path.join(PKG, "libmuon_ns.so")
SOURCES = ["muon_ns.hip", os.path.join("layer", "layer.hip"), os.path.join("layer", "block.hip"),
           os.path.join("layer", "gated.hip")]

HIPCC_FLAGS = [
    "--offload-arch=gfx950", "-O3", "-std=c++17", "-fPIC", "-shared", "-fvisibility=hidden",
    "-Wall", "-Wno-unused-function",
    # no packed-fp32 instructions in device code
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
]


def hipcc() -> str:
    for cand in (os.environ.get("HIPCC"), "/opt/rocm/bin/hipcc"):
        if cand and os.path.exists(cand):
            return cand
    return "hipcc"


BUILD = os.path.join(ROOT, "_build")
HOSTSAN_LIB = os.path.join(BUILD, "libmuon_ns_hostsan.so")


RESOURCES = "-Rpass-analysis=kernel-resource-usage"


def check_registers(remarks: str) -> int:
    """Raise if a kernel of the compiler's resource remarks (RESOURCES) uses accumulation registers; returns the
    number of kernels. The compiler moves an MFMA's result out of them (v_accvgpr_read) behind a branch without
    the wait states that the MFMA needs, so a kernel whose sums live there reads them too early. Kernels of at
    least two waves a SIMD (__launch_bounds__) keep their sums in vector registers, where it does wait."""
    used = re.findall(r"Function Name: (\S+).*?AGPRs: (\d+)", remarks, re.S)
    bad = [name for name, n in used if int(n)]
    if bad:
        raise RuntimeError("kernels with sums in accumulation registers: " + ", ".join(bad))
    return len(used)


def _run(cmds, verbose: bool, what: str) -> str:
    """Run the commands side by side; raise with the compiler's messages if one fails. Returns the remarks."""
    remarks = ""
    if verbose:
        for cmd in cmds:
            print(" ".join(cmd), flush=True)
    procs = [subprocess.Popen(c, stdout=subprocess.PIPE, stderr=subprocess.PIPE, text=True) for c in cmds]
    for p, (_, err) in zip(procs, [p.communicate() for p in procs]):
        remarks += "".join(l + "\n" for l in err.splitlines() if RESOURCES in l)
        errs = [l for l in err.splitlines() if "packed-fp32-ops" not in l and RESOURCES not in l]
        if p.returncode != 0:
            raise RuntimeError(f"{what} failed:\n" + "\n".join(errs))
        if verbose and errs:
            print("\n".join(errs))
    return remarks


def _object(source: str, suffix: str) -> str:
    return os.path.join(BUILD, os.path.splitext(os.path.basename(source))[0] + suffix)


def build(verbose: bool = False) -> str:
    os.makedirs(BUILD, exist_ok=True)
    tmp = LIB + ".tmp"
    objs = [_object(s, ".o") for s in SOURCES]
    flags = [f for f in HIPCC_FLAGS if f != "-shared"]
    remarks = _run([[hipcc(), *flags, RESOURCES, "-I", os.path.join(ROOT, "include"), "-I", CSRC, "-c", os.path.join(CSRC, s), "-o", o]
                    for s, o in zip(SOURCES, objs)], verbose, "hipcc")
    if not check_registers(remarks):
        raise RuntimeError("hipcc printed no resource remarks")
    _run([[hipcc(), *HIPCC_FLAGS, *objs, "-o", tmp]], verbose, "hipcc (link)")
    os.replace(tmp, LIB)
    return LIB


def llvm_tool(name: str) -> str:
    cand = os.path.join("/opt/rocm/llvm/bin", name)
    return cand if os.path.exists(cand) else name


def build_hostsan(verbose: bool = False) -> str:
    """A copy of the library whose host code (argument checks, workspace arithmetic, launch
    set-up) is built with AddressSanitizer and UndefinedBehaviorSanitizer, for CPU-side tests.
    Its device code is the built objects' own GPU binaries (their .hip_fatbin sections), so only
    the host pass is compiled here; no device code is instrumented. Load it only in a process
    that preloads the ASan runtime, and never on a GPU."""
    objs = [_object(s, ".o") for s in SOURCES]
    if not os.path.exists(LIB) or not all(os.path.exists(o) for o in objs):
        raise FileNotFoundError(f"{LIB} or its objects are missing: run build() first")
    fatbins = [_object(s, "_gfx950.hipfb") for s in SOURCES]
    _run([[llvm_tool("llvm-objcopy"), "-O", "binary", "--only-section=.hip_fatbin", o, f]
          for o, f in zip(objs, fatbins)], False, "extracting the GPU binary")
    if not all(os.path.getsize(f) for f in fatbins):
        raise RuntimeError("an object holds no GPU binary")
    flags = [f for f in HIPCC_FLAGS if f not in ("-O3", "-shared")]
    san = ["-Xarch_host", "-fsanitize=address", "-Xarch_host", "-fsanitize=undefined",
           "-Xarch_host", "-fno-sanitize-recover=undefined", "-Xarch_host", "-fno-omit-frame-pointer"]
    sans = [_object(s, "_hostsan.o") for s in SOURCES]
    _run([[hipcc(), *flags, "-O1", "-g", *san, "--cuda-host-only", "-Xclang", "-fcuda-include-gpubinary", "-Xclang", f,
           "-I", os.path.join(ROOT, "include"), "-I", CSRC, "-c", os.path.join(CSRC, s), "-o", o]
          for s, f, o in zip(SOURCES, fatbins, sans)], verbose, "hipcc (host sanitizers)")
    tmp = HOSTSAN_LIB + ".tmp"
    _run([[hipcc(), *flags, "-shared", *san, *sans, "-o", tmp]], verbose, "hipcc (host sanitizers, link)")
    os.replace(tmp, HOSTSAN_LIB)
    return HOSTSAN_LIB


if __name__ == "__main__":
    print(build(verbose="-v" in sys.argv))
    if "--hostsan" in sys.argv:
        print(build_hostsan(verbose="-v" in sys.argv))
