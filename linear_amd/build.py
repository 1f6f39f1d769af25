"""Build the gfx950 HIP library ``linear_amd/liblinear_amd.so`` with hipcc.

Run ``python -m linear_amd.build``.  Always recompiles (the build check must
really compile); object files go to ``_build/`` at the repository root.
"""
from __future__ import annotations

import concurrent.futures
import os
import re
import shutil
import subprocess
import sys

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
OUT = os.path.join(HERE, "liblinear_amd.so")
# measurement kernels for bench.py's ceilings, kept out of the layer's library
PROBE_OUT = os.path.join(HERE, "liblinear_probe.so")
PROBE_SOURCES = ["probe.hip"]
BUILD_DIR = os.path.join(ROOT, "_build")

SOURCES = ["gemm_f16.hip", "gemm_bf16.hip", "skinny.hip", "epilogue.hip", "indexed.hip", "product.hip", "gradnorm.hip",
           "gated_f16.hip", "gated_bf16.hip", "grad_f16.hip", "grad_bf16.hip",
           "linear_abi.hip", "train_abi.hip"]

# sources whose kernels set m0 in inline assembly (lds_dma16_raw), which the compiler is not told
RAW_M0_SOURCES = ("grad_f16.hip", "grad_bf16.hip")

HIPCC_FLAGS = [
    "--offload-arch=gfx950",
    "-O3",
    "-std=c++20",
    "-fPIC",
    "-Wall",
    "-fno-gpu-flush-denormals-to-zero",   # binary16 subnormals are kept (IEEE gradual underflow)
    "-ffp-contract=off",
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
    "-I" + os.path.join(ROOT, "include"),
    "-Rpass-analysis=kernel-resource-usage",   # per-kernel registers, spills, scratch (checked below)
]


def hipcc() -> str:
    for cand in (shutil.which("hipcc"), "/opt/rocm/bin/hipcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("hipcc not found")


def _resources(text: str) -> dict:
    """Kernel name -> {field: value} from hipcc's kernel-resource-usage remarks."""
    res, name = {}, None
    for line in text.splitlines():
        if "[-Rpass-analysis=kernel-resource-usage]" not in line:
            continue
        body = line.split("remark:", 1)[1].rsplit("[-Rpass", 1)[0].strip()
        key, _, val = body.partition(": ")
        if key == "Function Name":
            name = val
            res[name] = {}
        elif name is not None:
            res[name][key] = val
    return res


def _other_m0_uses(asm: str) -> list:
    """The instructions naming m0 that are not lds_dma16_raw's three: m0's write, the wait states
    and the direct-to-LDS load that reads it.  Any other would be the compiler's own use, whose
    value the inline assembly may have overwritten."""
    code = [l.split(";")[0].split("//")[0].strip() for l in asm.splitlines()]
    code = [l for l in code if l and not l.startswith(".") and not l.endswith(":")]
    bad = []
    for i, line in enumerate(code):
        if not re.search(r"\bm0\b", line):
            continue
        rest = [l.split() for l in code[i + 1:i + 3]] + [[""]] * 2
        if not (line.startswith("s_mov_b32 m0,") and rest[0] == ["s_nop", "3"] and
                rest[1][0] == "buffer_load_dwordx4" and rest[1][-1] == "lds"):
            bad.append(line)
    return bad


def _compile(src: str) -> str:
    obj = os.path.join(BUILD_DIR, os.path.splitext(src)[0] + ".o")
    cmd = [hipcc(), *HIPCC_FLAGS, "-c", os.path.join(CSRC, src), "-o", obj]
    if src in RAW_M0_SOURCES:
        cmd.append("-save-temps=obj")
    r = subprocess.run(cmd, capture_output=True, text=True)
    out = r.stdout + r.stderr
    noise = ("is not a recognized feature for this target", "kernel-resource-usage")
    msg = "\n".join(l for l in out.splitlines()
                    if not any(n in l for n in noise) and not l.lstrip().startswith(("|", "^", "In file included from"))
                    and not (l[:6].strip().isdigit() and " | " in l))
    if r.returncode != 0:
        raise RuntimeError("hipcc failed for %s:\n%s" % (src, msg))
    if msg.strip():
        print(msg, file=sys.stderr)
    # every kernel must run from registers and LDS: scratch memory (spills, or an
    # argument copy indexed at run time) costs a memory round trip per access
    res = _resources(out)
    bad = {k: v for k, v in res.items()
           if v.get("ScratchSize [bytes/lane]", "0") != "0" or v.get("VGPRs Spill", "0") != "0"}
    with open(os.path.join(BUILD_DIR, os.path.splitext(src)[0] + ".resources.txt"), "w") as f:
        for k, v in sorted(res.items()):
            f.write("%s %s\n" % (k, " ".join("%s=%s" % (a.replace(" ", "_"), b) for a, b in v.items())))
    if bad:
        raise RuntimeError("kernels in %s use scratch memory: %s" % (src, ", ".join(sorted(bad))))
    if src in RAW_M0_SOURCES:
        asm = os.path.join(BUILD_DIR, os.path.splitext(src)[0] + "-hip-amdgcn-amd-amdhsa-gfx950.s")
        with open(asm) as f:
            uses = _other_m0_uses(f.read())
        if uses:
            raise RuntimeError("%s: the compiler uses m0 itself beside the inline assembly: %s" % (src, uses[0]))
    return obj


def build(verbose: bool = True) -> str:
    os.makedirs(BUILD_DIR, exist_ok=True)
    # a failed build must not leave the previous library behind for tests and
    # benchmarks to load
    for out in (OUT, PROBE_OUT):
        if os.path.exists(out):
            os.remove(out)
    with concurrent.futures.ThreadPoolExecutor(max_workers=len(SOURCES) + len(PROBE_SOURCES)) as ex:
        objs = list(ex.map(_compile, SOURCES + PROBE_SOURCES))
    for out, part in ((OUT, objs[:len(SOURCES)]), (PROBE_OUT, objs[len(SOURCES):])):
        tmp = out + ".tmp%d" % os.getpid()
        cmd = [hipcc(), "--offload-arch=gfx950", "-shared", "-fPIC", *part, "-o", tmp]
        subprocess.run(cmd, check=True)
        os.replace(tmp, out)
        if verbose:
            print("built", out)
    return OUT


if __name__ == "__main__":
    build()
