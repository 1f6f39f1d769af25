"""Build the gfx950 HIP library ``linear_amd/liblinear_amd.so`` with hipcc.

Run ``python -m linear_amd.build``.  Always recompiles (the build check must
really compile); object files go to ``_build/`` at the repository root.
"""
from __future__ import annotations

import concurrent.futures
import importlib.util
import os
import re
import shutil
import subprocess
import sys
import sysconfig

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
           "loss_f16.hip", "loss_bf16.hip", "loss.hip", "adamw.hip",
           "linear_abi.hip", "train_abi.hip", "loss_abi.hip",
           "adamw_abi.hip"]

# the binding's marshalling of many tensors, host code against torch's headers
MARSHAL = "marshal.cpp"
MARSHAL_OUT = os.path.join(HERE, "_marshal.so")

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


def _asm_resources(asm: str) -> dict:
    """The same from the kernels' metadata at the end of their assembly (with -save-temps hipcc makes no
    remarks)."""
    fields = {"vgpr_count": "VGPRs", "agpr_count": "AGPRs", "sgpr_count": "TotalSGPRs", "vgpr_spill_count": "VGPRs Spill",
              "sgpr_spill_count": "SGPRs Spill", "private_segment_fixed_size": "ScratchSize [bytes/lane]",
              "group_segment_fixed_size": "LDS Size [bytes/block]"}
    res = {}
    for entry in re.split(r"^  - ", asm.partition("amdhsa.kernels:")[2], flags=re.M)[1:]:
        values = dict(re.findall(r"^ *\.(\w+): +(\S+)$", entry, flags=re.M))
        if "name" in values:
            res[values["name"]] = {label: values[key] for key, label in fields.items() if key in values}
    return res


def _check_resources(src: str, res: dict) -> None:
    """Every kernel must run from registers and LDS: scratch memory (spills, or an argument copy indexed
    at run time) costs a memory round trip per access."""
    if not res and not src.endswith("_abi.hip"):          # (host code alone)
        raise RuntimeError("no kernel's resources were found for %s" % src)
    bad = {k: v for k, v in res.items()
           if v.get("ScratchSize [bytes/lane]") != "0" or v.get("VGPRs Spill") != "0"}
    if bad:
        raise RuntimeError("kernels in %s use scratch memory: %s" % (src, ", ".join(sorted(bad))))


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
    asm = ""
    if src in RAW_M0_SOURCES:
        with open(os.path.join(BUILD_DIR, os.path.splitext(src)[0] + "-hip-amdgcn-amd-amdhsa-gfx950.s")) as f:
            asm = f.read()
    res = _asm_resources(asm) if asm else _resources(out)
    with open(os.path.join(BUILD_DIR, os.path.splitext(src)[0] + ".resources.txt"), "w") as f:
        for k, v in sorted(res.items()):
            f.write("%s %s\n" % (k, " ".join("%s=%s" % (a.replace(" ", "_"), b) for a, b in v.items())))
    _check_resources(src, res)
    uses = _other_m0_uses(asm)
    if uses:
        raise RuntimeError("%s: the compiler uses m0 itself beside the inline assembly: %s" % (src, uses[0]))
    return obj


def _marshal_needs() -> str | None:
    """What is missing here for the binding's module; the library itself needs none of it."""
    if shutil.which("g++") is None:
        return "g++"
    if not os.path.exists(os.path.join(sysconfig.get_paths()["include"], "Python.h")):
        return "Python's headers"
    spec = importlib.util.find_spec("torch")
    home = os.path.dirname(spec.origin) if spec is not None and spec.origin else ""
    if not os.path.exists(os.path.join(home, "include", "torch", "csrc", "autograd", "python_variable.h")):
        return "torch's headers"
    if not os.path.exists(os.path.join(home, "lib", "libtorch_python.so")):
        return "torch's libraries"
    return None


def _compile_marshal() -> str | None:
    """Builds the binding's module; where something for it is missing, says what, and the binding does without."""
    needs = _marshal_needs()
    if needs is not None:
        print("not built: %s (no %s); the binding reads tensors at more host time" % (MARSHAL_OUT, needs), file=sys.stderr)
        return None
    import torch
    home = os.path.dirname(torch.__file__)
    include = os.path.join(home, "include")
    tmp = MARSHAL_OUT + ".tmp%d" % os.getpid()
    cmd = ["g++", "-O2", "-std=c++17", "-shared", "-fPIC", "-D_GLIBCXX_USE_CXX11_ABI=%d" % torch._C._GLIBCXX_USE_CXX11_ABI,
           "-isystem", include, "-isystem", os.path.join(include, "torch", "csrc", "api", "include"),
           "-isystem", sysconfig.get_paths()["include"], os.path.join(CSRC, MARSHAL), "-o", tmp,
           "-L" + os.path.join(home, "lib"), "-ltorch_python", "-ltorch_cpu", "-lc10"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError("g++ failed for %s:\n%s" % (MARSHAL, r.stderr))
    os.replace(tmp, MARSHAL_OUT)
    return MARSHAL_OUT


def build(verbose: bool = True) -> str:
    os.makedirs(BUILD_DIR, exist_ok=True)
    # a failed build must not leave the previous library behind for tests and
    # benchmarks to load
    for out in (OUT, PROBE_OUT, MARSHAL_OUT):
        if os.path.exists(out):
            os.remove(out)
    with concurrent.futures.ThreadPoolExecutor(max_workers=len(SOURCES) + len(PROBE_SOURCES) + 1) as ex:
        marshal = ex.submit(_compile_marshal)
        objs = list(ex.map(_compile, SOURCES + PROBE_SOURCES))
    for out, part in ((OUT, objs[:len(SOURCES)]), (PROBE_OUT, objs[len(SOURCES):])):
        tmp = out + ".tmp%d" % os.getpid()
        cmd = [hipcc(), "--offload-arch=gfx950", "-shared", "-fPIC", *part, "-o", tmp]
        subprocess.run(cmd, check=True)
        os.replace(tmp, out)
        if verbose:
            print("built", out)
    if marshal.result() is not None and verbose:
        print("built", MARSHAL_OUT)
    return OUT


if __name__ == "__main__":
    build()
