"""The build's checks of its kernels: those that set m0 in inline assembly, on assembly text; registers
and scratch memory."""
import os
import shutil

import pytest
import torch

import linear_amd as la
from linear_amd import build

LOAD = "\ts_mov_b32 m0, s53\n\ts_nop 3\n\tbuffer_load_dwordx4 v1, s[4:7], 0 offen lds\n"


def test_only_the_inline_loads_may_use_m0():
    assert build._other_m0_uses("kernel:\n\tv_mov_b32_e32 v0, 0\n" + LOAD + "; m0 in a comment\n" + LOAD) == []
    for other in ("\tds_gws_barrier v0 offset:0\n\ts_add_u32 m0, m0, 16\n", "\ts_mov_b32 s3, m0\n",
                  "\ts_mov_b32 m0, s2\n\tv_movrels_b32_e32 v0, v1\n",
                  "\ts_mov_b32 m0, s2\n\ts_nop 0\n\tbuffer_load_dword v1, s[4:7], 0 offen lds\n"):
        assert len(build._other_m0_uses(LOAD + other + LOAD)) == 1
    assert build._other_m0_uses("\ts_mov_b32 m0, s2\n") == ["s_mov_b32 m0, s2"]


SCRATCH = """#include <hip/hip_runtime.h>
extern "C" __global__ void indexed_array(const int* at, float* out) {
    float local[64];
    for (int i = 0; i < 64; ++i) local[i] = out[i * at[i]];
    out[threadIdx.x] = local[at[threadIdx.x] & 63] + local[at[threadIdx.x + 64] & 63];
}
"""
PLAIN = """#include <hip/hip_runtime.h>
extern "C" __global__ void plain(float* out) { out[threadIdx.x] = 1.f; }
"""


@pytest.mark.skipif(not (shutil.which("hipcc") or os.path.exists("/opt/rocm/bin/hipcc")), reason="no hipcc")
@pytest.mark.parametrize("raw_m0", [False, True], ids=["remarks", "assembly"])
def test_a_kernel_with_scratch_memory_fails_the_build(raw_m0, tmp_path, monkeypatch):
    """Both where hipcc reports its kernels' resources and where the assembly is kept."""
    monkeypatch.setattr(build, "CSRC", str(tmp_path))
    monkeypatch.setattr(build, "BUILD_DIR", str(tmp_path))
    monkeypatch.setattr(build, "RAW_M0_SOURCES", ("scratch.hip", "plain.hip") if raw_m0 else ())
    for name, text in (("scratch", SCRATCH), ("plain", PLAIN)):
        (tmp_path / (name + ".hip")).write_text(text)
    with pytest.raises(RuntimeError, match="scratch memory: indexed_array"):
        build._compile("scratch.hip")
    build._compile("plain.hip")
    report = (tmp_path / "plain.resources.txt").read_text()
    assert report.startswith("plain ") and "ScratchSize_[bytes/lane]=0" in report and "VGPRs_Spill=0" in report


def test_a_source_whose_kernels_are_not_found_fails_the_build():
    with pytest.raises(RuntimeError, match="no kernel"):
        build._check_resources("grad_f16.hip", {})
    build._check_resources("train_abi.hip", {})
    with pytest.raises(RuntimeError, match="scratch"):
        build._check_resources("loss.hip", {"k": {"VGPRs Spill": "0"}})


def test_the_library_is_built_without_what_the_bindings_module_needs(tmp_path, monkeypatch, capsys):
    """g++, Python's and torch's headers are the module's alone; the library's build goes on without them."""
    monkeypatch.setattr(build, "MARSHAL_OUT", str(tmp_path / "_marshal.so"))
    with monkeypatch.context() as c:
        c.setattr(build.shutil, "which", lambda name: None)
        assert build._compile_marshal() is None and "no g++" in capsys.readouterr().err
    with monkeypatch.context() as c:
        c.setattr(build.sysconfig, "get_paths", lambda: {"include": str(tmp_path)})
        assert build._compile_marshal() is None and "Python's headers" in capsys.readouterr().err
    with monkeypatch.context() as c:
        c.setattr(build.importlib.util, "find_spec", lambda name: None)
        assert build._compile_marshal() is None and "torch's headers" in capsys.readouterr().err
    assert not os.listdir(tmp_path)


def test_the_binding_without_its_module(tmp_path, monkeypatch):
    """The module's calls give None, so every call goes through the binding's checks."""
    monkeypatch.setattr(la, "MARSHAL_PATH", str(tmp_path / "_marshal.so"))
    la._marshal.cache_clear()
    try:
        with pytest.warns(UserWarning, match="not built"):
            n = la._marshal()
        t = torch.zeros(4)
        assert n.adamw([t], [t], [t], [t], None) is None and n.states([t], [t]) is None and n.scratch(16, 0) is None
        assert n.cross_entropy(t, t, t, None, False) is None and n.cross_entropy_backward() is None
        with pytest.raises(ValueError):                # host tensors: the binding's own refusal
            la.linear_adamw([t], [t], [t.clone()], [t.clone()], lr=0.1, step=1)
    finally:
        la._marshal.cache_clear()
