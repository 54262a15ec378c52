"""The operators between the GEMVs without a GPU, where they had gone wrong: empty calls, the build."""
import os
import subprocess
import sys

import pytest

import quant_dequant_gemv_q4_b200 as qg
from quant_dequant_gemv_q4_b200 import build
from test_decode_ops_host import A, L, heads, norm_rope  # noqa: F401


def test_no_tokens_need_no_addresses(L):
    """T = 0 with a rotation: an empty array's address is null."""
    assert norm_rope(L, T=0, pos=None) == qg.QG_OK
    assert norm_rope(L, T=0, pos=None, q=heads(ptr=None), k=heads(ptr=None), qo=heads(ptr=None), ko=heads(ptr=None)) == qg.QG_OK
    assert norm_rope(L, T=0, pos=None, R=65) == qg.QG_ERR_SHAPE and norm_rope(L, T=0, pos=None, pairing=3) == qg.QG_ERR_VARIANT
    none = heads(ptr=None)
    assert L.qg_kv4_append(none, none, 0, 2, 128, None, 0.0, None, A, 64, 0, None, A, 4, 32, None) == qg.QG_OK
    assert L.qg_kv4_append(none, none, 0, 2, 128, None, 0.0, None, A, 64, 0, None, None, 0, 32, None) == qg.QG_OK
    assert L.qg_kv4_read(A, 4, 32, 2, 128, None, 0, none, none, None) == qg.QG_OK
    assert L.qg_attn_kv4(none, 0, 0, None, 0, 4, 2, 128, None, 0, 32, None, 0, None, 1.0, none, None, 0, None) == qg.QG_OK
    assert L.qg_sample(None, 0, 100, 100, 1, None, None, None, None, None, None, None, 0, None) == qg.QG_OK


def test_attention_device_error_needs_a_flag(L):
    assert L.qg_attn_kv4_device_error(None, None) == qg.QG_ERR_NULL


def test_status_texts_cover_the_operators(L):
    """A status that an operator between the GEMVs gives is not explained by the GEMVs' reasons alone."""
    text = {s: L.qg_status_string(s).decode() for s in range(11)}
    assert "workspace" in text[qg.QG_ERR_SCRATCH] and "element type" in text[qg.QG_ERR_FMT] and "eps" in text[qg.QG_ERR_RANGE]
    assert "pairing" in text[qg.QG_ERR_VARIANT] and "size" in text[qg.QG_ERR_SHAPE] and "cache" in text[qg.QG_ERR_ALIGN]
    assert len(set(text.values())) == 11


def test_the_library_is_built_without_torch(L, tmp_path):
    """Where torch is missing, build() leaves the binding out and makes libqg.so."""
    run = ("import sys; sys.modules['torch'] = None; from quant_dequant_gemv_q4_b200 import build; "
           f"build.BINDING = {str(tmp_path / 'qg_binding.so')!r}; print(build.build())")
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    done = subprocess.run([sys.executable, "-c", run], cwd=root, capture_output=True, text=True)
    assert done.returncode == 0, done.stderr
    assert done.stdout.strip() == build.LIB and os.listdir(tmp_path) == []


def test_the_binding_is_built_again_for_another_torch(L, tmp_path, monkeypatch):
    made = []

    def compiler(cmd):
        made.append(cmd)
        open(cmd[cmd.index("-o") + 1], "w").close()

    path = str(tmp_path / "qg_binding.so")
    monkeypatch.setattr(build, "BINDING", path)
    monkeypatch.setattr(build.subprocess, "check_call", compiler)
    build.build_binding()
    assert len(made) == 1 and build.binding_is_for(path) == build.built_for()
    build.build_binding()
    assert len(made) == 1
    monkeypatch.setattr(build, "built_for", lambda: "torch 99, cpython-0")
    build.build_binding()
    assert len(made) == 2 and build.binding_is_for(path) == "torch 99, cpython-0"
    os.remove(path + ".for")
    build.build_binding()
    assert len(made) == 3


def test_a_binding_of_another_torch_is_refused(L, monkeypatch):
    monkeypatch.setattr(qg, "_binding", None)
    qg._bound()
    monkeypatch.setattr(qg, "_binding", None)
    monkeypatch.setattr(build, "built_for", lambda: "torch 99, cpython-0")
    with pytest.raises(RuntimeError, match="build it again"):
        qg._bound()


def test_the_hashes_of_the_gemv_kernels_cover_what_they_include():
    """The captured DRAM traffic is reported only while the kernel's sources are those of the capture: its list of files
    has to hold every header that its files include."""
    import re

    import bench
    csrc = os.path.join(os.path.dirname(build.__file__), "csrc")
    for files, own in ((bench.ROWS_KERNEL_FILES, "qg_rows.cuh"), (bench.MMA_KERNEL_FILES, "qg_mma.cuh"), (bench.UMMA_KERNEL_FILES, "qg_umma.cuh")):
        assert own in files
        todo = [f for f in files if f.endswith(".cuh")]
        for f in todo:
            with open(os.path.join(csrc, f)) as h:
                for name in re.findall(r'#include "(qg_\w+\.cuh)"', h.read()):
                    assert name in files, (own, f, name)
