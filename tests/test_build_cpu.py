"""What build() makes of a machine without torch or without a working host
compiler, and of another torch than the binding was built for.  The sources are
stand-ins in a temporary folder."""
import os
import subprocess
import sysconfig

import pytest

from exact_tiled_attention_fa2_gb300 import build as fa2_build

BINDING = """
#include <Python.h>
static PyModuleDef def = {PyModuleDef_HEAD_INIT, "_paged_binding", 0, -1, 0};
PyMODINIT_FUNC PyInit__paged_binding() { return PyModule_Create(&def); }
"""


@pytest.fixture
def tree(tmp_path, monkeypatch):
    """A package folder with one kernel-less CUDA source and a small binding."""
    (tmp_path / "csrc").mkdir()
    (tmp_path / "csrc" / "a.cu").write_text('extern "C" int fa2_version() { return 1; }\n')
    (tmp_path / "csrc" / "paged_binding.cpp").write_text(BINDING)
    for name, at in (("HERE", ""), ("CSRC", "csrc"), ("BUILD_DIR", "_build"), ("LIB_PATH", fa2_build.LIB_NAME)):
        monkeypatch.setattr(fa2_build, name, str(tmp_path / at))
    monkeypatch.setattr(fa2_build, "BINDING_PATH", str(tmp_path / os.path.basename(fa2_build.BINDING_PATH)))
    monkeypatch.setattr(fa2_build, "SOURCES", ["a.cu"])
    monkeypatch.setattr(fa2_build, "HEADERS", [])
    monkeypatch.setattr(fa2_build, "PUBLIC_HEADER", str(tmp_path / "csrc" / "a.cu"), raising=False)
    return tmp_path


def test_library_is_linked_where_the_binding_does_not_compile(tree):
    (tree / "csrc" / "paged_binding.cpp").write_text("#error no\n")
    with pytest.raises(RuntimeError, match="paged_binding.cpp"):
        fa2_build.build()
    assert os.path.exists(fa2_build.LIB_PATH)


def test_library_is_built_without_torch(tree, monkeypatch):
    monkeypatch.setitem(__import__("sys").modules, "torch", None)
    assert fa2_build.build() == fa2_build.LIB_PATH
    assert os.path.exists(fa2_build.LIB_PATH) and not os.path.exists(fa2_build.BINDING_PATH)


def test_binding_carries_its_abi_and_follows_torch(tree, monkeypatch):
    import torch
    assert fa2_build.BINDING_PATH.endswith("_paged_binding" + sysconfig.get_config_var("EXT_SUFFIX"))
    calls = []
    popen = subprocess.Popen   # subprocess.run goes through it too
    monkeypatch.setattr(subprocess, "Popen", lambda cmd, **kw: (calls.append(cmd), popen(cmd, **kw))[1])

    def compiled():
        calls.clear()
        fa2_build.build()
        return [c for c in calls if c[0] == "g++"]

    assert len(compiled()) == 2          # compile, link
    assert compiled() == []              # nothing is stale
    monkeypatch.setattr(torch, "__version__", "0.0.0")
    assert len(compiled()) == 2
    assert compiled() == []
