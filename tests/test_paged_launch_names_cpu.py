"""Every source that launches programmatic dependents, by any of the launchers'
names, is known here and holds no read-only load (test_paged_loads_cpu and
test_paged_chained_loads_cpu look for one name each, and for none with
clusters)."""
import os
import re

from exact_tiled_attention_fa2_gb300 import build as fa2_build

LAUNCHERS = re.compile(r"\blaunch_(dependent|dependent_clusters|chained)\s*\(")
ATTRIBUTE = "cudaLaunchAttributeProgrammaticStreamSerialization"
SOURCES = ["fa2_paged.cuh", "fa2_paged_cache.cu", "fa2_paged_fp8.cuh", "fa2_paged_fp8_cache.cu", "fa2_paged_shared.cuh"]
# what these kernels are made of beside their own source
SHARED = ["fa2_paged.h", "fa2_paged_fp8.h", "sm103_ptx.cuh", "sm103_ptx_fp8.cuh"]
READ_ONLY = re.compile(r"__ldg\s*\(|ld\.global(\.\w+)*\.nc|__restrict__")


def code(name):
    text = open(os.path.join(fa2_build.CSRC, name)).read()
    return re.sub(r"//[^\n]*|/\*.*?\*/", "", text, flags=re.S)


def test_launching_sources_are_known():
    files = sorted(n for n in os.listdir(fa2_build.CSRC) if n.endswith((".cu", ".cuh", ".h", ".cpp")))
    assert [n for n in files if LAUNCHERS.search(code(n)) and n != "fa2_paged.h"] == SOURCES
    # (the decoding merge's launch is its own: what it reads was complete before the kernel that lets it in began)
    assert [n for n in files if ATTRIBUTE in code(n)] == ["fa2_decode.cuh", "fa2_paged.h"]


def test_they_wait_and_hold_no_read_only_load():
    for name in SOURCES:
        assert "grid_dependency_wait()" in code(name), name
    for name in SOURCES + SHARED:
        assert READ_ONLY.findall(code(name)) == [], name


def test_a_read_only_load_is_found():
    assert READ_ONLY.findall("x = __ldg(p); asm(\"ld.global.v4.nc.u32\"); const int* __restrict__ q") != []
    assert LAUNCHERS.search("launch_dependent_clusters(kern, 2") and not LAUNCHERS.search("grid_launch_dependents()")
