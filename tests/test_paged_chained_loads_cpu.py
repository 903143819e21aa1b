"""The sources that launch programmatic dependents by the name launch_chained
hold no read-only (non-coherent) load, which may be moved across the wait for
the kernel before (as the paged kernels' other sources, test_paged_loads_cpu)."""
import os
import re

from exact_tiled_attention_fa2_gb300 import build as fa2_build

READ_ONLY = re.compile(r"__ldg\s*\(|ld\.global(\.\w+)*\.nc|__restrict__")


def code(name):
    text = open(os.path.join(fa2_build.CSRC, name)).read()
    return re.sub(r"//[^\n]*|/\*.*?\*/", "", text, flags=re.S)


def test_chained_kernels_wait_and_hold_no_read_only_load():
    found = [n for n in os.listdir(fa2_build.CSRC) if "launch_chained(" in code(n) and n != "fa2_paged.h"]
    assert len(found) >= 2
    for name in found:
        text = code(name)
        assert "grid_dependency_wait()" in text, name
        assert READ_ONLY.findall(text) == [], name


def test_every_source_and_header_is_built():
    """The build lists every file under csrc/, so that none goes stale unseen."""
    named = set(fa2_build.SOURCES) | set(fa2_build.HEADERS) | {"fa2_internal.h", fa2_build.BINDING_SOURCE}
    here = {n for n in os.listdir(fa2_build.CSRC) if n.endswith((".cu", ".cuh", ".h", ".cpp"))}
    assert here == named
