"""Kernels that launch as programmatic dependents start while the kernel before
them may still write what they read.  A read-only (non-coherent) load asks for
data that is constant for the kernel's whole lifetime and may be moved across
the wait for that kernel, so the sources of such kernels hold none."""
import os
import re

import pytest

from exact_tiled_attention_fa2_gb300 import build as fa2_build

# launched through launch_dependent behind whatever the caller queued before
SOURCES = ["fa2_paged.cuh", "fa2_paged_cache.cu"]
READ_ONLY = re.compile(r"__ldg\s*\(|ld\.global(\.\w+)*\.nc|__restrict__")


def code(name):
    text = open(os.path.join(fa2_build.CSRC, name)).read()
    return re.sub(r"//[^\n]*|/\*.*?\*/", "", text, flags=re.S)


@pytest.mark.parametrize("name", SOURCES)
def test_dependent_kernels_hold_no_read_only_load(name):
    text = code(name)
    assert "launch_dependent(" in text and "grid_dependency_wait()" in text
    assert READ_ONLY.findall(text) == []


def test_every_source_that_launches_dependents_is_looked_at():
    found = [n for n in os.listdir(fa2_build.CSRC) if "launch_dependent(" in code(n) and n != "fa2_paged.h"]
    assert sorted(found) == sorted(SOURCES)
