"""What the sources of kernels that begin before the kernel in front has ended may not do
(no GPU needed).

A kernel launched with programmatic stream serialization lives from before its
griddepcontrol.wait on, while the kernel in front may still write.  ld.global.nc, which
__ldg stands for and which the compiler may take for __restrict__ pointers to constants, is
for data that nothing changes during the kernel's life: such a kernel may not use it for
anything that work in front of it may write, so its source has no such load at all.
"""

import glob
import os
import re

import pytest

from long_context_causal_gqa_gb300 import build_lib

SOURCES = sorted(glob.glob(os.path.join(build_lib.CSRC, "*.cu")))


def code_of(path):
    """The source and the headers it includes from beside it, without comments."""
    seen, todo, text = set(), [path], ""
    while todo:
        p = todo.pop()
        if p in seen or not os.path.exists(p):
            continue
        seen.add(p)
        with open(p) as f:
            s = f.read()
        todo += [os.path.join(build_lib.CSRC, n) for n in re.findall(r'#include "([^"]+)"', s)]
        text += re.sub(r"//[^\n]*|/\*.*?\*/", "", s, flags=re.S)
    return text


OVERLAPPED = [p for p in SOURCES
              if "ProgrammaticStreamSerialization" in code_of(p) or "griddepcontrol.wait" in code_of(p)]


def test_the_overlapped_sources_are_found():
    names = {os.path.basename(p) for p in OVERLAPPED}
    assert {"tails.cu", "prefill.cu", "paged_e4m3.cu", "select_blocks.cu"} <= names


@pytest.mark.parametrize("path", OVERLAPPED, ids=os.path.basename)
def test_overlapped_kernels_have_no_read_only_loads(path):
    found = re.findall(r"__ldg\w*|ld\.global\.nc[\w.]*|\w+\.global\.nc[\w.]*|__restrict__",
                       code_of(path))
    assert not found


@pytest.mark.parametrize("path", OVERLAPPED, ids=os.path.basename)
def test_overlapped_kernels_wait(path):
    assert "griddepcontrol.wait" in code_of(path)
