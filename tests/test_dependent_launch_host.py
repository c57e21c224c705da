"""Kernels that may start before the launch before them has ended (kda_dependent.cuh) read what that launch wrote: by ordinary
loads behind the wait, never by read-only ones, which are allowed to pass it."""
import glob
import os
import re

import pytest

from kda_recurrent_gb300 import build as kbuild


def overlapping_sources():
    """The sources whose kernels are launched so, and the headers of the library that they include."""
    found = [f for f in kbuild.sources() if '"kda_dependent.cuh"' in open(f).read()]
    todo = list(found)
    while todo:
        for name in re.findall(r'#include "(\w+\.cuh)"', open(todo.pop()).read()):
            path = os.path.join(kbuild.CSRC, name)
            if path not in found:
                found.append(path)
                todo.append(path)
    return sorted(os.path.basename(f) for f in found)


def test_the_sources_are_found():
    found = overlapping_sources()
    assert {"kda_attn_prefix.cu", "kda_attn_stream.cuh", "kda_page_resize.cu", "kda_qk_rope.cu", "kda_linear_decode.cu"} <= set(found)
    assert len(found) < len(glob.glob(os.path.join(kbuild.CSRC, "*.cu*")))


@pytest.mark.parametrize("name", overlapping_sources())
def test_no_read_only_loads(name):
    code = re.sub(r"//[^\n]*", "", open(os.path.join(kbuild.CSRC, name)).read())
    assert not re.findall(r"__ldg|ld\.global\.nc|__restrict__", code)
