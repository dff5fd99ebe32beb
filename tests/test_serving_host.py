"""Serving kernels and calls as far as they can be checked without a GPU."""
import os
import re

import pytest

from jagged_hstu_attention_gb300 import build_ext

SERVING = ("rope.cu", "rope.cuh", "cache.cu", "cache.cuh", "paged.cu", "paged.cuh", "paged_many.cuh")


def _code(name):
    """A source without its comments."""
    with open(os.path.join(build_ext.CSRC, name)) as f:
        return re.sub(r"//[^\n]*", "", f.read())


@pytest.mark.parametrize("name", SERVING)
def test_chained_kernels_load_nothing_through_the_read_only_path(name):
    """They begin while the kernel before them still writes (cached rows, scales,
    rotated q): memory that is written while a kernel lives is not for
    non-coherent loads, which also need not stay behind the kernel's wait."""
    code = _code(name)
    for word in ("__ldg", "ld.global.nc", "__restrict__", "load_row_intervals"):
        assert word not in code, word


@pytest.mark.parametrize("name", SERVING)
def test_serving_kernels_wait_before_anything_else(name):
    """Every kernel of these files begins with chain(), before any load."""
    code = _code(name)
    for m in re.finditer(r"__global__ void[^{;]*\{", code):
        body = code[m.end():]
        before = body[:body.index("chain();")]
        assert not re.search(r"[\[(]\s*\*?p\.|\bp\.", before), before
