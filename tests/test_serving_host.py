"""Serving kernels and calls as far as they can be checked without a GPU."""
import ctypes
import os
import re

import pytest

from jagged_hstu_attention_gb300 import binding as hb
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


@pytest.fixture(scope="module")
def lib():
    build_ext.build()
    return hb.load()


vp = ctypes.c_void_p
BASE = 1 << 24  # addresses are never dereferenced: every call fails a host check


def _rope(lib, q, qs, k, ks, qo, qos, ko, kos, tokens=8, H=4, D=64):
    table = hb.Rope(1 << 20, D, 0, 1.0)
    return lib.hstu_attn_rope(vp(q), qs, vp(k) if k else None, ks, vp(qo), qos, vp(ko) if ko else None, kos,
                              vp(1 << 20), tokens, H, D, 0, ctypes.byref(table), 0, None)


def test_rotation_refuses_outputs_that_share_memory(lib):
    row, far = 4 * 64 * 2, 1 << 22  # bytes of a row
    q, k, qo, ko = BASE, BASE + far, BASE + 2 * far, BASE + 3 * far
    for by in (16, row, 3 * row, 7 * row, 8 * row - 16):  # contiguous rows, moved by less than all of them
        for at in (-by, by):
            assert _rope(lib, q, 256, None, 0, q + at, 256, None, 0) == 1, at
            assert _rope(lib, q, 256, k, 256, qo, 256, k + at, 256) == 1, at
            assert _rope(lib, q, 256, k, 256, k + at, 256, ko, 256) == 1, at
            assert _rope(lib, q, 256, k, 256, qo, 256, q + at, 256) == 1, at
            assert _rope(lib, q, 256, k, 256, qo, 256, qo + at, 256) == 1, at
    # slices of rows of 1024: half a slice on, in the same and in other rows; in place but for k's gap
    for at in (row // 2, -row // 2, row * 4 + row // 2, row * 4 * 7 - 16, -row * 4 * 7 + 16):
        assert _rope(lib, q, 1024, None, 0, q + at, 1024, None, 0) == 1, at
    assert _rope(lib, q, 1024, q + row // 2, 1024, q, 1024, q + row // 2, 1024) == 1
    # other strides: a contiguous output inside the span of the slices
    assert _rope(lib, q, 1024, None, 0, q + row, 256, None, 0) == 1  # its rows run into the next slice
    assert _rope(lib, q, 256, None, 0, q - 1024, 512, None, 0) == 1


def test_attention_refuses_an_output_that_shares_memory(lib):
    cache = hb.Cache(1 << 20, 1 << 20, None, None, 10, 64, 4, 64, 32, 0, 0)
    f = vp(1 << 20)

    def paged(q, qs, o):
        return lib.hstu_attn_fwd_paged(vp(q), qs, vp(o), ctypes.byref(cache), f, 3, f, 4, f, 7, None, 0, 100, 0.1, f,
                                       1 << 20, 0, None)
    for at in (0, 16, 512, -16, -6 * 256, 6 * 512):
        assert paged(BASE, 256, BASE + at) == 1, at
    for at in (0, 256, 2048 + 256, -6 * 256 - 16, 2048 * 6):
        assert paged(BASE, 1024, BASE + at) == 1, at


def test_reading_back_refuses_outputs_that_share_memory(lib):
    cache = hb.Cache(1 << 20, 1 << 20, None, None, 10, 64, 4, 64, 32, 0, 0)
    f = vp(1 << 20)
    for name in ("hstu_attn_cache_read", "hstu_attn_cache_read_zeroed"):
        for at in (0, 16, 8 * 512, -16, -9 * 256 + 16, 9 * 512 - 16):
            assert getattr(lib, name)(ctypes.byref(cache), vp(BASE), vp(BASE + at), f, 3, 9, None, f, 4, None, 0,
                                      None) == 1, at
