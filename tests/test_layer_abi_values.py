"""Values that the layer's row operators refuse before anything is enqueued, without a GPU."""
import ctypes

import pytest

from jagged_hstu_attention_gb300 import binding as hb
from jagged_hstu_attention_gb300 import build_ext

vp = ctypes.c_void_p


@pytest.fixture(scope="module")
def lib():
    build_ext.build()
    return hb.load()


def at(i):
    """An address of its own; never dereferenced: every call fails a host check."""
    return vp((i + 1) << 40)


@pytest.mark.parametrize("scale", [float("inf"), -float("inf"), float("nan")])
def test_embed_refuses_a_scale_that_is_not_finite(lib, scale):
    """It would make NaN of the zero rows of padding."""
    assert lib.hstu_attn_embed(at(0), 0, 100, 64, at(1), 4, 5, scale, at(2), 0, None, 0, None) == 1
