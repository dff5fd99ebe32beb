"""8-bit pages at the ends of the rows' range."""
import numpy as np
import pytest
import torch

from jagged_hstu_attention_gb300 import binding as hb
import serving_testutil as su

pytestmark = pytest.mark.gpu


def _int32(v):
    return torch.tensor(np.ascontiguousarray(v), dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("D", [32, 64, 128])
@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
def test_the_largest_values_come_back_finite(dtype, D):
    """A code stands for at most 1 + 2^-4 times the value, which for the largest
    values is past the type's range; reading gives the type's largest then."""
    H, T, top = 2, 40, torch.finfo(dtype).max
    rng = np.random.default_rng(0)
    x = rng.uniform(-1, 1, size=(T, H, D))
    x[:, :, 0] = np.linspace(0.9, 1.0, T)[:, None]
    x[:, :, 1] = -np.linspace(0.9, 1.0, T)[:, None]
    k = torch.tensor(x * top).clamp(-top, top).to(dtype).cuda()
    k[-1, :, :2] = torch.tensor([top, -top], dtype=dtype)
    k[3, 0, 5], k[4, 1, 6] = float("nan"), float("inf")
    assert torch.isfinite(k).sum() == k.numel() - 2
    v = -k
    pages = su.Pages([T], H, D, D, 16, dtype, True)
    off = _int32([0, T])
    hb.cache_write(pages.cache, k, v, off, _int32([0]), pages.d_table)
    for x, got in zip((k, v), hb.cache_read(pages.cache, off, T, pages.d_table)):
        value, _ = su.quantise(su.f64(x))
        want = torch.tensor(np.clip(value, -top, top)).to(dtype)
        assert (np.abs(value) > top).any()  # the range is reached
        assert torch.equal(torch.isnan(got), ~torch.isfinite(x)) and not torch.isinf(got).any()
        fine = torch.isfinite(x).cpu()
        assert torch.equal(got.cpu()[fine], want[fine])


def test_rotated_rows_past_the_range():
    """A rotation takes a pair up to sqrt(2) times its larger value: codes hold
    that, and reading cuts it."""
    H, D, T, dtype = 1, 64, 33, torch.float16
    k = torch.full((T, H, D), 60000.0, dtype=dtype, device="cuda")
    pages = su.Pages([T], H, D, D, 16, dtype, True)
    off, table = _int32([0, T]), hb.rope_table(D)
    hb.cache_write(pages.cache, k, k, off, _int32([0]), pages.d_table, rope=table)
    got = su.f64(hb.cache_read(pages.cache, off, T, pages.d_table)[0])
    f, m = su.frequencies(D)
    want = su.rotate(su.f64(k), np.arange(T), f, m)
    assert (np.abs(want) > 70000).any() and np.isfinite(got).all()
    # half a step of a code, relative, or of the smallest normal one under the
    # scale (2^8 or 2^9); then the rotation's own error
    tol = 2.0 ** -4 * np.abs(want) + 2.0 ** -10 * 2.0 ** 9 + 1.1 * su.rotate_slack(su.f64(k), f, m)
    assert np.all(np.abs(got - np.clip(want, -65504, 65504)) <= tol)
