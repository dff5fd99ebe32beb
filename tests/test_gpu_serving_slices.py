"""Outputs in other slices of the rows that hold the inputs: between each other,
without sharing memory."""
import pytest
import torch

from jagged_hstu_attention_gb300 import binding as hb
import serving_testutil as su

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T", [1, 2, 77])
def test_rotation_into_slices_of_the_same_rows(T):
    H, D = 4, 64
    w = H * D
    rows = su.rows_of((T, 6 * w), torch.Generator().manual_seed(3), torch.bfloat16)
    part = lambda i: rows[:, i * w:(i + 1) * w].unflatten(1, (H, D))  # noqa: E731
    pos = torch.arange(T, dtype=torch.int32, device="cuda") * 3
    table = hb.rope_table(D)
    want_q, want_k = hb.rope(part(2).contiguous(), part(4).contiguous(), pos, table)
    before = rows.clone()
    hb.rope(part(2), part(4), pos, table, outs=(part(1), part(5)))
    assert torch.equal(part(1), want_q) and torch.equal(part(5), want_k)
    for i in (0, 2, 3, 4):
        assert torch.equal(part(i), before[:, i * w:(i + 1) * w].unflatten(1, (H, D)))
    hb.rope(part(2), part(4), pos, table, outs=(part(2), part(0)))  # one of them in place
    assert torch.equal(part(2), want_q) and torch.equal(part(0), want_k)
    # one buffer, q's rows in front of its output's
    flat = torch.cat([before[:, 2 * w:3 * w].reshape(-1), torch.zeros(T * w, dtype=rows.dtype, device="cuda")])
    q, out = (x.view(T, H, D) for x in flat.split(T * w))
    hb.rope(q, None, pos, table, outs=(out, None))
    assert torch.equal(out, want_q)
    with pytest.raises(hb.HstuError):
        hb.rope(q, None, pos, table, outs=(flat[8:8 + T * w].view(T, H, D), None))


def test_a_reader_of_one_buffer():
    pages = su.Pages([33], 2, 64, 32, 16, torch.bfloat16, False)
    cache = pages.cache
    cache.k.normal_()
    cache.v.normal_()
    off = torch.tensor([0, 33], dtype=torch.int32, device="cuda")
    want = hb.cache_read(cache, off, 33, pages.d_table)
    flat = torch.empty(33 * 2 * 96, dtype=torch.bfloat16, device="cuda")
    outs = flat[:33 * 128].view(33, 2, 64), flat[33 * 128:].view(33, 2, 32)
    hb.cache_read(cache, off, 33, pages.d_table, outs=outs)
    assert all(torch.equal(a, b) for a, b in zip(outs, want))
    with pytest.raises(hb.HstuError):
        hb.cache_read(cache, off, 33, pages.d_table, outs=(outs[0], flat[:33 * 64].view(33, 2, 32)))
