"""Workspaces that a serving call cannot report its status in are refused."""
import pytest
import torch

from jagged_hstu_attention_gb300 import binding as hb
import serving_testutil as su

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("size", [0, 16, 255])
def test_a_workspace_without_room_for_the_error_word(size):
    pages = su.Pages([40], 2, 64, 64, 16, torch.bfloat16, False)
    ws = torch.empty(size, dtype=torch.uint8, device="cuda")
    rows = torch.zeros((40, 2, 64), dtype=torch.bfloat16, device="cuda")
    off = torch.tensor([0, 40], dtype=torch.int32, device="cuda")
    for call in (lambda: hb.cache_write(pages.cache, rows, rows, off, off[:1], pages.d_table, ws=ws),
                 lambda: hb.cache_read(pages.cache, off, 40, pages.d_table, ws=ws),
                 lambda: hb.fwd_paged(rows[:1], pages.cache, pages.d_lens, pages.d_table, 40, ws=ws)):
        with pytest.raises((ValueError, hb.HstuError)):
            call()
    assert torch.isnan(pages.cache.k).all()  # nothing was written
