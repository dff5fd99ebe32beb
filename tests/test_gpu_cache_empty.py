"""Cache calls without rows: the offsets are checked all the same where there is
an error word to report to."""
import numpy as np
import pytest
import torch

from jagged_hstu_attention_gb300 import binding as hb

pytestmark = pytest.mark.gpu


def _int32(v):
    return torch.tensor(np.ascontiguousarray(v), dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("quantised", [False, True])
@pytest.mark.parametrize("offsets,status", [([0, 0, 0], 0), ([0, 0, 5], 5), ([-1, 0, 0], 5), ([0, 3, 0], 5)])
def test_no_rows(offsets, status, quantised):
    cache = hb.alloc_cache(3, 16, 2, 64, quantised=quantised)
    for t in (cache.k, cache.v):
        t.fill_(7)
    table, lens, off = _int32([[0], [1]]), _int32([3, 0]), _int32(offsets)
    rows = torch.empty((0, 2, 64), dtype=torch.bfloat16, device="cuda")
    ws = torch.full((256,), 255, dtype=torch.uint8, device="cuda")
    hb.cache_write(cache, rows, rows, off, lens, table, ws=ws)
    assert hb.device_status(ws) == status
    ws.fill_(255)
    k, v = hb.cache_read(cache, off, 0, table, ws=ws)
    assert hb.device_status(ws) == status and k.shape == v.shape == (0, 2, 64)
    hb.cache_write(cache, rows, rows, off, lens, table)  # nothing to report to
    hb.cache_read(cache, off, 0, table)
    torch.cuda.synchronize()
    assert (cache.k == 7).all() and (cache.v == 7).all()
