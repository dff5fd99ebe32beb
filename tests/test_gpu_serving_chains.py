"""Serving calls that follow one another on a stream with nothing between them:
each kernel begins while the one before it ends, and reads what that one wrote."""
import numpy as np
import pytest
import torch

from jagged_hstu_attention_gb300 import binding as hb
import serving_testutil as su

pytestmark = pytest.mark.gpu


def _int32(v):
    return torch.tensor(np.ascontiguousarray(v), dtype=torch.int32, device="cuda")


def _offsets(counts):
    return _int32(np.concatenate([[0], np.cumsum(counts)]))


@pytest.mark.parametrize("dtype,quantised", [(torch.bfloat16, True), (torch.bfloat16, False), (torch.float16, True)])
@pytest.mark.parametrize("counts", [[1, 1, 1, 1], [3, 0, 12, 5], [40, 17, 9, 33]])
def test_rows_written_by_the_kernel_before(counts, dtype, quantised):
    """The same slots are written again and again, and read by the next kernel:
    rotation to candidates, writer to reader, writer to attention."""
    lens, H, D, N, rounds = [300, 41, 777, 128], 2, 128, 800, 200
    pages = su.Pages(lens, H, D, D, 32, dtype, quantised)
    g = torch.Generator().manual_seed(sum(counts))
    T, C = sum(lens), sum(counts)
    off, zero, cand = _offsets(lens), _int32([0] * 4), _offsets(counts)
    pos, table = _int32(np.arange(C) * 7), hb.rope_table(D)
    sets = [[su.rows_of((n, H, D), g, dtype) for n in (T, T, C)] for _ in range(3)]

    def outputs():
        return [torch.empty((n, H, D), dtype=dtype, device="cuda") for n in (C, C, T, T)]

    def step(i, outs, between=lambda: None):
        k, v, q = sets[i % 3]
        ws = spaces[i % 2]
        hb.cache_write(pages.cache, k, v, off, zero, pages.d_table, rope=table)
        between()
        hb.rope(q, None, pos, table, outs=(outs[0], None))
        between()
        hb.fwd_paged(outs[0], pages.cache, pages.d_lens, pages.d_table, N, cand_offsets=cand, ws=ws, out=outs[1])
        between()
        hb.cache_write(pages.cache, v, k, off, zero, pages.d_table)
        between()
        hb.cache_read(pages.cache, off, T, pages.d_table, outs=(outs[2], outs[3]))
        between()

    spaces = [hb.paged_workspace(pages.cache, 4, C, N) for _ in range(2)]
    want = [outputs() for _ in range(3)]
    for i in range(3):
        step(i, want[i], torch.cuda.synchronize)
    got = [outputs() for _ in range(rounds)]
    torch.cuda.synchronize()
    for i in range(rounds):
        step(i, got[i])
    torch.cuda.synchronize()
    for i in range(rounds):
        for a, b in zip(got[i], want[i % 3]):
            assert torch.equal(a, b), i
