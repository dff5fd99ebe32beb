"""New outputs of the serving calls: rows that a call leaves out hold zeros, not
what the memory held before (another request's rows, say)."""
import numpy as np
import pytest
import torch

from jagged_hstu_attention_gb300 import binding as hb
import serving_testutil as su

pytestmark = pytest.mark.gpu


def _int32(v):
    return torch.tensor(np.ascontiguousarray(v), dtype=torch.int32, device="cuda")


def _offsets(counts):
    return np.concatenate([[0], np.cumsum(counts)])


def _used_memory(shape, dtype):
    """Leaves the allocator with blocks of that size that hold 55."""
    torch.cuda.synchronize()
    held = [torch.full(shape, 55.0, dtype=dtype, device="cuda") for _ in range(6)]
    del held


CASES = [
    # candidates a sequence, N, width: one split and several; few candidates, many, tensor memory
    ([1, 1, 1, 1], 600, 64), ([1, 1, 1, 1], 1500, 64), ([2, 0, 5, 1], 600, 32), ([2, 0, 20, 1], 1500, 64),
    ([20, 0, 70, 9], 600, 128), ([20, 0, 70, 9], 1500, 128), ([30, 40, 70, 9], 400, 64), ([30, 40, 70, 9], 1500, 64),
]


@pytest.mark.parametrize("dtype,quantised", [(torch.bfloat16, False), (torch.float16, True)])
@pytest.mark.parametrize("counts,N,D", CASES)
def test_candidates_of_bad_sequences(counts, N, D, dtype, quantised):
    lens, H = [min(N, n) for n in (350, 90, 1400, 17)], 3
    pages = su.Pages(lens, H, D, D, 32, dtype, quantised)
    pages.fill(np.random.default_rng(1))
    at = _offsets(counts)
    C = int(at[-1])
    q = su.rows_of((C, H, D), torch.Generator().manual_seed(1), dtype)
    single = counts == [1, 1, 1, 1]

    def run(lens=None, table=None, offsets=None):
        given = None if single and offsets is None else _int32(at if offsets is None else offsets)
        d_lens = pages.d_lens if lens is None else _int32(lens)
        table = pages.d_table if table is None else table
        _used_memory((C, H, D), dtype)
        return hb.fwd_paged(q, pages.cache, d_lens, table, N, cand_offsets=given)

    def left_out(out, which):
        for b in range(4):
            rows = slice(int(at[b]), int(at[b + 1]))
            if b in which:
                assert (out[rows] == 0).all(), b
            else:
                assert torch.equal(out[rows], good[rows]), b

    good = run()
    assert (good != 0).any(-1).all()
    for b in (0, 2):
        for entry in (0, (lens[b] - 1) // 32):
            for bad in (-1, pages.num_pages):
                table = pages.d_table.clone()
                table[b, entry] = bad
                left_out(run(table=table), [b])
    for bad in (-1, N + 1, 2**31 - 1):
        left_out(run(lens=[lens[0], lens[1], bad, lens[3]]), [2])
    o = [int(x) for x in at]
    for wrong in ([1] + o[1:], o[:4] + [C - 1], o[:4] + [C + 1], [-1] + o[1:]):
        assert (run(offsets=wrong) == 0).all()
    # out of order, or past the ends in between: rows hold results of a sequence that claims them, or zeros
    for wrong in ([0, C, 1, 0, C], [0, C + 9, 1, 2, C], [0, -5, o[2], o[3], C], [0, o[1], C + 1, -1, C],
                  [0, 2**31 - 1, -2**31, 0, C]):
        out = run(offsets=wrong)
        assert torch.isfinite(out).all() and not (out == 55.0).any()


def test_rows_of_a_timed_out_sequence():
    lens, counts, H, D, N = [300, 700, 40], [40, 130, 100], 2, 128, 700
    pages = su.Pages(lens, H, D, D, 32, torch.bfloat16, False)
    pages.fill(np.random.default_rng(6))
    q = su.rows_of((270, H, D), torch.Generator().manual_seed(6), torch.bfloat16)
    off = _int32(_offsets(counts))
    good = hb.fwd_paged(q, pages.cache, pages.d_lens, pages.d_table, N, cand_offsets=off)
    _used_memory((270, H, D), torch.bfloat16)
    hb.set_handoff_limit_for_tests(1)  # each sequence's last 64 candidates give up
    try:
        out = hb.fwd_paged(q, pages.cache, pages.d_lens, pages.d_table, N, cand_offsets=off)
        torch.cuda.synchronize()
    finally:
        hb.set_handoff_limit_for_tests(0)
    assert (out[:170] == 0).all() and torch.equal(out[170:234], good[170:234]) and (out[234:] == 0).all()


@pytest.mark.parametrize("quantised", [False, True])
@pytest.mark.parametrize("H,D,Dv", [(2, 32, 128), (5, 128, 64)])
@pytest.mark.parametrize("new", [[20, 10, 5], [3000, 10, 2500]])
def test_cached_rows_without_a_place(new, H, D, Dv, quantised):
    dtype = torch.bfloat16
    pages = su.Pages(new, H, D, Dv, 16, dtype, quantised)
    pages.fill(np.random.default_rng(2))
    T = sum(new)

    def read(table=None, offsets=None, rows=T):
        off = _int32(_offsets(new) if offsets is None else offsets)
        table = pages.d_table if table is None else table
        _used_memory((rows, H, D), dtype)
        _used_memory((rows, H, Dv), dtype)
        return hb.cache_read(pages.cache, off, rows, table)

    good = read()
    table = pages.d_table.clone()
    table[0, 1] = pages.num_pages
    for got, want in zip(read(table=table), good):
        assert (got[16:20] == 0).all()
        got[16:min(32, new[0])] = want[16:min(32, new[0])]
        assert torch.equal(got, want)
    for got, want in zip(read(rows=T + 7), good):  # a padded batch
        assert torch.equal(got[:T], want) and (got[T:] == 0).all()
    for got in read(offsets=[-3, -2, -1, 0]):
        assert (got == 0).all()
    for got in read(offsets=[0, -2, T + 9, T]):
        assert torch.isfinite(got).all() and not (got == 55.0).any()
