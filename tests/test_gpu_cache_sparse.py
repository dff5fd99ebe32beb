"""Cache calls of a batch of fixed capacity, most of whose sequences have no rows."""
import numpy as np
import pytest
import torch

from jagged_hstu_attention_gb300 import binding as hb
import serving_testutil as su

pytestmark = pytest.mark.gpu


def _int32(v):
    return torch.tensor(np.ascontiguousarray(v), dtype=torch.int32, device="cuda")


def _call(B, rows_of, H, D, seed=0):
    """(cache, k, v, offsets, lens, table, counts): rows_of maps sequences to their new rows; one
    page for each sequence that has some."""
    counts = np.zeros(B, dtype=np.int64)
    for b, n in rows_of.items():
        counts[b] = n
    g = torch.Generator().manual_seed(seed)
    T = int(counts.sum())
    cache = hb.alloc_cache(len(rows_of) + 1, 64, H, D)
    table = np.full((B, 1), -1)
    for i, b in enumerate(sorted(rows_of)):
        table[b] = i + 1
    k, v = su.rows_of((T, H, D), g, torch.bfloat16), su.rows_of((T, H, D), g, torch.bfloat16)
    off = np.concatenate([[0], np.cumsum(counts)])
    return cache, k, v, _int32(off), _int32(np.zeros(B)), _int32(table), counts


@pytest.mark.parametrize("H,D", [(2, 32), (1, 128), (40, 64)])
@pytest.mark.parametrize("B,rows_of", [
    (4096, {0: 1}), (4096, {4095: 3}), (5000, {0: 2, 1: 1, 3: 1, 4: 5, 9: 1, 20: 1, 2047: 2, 4999: 7}),
    (1025, {b: 1 + b % 3 for b in range(0, 1025, 41)}), (70, {b: 1 for b in range(70)}), (1, {0: 50}), (2, {1: 1}),
    (100000, {0: 1, 99999: 1}),
])
def test_rows_find_their_sequences(B, rows_of, H, D):
    cache, k, v, off, lens, table, counts = _call(B, rows_of, H, D)
    ws = torch.empty(256, dtype=torch.uint8, device="cuda")
    hb.cache_write(cache, k, v, off, lens, table, ws=ws)
    assert hb.device_status(ws) == hb.HSTU_OK
    at = 0
    for i, b in enumerate(sorted(rows_of)):
        n = rows_of[b]
        assert torch.equal(cache.k[i + 1, :, :n].transpose(0, 1), k[at:at + n])
        assert torch.equal(cache.v[i + 1, :, :n].transpose(0, 1), v[at:at + n])
        at += n
    k2, v2 = hb.cache_read(cache, off, k.shape[0], table, ws=ws)
    assert hb.device_status(ws) == hb.HSTU_OK
    assert torch.equal(k2, k) and torch.equal(v2, v)


@pytest.mark.parametrize("rows_of", [{0: 1}, {0: 1, (1 << 18) - 1: 1}])
def test_empty_sequences_cost_a_search_not_a_walk(rows_of):
    """A quarter of a million sequences, one or two rows: a walk over them takes
    milliseconds (each step a load that waits for the one before), a search a few
    microseconds."""
    cache, k, v, off, lens, table, _ = _call(1 << 18, rows_of, 1, 128)

    def best(fn):
        times = []
        for _ in range(5):
            e = [torch.cuda.Event(enable_timing=True) for _ in range(2)]
            e[0].record()
            fn()
            e[1].record()
            torch.cuda.synchronize()
            times.append(e[0].elapsed_time(e[1]))
        return min(times)

    assert best(lambda: hb.cache_write(cache, k, v, off, lens, table)) < 0.5
    assert best(lambda: hb.cache_read(cache, off, k.shape[0], table)) < 0.5
