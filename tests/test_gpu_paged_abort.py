"""The way out of the candidate kernel's bounded waits, without a fault: the wait
for the scores of each sequence's last 64 candidates is made to give up at once
(hstu_attn_test_set_handoff_limit with 1 ns), with a product and copies in flight."""
import time

import numpy as np
import pytest
import torch

from jagged_hstu_attention_gb300 import binding as hb
import serving_testutil as su

pytestmark = pytest.mark.gpu

HSTU_ERR_TIMEOUT = 6


def _int32(v):
    return torch.tensor(np.ascontiguousarray(v), dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("dtype,quantised", [(torch.bfloat16, False), (torch.bfloat16, True), (torch.float16, True)])
def test_a_wait_runs_out_and_the_workspace_recovers(dtype, quantised):
    # one split, two, nothing cached (no product to wait for), one split and two groups of candidates
    lens, counts, H, D, N = [300, 700, 0, 40] * 20, [40, 130, 17, 100] * 20, 2, 128, 700
    pages = su.Pages(lens, H, D, D, 32, dtype, quantised)
    pages.fill(np.random.default_rng(6))
    at = np.concatenate([[0], np.cumsum(counts)])
    C = int(at[-1])
    q = su.rows_of((C, H, D), torch.Generator().manual_seed(6), dtype)
    off, ws = _int32(at), hb.paged_workspace(pages.cache, len(lens), C, N)

    def run():
        out = torch.full((C, H, D), 55.0, dtype=dtype, device="cuda")
        t0 = time.monotonic()
        hb.fwd_paged(q, pages.cache, pages.d_lens, pages.d_table, N, cand_offsets=off, ws=ws, out=out)
        return hb.device_status(ws), out, time.monotonic() - t0

    st, good, _ = run()
    assert st == hb.HSTU_OK
    for _ in range(3):
        hb.set_handoff_limit_for_tests(1)
        try:
            st, out, seconds = run()
        finally:
            hb.set_handoff_limit_for_tests(0)
        assert st == HSTU_ERR_TIMEOUT and seconds < 1.0  # far inside the 2 s of a wait
        for b in range(len(lens)):
            rows = slice(int(at[b]), int(at[b + 1]))
            done = {0: 0, 1: 0, 2: 17, 3: 64}[b % 4]  # candidates that were finished
            assert torch.equal(out[rows][:done], good[rows][:done]) and (out[rows][done:] == 55.0).all(), b
        st, out, _ = run()  # the same workspace, tensor memory free again
        assert st == hb.HSTU_OK and torch.equal(out, good)
