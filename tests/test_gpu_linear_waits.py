"""Waits of the linear maps' kernels that give up: both CTAs of a pair end together, with nothing in
flight and well before the limit of a wait, and the next call is right."""
import time

import pytest
import torch

from jagged_hstu_attention_gb300 import binding as hb
import layer_testutil as lt

pytestmark = pytest.mark.gpu
BF, F16 = torch.bfloat16, torch.float16
TIMEOUT = 6


def _given_up(call, ws, times):
    """Runs `call` with a limit that ends its hand-off waits at once; returns the longest time of one, in s."""
    longest = 0.0
    hb.set_handoff_limit_for_tests(1)
    try:
        for _ in range(times):
            torch.cuda.synchronize()
            t0 = time.perf_counter()
            call()
            assert hb.device_status(ws) == TIMEOUT
            longest = max(longest, time.perf_counter() - t0)
    finally:
        hb.set_handoff_limit_for_tests(0)
    return longest


# More tiles than pairs of SMs, a K block or several to a tile, so that producers are stopped in all
# places of the ring; 128-column tiles too.
@pytest.mark.parametrize("T,K,N,codes", [(20000, 64, 1024, False), (8192, 512, 2048, False), (60000, 328, 120, False),
                                         (16000, 1040, 1024, True)])
def test_a_pair_that_gives_up_leaves_together(T, K, N, codes):
    x, w = lt.randn((T, K), BF, 1), lt.randn((N, K), BF, 2, K ** -0.5)
    if codes:
        x, w = hb.quantise_rows(x), hb.quantise_rows(w)
    ws = torch.empty(256, dtype=torch.uint8, device="cuda")
    want = hb.linear(x, w, act="silu", ws=ws)[0]
    assert hb.device_status(ws) == hb.HSTU_OK
    assert _given_up(lambda: hb.linear(x, w, act="silu", ws=ws), ws, 20) < 1.0  # a wait's limit is 2 s
    assert torch.equal(want, hb.linear(x, w, act="silu", ws=ws)[0]) and hb.device_status(ws) == hb.HSTU_OK


def test_a_backward_that_gives_up_leaves_together():
    T, K, N = 45000, 640, 64
    x, w, dy = lt.randn((T, K), F16, 1), lt.randn((N, K), F16, 2, K ** -0.5), lt.randn((T, N), F16, 3)
    ws = hb.linear_workspace(T, K, N)
    call = lambda: hb.linear_bwd(dy, None, x, w, ws=ws)  # noqa: E731
    want = call()
    assert hb.device_status(ws) == hb.HSTU_OK
    assert _given_up(call, ws, 20) < 1.0
    for a, b in zip(want, call()):
        assert torch.equal(a, b)
    assert hb.device_status(ws) == hb.HSTU_OK


# A CTA or several to a cluster, a K block to a CTA or more than it has stages for, tiles of 16, 32 and 64 rows.
@pytest.mark.parametrize("T,K,N,codes", [(1, 64, 8, False), (64, 512, 2048, False), (7, 8192, 264, False),
                                         (64, 4096, 4096, False), (33, 4096, 1032, True)])
def test_few_rows_that_give_up(T, K, N, codes):
    x, w = lt.randn((T, K), F16, 1), lt.randn((N, K), F16, 2, K ** -0.5)
    if codes:
        x, w = hb.quantise_rows(x), hb.quantise_rows(w)
    ws = torch.empty(256, dtype=torch.uint8, device="cuda")
    call = lambda: hb.linear(x, w, act="gelu", dtype=F16, ws=ws)[0]  # noqa: E731
    want = call()
    assert hb.device_status(ws) == hb.HSTU_OK
    assert _given_up(call, ws, 20) < 1.0
    assert torch.equal(want, call()) and hb.device_status(ws) == hb.HSTU_OK


@pytest.mark.parametrize("T,K,N", [(1, 64, 8), (64, 512, 2048), (40, 2048, 1000)])
def test_a_backward_of_few_rows_that_gives_up(T, K, N):
    x, w, dy = lt.randn((T, K), BF, 1), lt.randn((N, K), BF, 2, K ** -0.5), lt.randn((T, N), BF, 3)
    ws = hb.linear_workspace(T, K, N)
    call = lambda: hb.linear_bwd(dy, None, x, w, ws=ws)  # noqa: E731
    want = call()
    assert hb.device_status(ws) == hb.HSTU_OK
    assert _given_up(call, ws, 20) < 1.0
    for a, b in zip(want, call()):
        assert torch.equal(a, b)
    assert hb.device_status(ws) == hb.HSTU_OK
