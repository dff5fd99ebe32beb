"""Rotary positions on the GPU against the 64-bit form."""
import numpy as np
import pytest
import torch

from jagged_hstu_attention_gb300 import binding as hb
import serving_testutil as su

pytestmark = pytest.mark.gpu


def _positions(T, rng, far):
    p = rng.integers(0, far, size=T)
    p[:1] = far - 1
    if T > 2:
        p[1], p[2] = 0, -3
    return p.astype(np.int32)


def _check(x, got, pos, f, m, interleaved, backward, dtype):
    want = su.rotate(su.f64(x), pos, f, m, interleaved, backward)
    tol = su.rotate_slack(su.f64(x), f, m, interleaved) + su.half_step(dtype) * np.abs(want) * 1.01 + \
        su.smallest_half_step(dtype)
    assert np.all(np.abs(su.f64(got) - want) <= tol)
    assert torch.equal(got[..., 2 * len(f):], x[..., 2 * len(f):])  # columns past the rotated ones


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("T,H,D,R", [(1, 1, 32, 32), (1, 4, 128, 128), (7, 3, 64, 48), (129, 2, 128, 16),
                                     (1000, 5, 32, 16), (4097, 4, 128, 96), (333, 9, 64, 64),
                                     # enough tokens for four heads a thread
                                     (20011, 5, 32, 32), (10007, 6, 64, 48), (5003, 4, 128, 128)])
@pytest.mark.parametrize("interleaved", [False, True])
def test_rotation_and_its_transpose(T, H, D, R, interleaved, dtype):
    rng, g = np.random.default_rng(T + R), torch.Generator().manual_seed(T)
    q, k = su.rows_of((T, H, D), g, dtype), su.rows_of((T, H, D), g, dtype)
    pos = _positions(T, rng, 5000)
    table = hb.rope_table(R, interleaved=interleaved)
    f, m = su.frequencies(R)
    d_pos = torch.tensor(pos, device="cuda")
    for backward in (False, True):
        qo, ko = hb.rope(q, k, d_pos, table, backward=backward)
        _check(q, qo, pos, f, m, interleaved, backward, dtype)
        _check(k, ko, pos, f, m, interleaved, backward, dtype)


@pytest.mark.parametrize("scaling", ["linear", "ntk", "yarn"])
def test_scaled_frequencies_at_far_positions(scaling):
    T, H, D, R = 500, 2, 128, 128
    rng, g = np.random.default_rng(1), torch.Generator().manual_seed(1)
    q = su.rows_of((T, H, D), g, torch.float16)
    pos = _positions(T, rng, 1 << 24)
    table = hb.rope_table(R, base=50000.0, scaling=scaling, factor=16.0, original_len=4096)
    f, m = su.frequencies(R, 50000.0, scaling, 16.0, 4096)
    assert abs(table.magnitude - m) <= 2.0 ** -24 * m
    qo, ko = hb.rope(q, None, torch.tensor(pos, device="cuda"), table)
    assert ko is None
    # The 64-bit angles themselves are rounded: position 2^24 times a frequency
    # with 53 bits, on both sides, is 2^24 * 2^-52 radians.
    want = su.rotate(su.f64(q), pos, f, m)
    tol = su.rotate_slack(su.f64(q), f, m) + su.half_step(q.dtype) * np.abs(want) * 1.01 + 2.0 ** -24
    assert np.all(np.abs(su.f64(qo) - want) <= tol)


def test_slices_of_a_projection_and_in_place():
    T, H, D = 77, 4, 64
    g = torch.Generator().manual_seed(3)
    rows = su.rows_of((T, 4 * H * D), g, torch.bfloat16)
    before = rows.clone()
    q, k = (rows[:, i * H * D:(i + 1) * H * D].unflatten(1, (H, D)) for i in (2, 3))
    pos = torch.arange(T, dtype=torch.int32, device="cuda") * 3
    table = hb.rope_table(32, interleaved=True)
    qo, ko = hb.rope(q, k, pos, table)
    same_q, same_k = hb.rope(q.contiguous(), k.contiguous(), pos, table)
    assert torch.equal(qo, same_q) and torch.equal(ko, same_k)
    hb.rope(q, k, pos, table, outs=(q, k))
    assert torch.equal(q, qo) and torch.equal(k, ko)
    assert torch.equal(rows[:, :2 * H * D], before[:, :2 * H * D])  # u and v of the rows untouched


def test_no_rows():
    q = torch.empty((0, 2, 64), dtype=torch.bfloat16, device="cuda")
    qo, _ = hb.rope(q, None, torch.empty(0, dtype=torch.int32, device="cuda"), hb.rope_table(64))
    assert qo.shape == q.shape


def test_gradient_against_differences():
    """The backward pass is the gradient: w . J d, by central differences of the
    64-bit form along d, equals (J^T w) . d."""
    T, H, D, R = 20, 2, 64, 32
    rng, g = np.random.default_rng(2), torch.Generator().manual_seed(2)
    x, w = su.rows_of((T, H, D), g, torch.float16), su.rows_of((T, H, D), g, torch.float16)
    pos = _positions(T, rng, 900)
    f, m = su.frequencies(R, scaling="yarn", factor=8.0, original_len=512)
    table = hb.rope_table(R, scaling="yarn", factor=8.0, original_len=512)
    dx, _ = hb.rope(w, None, torch.tensor(pos, device="cuda"), table, backward=True)
    d = rng.standard_normal((T, H, D))
    eps = 1e-4
    up, down = (su.rotate(su.f64(x) + s * eps * d, pos, f, m) for s in (1, -1))
    slope = np.sum(su.f64(w) * (up - down) / (2 * eps))
    # dx carries one fp16 rounding an element (and the fp32 slack far below it)
    bound = np.sum(np.abs(d) * (su.half_step(x.dtype) * np.abs(su.f64(dx)) * 1.02 + 2.0 ** -19)) + 1e-6
    assert abs(np.sum(su.f64(dx) * d) - slope) <= bound


def test_values_that_are_not_finite_stay_in_their_pairs():
    T, H, D, R = 3, 1, 64, 32
    g = torch.Generator().manual_seed(5)
    q = su.rows_of((T, H, D), g, torch.bfloat16)
    clean, _ = hb.rope(q, None, torch.arange(T, dtype=torch.int32, device="cuda"), hb.rope_table(R))
    q[1, 0, 5] = float("inf")
    got, _ = hb.rope(q, None, torch.arange(T, dtype=torch.int32, device="cuda"), hb.rope_table(R))
    other = torch.ones_like(q, dtype=torch.bool)
    other[1, 0, 5] = other[1, 0, 5 + R // 2] = False
    assert torch.equal(got[other], clean[other])
    assert not torch.isfinite(got[1, 0, 5])


def test_captured_and_replayed():
    T, H, D = 64, 4, 128
    g = torch.Generator().manual_seed(6)
    q, k = su.rows_of((T, H, D), g, torch.bfloat16), su.rows_of((T, H, D), g, torch.bfloat16)
    pos = torch.zeros(T, dtype=torch.int32, device="cuda")
    table, outs = hb.rope_table(128), (torch.empty_like(q), torch.empty_like(k))
    hb.rope(q, k, pos, table, outs=outs)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        hb.rope(q, k, pos, table, outs=outs)
    for step in (5, 1234):
        pos.fill_(step)
        graph.replay()
        want, _ = hb.rope(q, k, pos, table)
        assert torch.equal(outs[0], want)
