"""Linear maps with their epilogues and gradients against plain 64-bit forms."""
import numpy as np
import pytest
import torch

from jagged_hstu_attention_gb300 import binding as hb
import layer_testutil as lt

pytestmark = pytest.mark.gpu
BF, F16 = torch.bfloat16, torch.float16

# rows, d_in, d_out: tails of the tiles and of the K blocks, single rows, several tiles a CTA
SIZES = [(1, 8, 8), (1, 512, 2048), (3, 24, 40), (64, 512, 264), (65, 72, 520), (127, 136, 64), (129, 64, 128),
         (256, 128, 256), (257, 200, 264), (300, 1032, 1000), (5000, 72, 1032)]


def _inputs(T, K, N, dtype, seed=0, pad=0):
    x = lt.randn((T, K + pad), dtype, seed + 1)[:, :K]
    w = lt.randn((N, K), dtype, seed + 2, K ** -0.5)
    b = lt.randn((N,), dtype, seed + 3, 0.5)
    r = lt.randn((T, N + pad), dtype, seed + 4)[:, :N]
    return x, w, b, r


def _forward_ref(x, w, b, r, act, err=0.0):
    """(z, its bound, y, its bound) before their rounding."""
    z = x @ w.T
    ez = lt.product_err(x, w.T) + err
    if b is not None:
        z = z + b
        ez = ez + lt.STEP32 * np.abs(z)
    y = lt.act(z, act)
    # |act'| is below 1.13
    ey = 1.13 * ez + lt.act_rel(z, act) * np.abs(y) + 1e-30
    if r is not None:
        y = y + r
        ey = ey + lt.STEP32 * np.abs(y)
    return z, ez, y, ey


def _round(dtype, v):
    return lt.half_step(dtype) * np.abs(v) + lt.smallest_half_step(dtype)


def _check_forward(x, w, b, r, act, want_z, dtype, got):
    opt = lambda t: None if t is None else lt.f64(t)  # noqa: E731
    z, ez, y, ey = _forward_ref(lt.f64(x), lt.f64(w), opt(b), opt(r), act)
    assert lt.worst(lt.f64(got[0]), y, 1.01 * ey + _round(dtype, np.abs(y) + ey)) <= 1.0
    if want_z:
        assert lt.worst(lt.f64(got[1]), z, ez + _round(dtype, np.abs(z) + ez)) <= 1.0
    else:
        assert got[1] is None


@pytest.mark.parametrize("T,K,N", SIZES)
@pytest.mark.parametrize("act,bias,residual,want_z,dtype", [
    ("none", False, False, False, BF), ("silu", True, False, True, BF), ("gelu", True, True, False, F16),
    ("relu", False, True, True, BF), ("none", True, True, False, F16)])
def test_forward(T, K, N, act, bias, residual, want_z, dtype):
    x, w, b, r = _inputs(T, K, N, dtype, pad=8 if residual else 0)
    b, r = b if bias else None, r if residual else None
    got = hb.linear(x, w, bias=b, act=act, residual=r, want_z=want_z)
    _check_forward(x, w, b, r, act, want_z, dtype, got)
    again = hb.linear(x, w, bias=b, act=act, residual=r, want_z=want_z)
    assert torch.equal(got[0], again[0])


@pytest.mark.parametrize("act,residual,want_z", [("silu", False, True), ("none", True, False), ("gelu", True, True)])
def test_many_tiles(act, residual, want_z):
    """More tiles than pairs of SMs: accumulators and staging buffers go around."""
    T, K, N = 5200, 72, 2088
    x, w, b, r = _inputs(T, K, N, BF, seed=5)
    r = r if residual else None
    got = hb.linear(x, w, bias=b, act=act, residual=r, want_z=want_z)
    _check_forward(x, w, b, r, act, want_z, BF, got)


@pytest.mark.parametrize("T,K,N", [(1, 16, 8), (1, 512, 2048), (33, 48, 264), (64, 512, 128), (200, 144, 520),
                                   (300, 1040, 1000), (2600, 80, 4104)])
@pytest.mark.parametrize("act,bias,residual,want_z,dtype", [
    ("none", False, False, False, BF), ("silu", True, False, True, F16), ("gelu", True, True, False, BF)])
def test_eight_bit_operands(T, K, N, act, bias, residual, want_z, dtype):
    x, w, b, r = _inputs(T, K, N, dtype, seed=3)
    b, r = b if bias else None, r if residual else None
    scale = torch.logspace(-2, 2, N, device="cuda")[:, None]
    qx, qw = hb.quantise_rows(x), hb.quantise_rows((w.float() * scale / scale.max()).to(dtype))
    got = hb.linear(qx, qw, bias=b, act=act, residual=r, want_z=want_z, dtype=dtype)
    X = lt.e4m3(qx.codes) * lt.scale_of(qx.scale)[:, None]
    W = lt.e4m3(qw.codes) * lt.scale_of(qw.scale)[:, None]
    opt = lambda t: None if t is None else lt.f64(t)  # noqa: E731
    z, ez, y, ey = _forward_ref(X, W, opt(b), opt(r), act)
    assert got[0].dtype == dtype
    assert lt.worst(lt.f64(got[0]), y, 1.01 * ey + _round(dtype, np.abs(y) + ey)) <= 1.0
    if want_z:
        assert lt.worst(lt.f64(got[1]), z, ez + _round(dtype, np.abs(z) + ez)) <= 1.0


def test_eight_bit_rows_of_a_wider_matrix():
    x, w, _, _ = _inputs(40, 64, 72, BF, seed=4)
    q, qw = hb.quantise_rows(x), hb.quantise_rows(w)
    wide = torch.zeros((40, 160), dtype=torch.uint8, device="cuda")
    wide[:, 48:112] = q.codes
    a = hb.linear(q, qw)[0]
    assert torch.equal(a, hb.linear(hb.QuantisedRows(wide[:, 48:112], q.scale), qw)[0])


@pytest.mark.parametrize("T,K,N", SIZES + [(5000, 264, 72), (20000, 40, 8), (9001, 512, 200), (41000, 256, 136),
                                           (4097, 504, 328), (4500, 520, 96), (61, 72, 2584), (700, 16, 1056)])
@pytest.mark.parametrize("act,dtype", [("none", BF), ("silu", BF), ("gelu", F16), ("relu", F16)])
def test_gradients(T, K, N, act, dtype):
    x, w, b, _ = _inputs(T, K, N, dtype, seed=11, pad=8)
    dy = lt.randn((T, N + 16), dtype, 12)[:, :N]
    _, z = hb.linear(x, w, bias=b, act=act, want_z=act != "none")
    dx, dw, db = hb.linear_bwd(dy, z, x, w, act=act)
    X, W, DY = lt.f64(x), lt.f64(w), lt.f64(dy)
    if act == "none":
        g, eg = DY, np.zeros_like(DY)
    else:
        Z = lt.f64(z)
        g = DY * lt.act_grad(Z, act)
        eg = np.abs(DY) * lt.act_grad_err(Z, act) + 2 * lt.STEP32 * np.abs(g)
        eg = eg + _round(dtype, np.abs(g) + eg)
    A = np.abs(g) + eg
    for got, ref, err in ((dx, g @ W, eg @ np.abs(W) + lt.product_err(A, W)),
                          (dw, g.T @ X, eg.T @ np.abs(X) + lt.product_err(A.T, X)),
                          (db, g.sum(0), eg.sum(0) + T * lt.STEP32 * A.sum(0))):
        assert lt.worst(lt.f64(got), ref, err + _round(dtype, np.abs(ref) + err)) <= 1.0
    again = hb.linear_bwd(dy, z, x, w, act=act, want_dbias=False)
    assert torch.equal(dx, again[0]) and torch.equal(dw, again[1]) and again[2] is None


@pytest.mark.parametrize("act", ["silu", "gelu"])
def test_gradients_are_those_of_the_sum(act):
    """Against central differences of the 64-bit map along random directions."""
    T, K, N = 23, 40, 24
    x, w, b, _ = _inputs(T, K, N, F16, seed=2)
    dy = lt.randn((T, N), F16, 3)
    _, z = hb.linear(x, w, bias=b, act=act, want_z=True)
    dx, dw, db = hb.linear_bwd(dy, z, x, w, act=act)
    X, W, B, DY = (lt.f64(t) for t in (x, w, b, dy))
    # z is kept in 16 bits: act'' is below 1.2, and g is rounded once more
    Z = X @ W.T + B
    eg = np.abs(DY) * (1.2 * lt.half_step(F16) * np.abs(Z) * 1.01 + 1e-5) + lt.half_step(F16) * 1.2 * np.abs(DY)
    s, r = 1e-5, np.random.default_rng(0)
    half = lt.half_step(F16)
    for got, shape, f, err in (
            (dx, X.shape, lambda v: lt.act((X + v) @ W.T + B, act), eg @ np.abs(W)),
            (dw, W.shape, lambda v: lt.act(X @ (W + v).T + B, act), eg.T @ np.abs(X)),
            (db, B.shape, lambda v: lt.act(X @ W.T + B + v, act), eg.sum(0))):
        v = r.standard_normal(shape)
        slope = ((f(s * v) - f(-s * v)) * DY).sum() / (2 * s)
        bound = ((err + half * np.abs(lt.f64(got)) * 1.01) * np.abs(v)).sum()
        assert abs((lt.f64(got) * v).sum() - slope) <= bound + 1e-6


def test_rows_past_two_to_the_31_values():
    """Inputs' and outputs' offsets past 32 bits: rows from both ends, and the same rows alone."""
    T, K, N = 1100000, 64, 2048
    x, w, b, _ = _inputs(T, K, N, BF, seed=5)
    y, _ = hb.linear(x, w, bias=b, act="silu")
    dx, dw, _ = hb.linear_bwd(y, None, x, w, want_dbias=False)
    for r in (slice(0, 300), slice(T - 300, T)):
        for got in (y[r], hb.linear(x[r], w, bias=b, act="silu")[0]):
            _check_forward(x[r], w, b, None, "silu", False, BF, (got, None))
        # few rows are summed in another order: each within the bound of its sums, and rounded
        Y, W = lt.f64(y[r]), lt.f64(w)
        ref = Y @ W
        err = lt.product_err(Y, W)
        for got in (dx[r], hb.linear_bwd(y[r], None, x[r], w, want_dbias=False)[0]):
            assert lt.worst(lt.f64(got), ref, err + _round(BF, np.abs(ref) + err)) <= 1.0


def test_values_that_are_not_finite_stay_in_their_row():
    x, w, b, _ = _inputs(40, 64, 72, BF, seed=6)
    clean = hb.linear(x, w, bias=b, act="silu")[0]
    x = x.clone()
    x[7, 3], x[30, 1] = float("nan"), float("inf")
    y = hb.linear(x, w, bias=b, act="silu")[0]
    rows = torch.ones(40, dtype=torch.bool, device="cuda")
    rows[7] = rows[30] = False
    assert torch.equal(y[rows], clean[rows]) and torch.isnan(y[7]).all()


@pytest.mark.parametrize("T", [5, 200, 1500])
@pytest.mark.parametrize("act", ["none", "silu", "gelu", "relu"])
def test_extreme_columns(T, act):
    """Outputs whose bias is the type's lowest or largest value, an infinity or NaN: the activation's
    limits there, and nothing else changes."""
    x, w, b, _ = _inputs(T, 64, 264, BF, seed=8)
    clean = hb.linear(x, w, bias=b, act=act)[0]
    low, top = torch.finfo(BF).min, torch.finfo(BF).max
    at, values = [3, 64, 100, 131, 200, 263], [low, float("inf"), float("nan"), -1e4, -1e20, 3e38]
    b = b.clone()
    b[at] = torch.tensor(values, dtype=BF, device="cuda")
    y, z = hb.linear(x, w, bias=b, act=act, want_z=True)
    rest = torch.ones(264, dtype=torch.bool, device="cuda")
    rest[at] = False
    assert torch.equal(y[:, rest], clean[:, rest])
    assert torch.isnan(y[:, 100]).all() and torch.isinf(y[:, 64]).all() and (y[:, 263].float() >= 2.9e38).all()
    if act != "none":
        assert (y[:, [3, 131, 200]].float().abs() <= 6e-17).all()
    dy = lt.randn((T, 264), BF, 9)
    dx, dw, db = hb.linear_bwd(dy, z, x, w, act=act)
    # the gradient of a column that is not finite stays with it
    assert torch.isfinite(dw[rest].float()).all() and torch.isfinite(db[rest].float()).all()
    if act != "none":
        assert (dw[[3, 131, 200]].float().abs() <= 1e-12 * T).all()
        ones = hb.linear_bwd(dy, z, x, w)[2]  # slope 1 far above
        assert torch.equal(db[263], ones[263])


def test_no_rows():
    x, w, b, _ = _inputs(0, 64, 72, BF)
    y, z = hb.linear(x, w, bias=b, act="silu", want_z=True)
    assert y.shape == z.shape == (0, 72)
    dx, dw, db = hb.linear_bwd(y, z, x, w, act="silu")
    assert dx.shape == (0, 64) and (dw == 0).all() and (db == 0).all()


def test_a_wait_that_gives_up_is_reported():
    x, w, b, _ = _inputs(4096, 64, 4096, BF)
    ws = torch.empty(256, dtype=torch.uint8, device="cuda")
    want = hb.linear(x, w, bias=b, ws=ws)[0]
    assert hb.device_status(ws) == hb.HSTU_OK
    hb.set_handoff_limit_for_tests(1)
    try:
        hb.linear(x, w, bias=b, ws=ws)
        assert hb.device_status(ws) == 6
    finally:
        hb.set_handoff_limit_for_tests(0)
    assert torch.equal(want, hb.linear(x, w, bias=b, ws=ws)[0]) and hb.device_status(ws) == hb.HSTU_OK


def test_a_wait_of_the_backward_that_gives_up_is_reported():
    T, K, N = 45000, 640, 64
    x, w, b, _ = _inputs(T, K, N, BF)
    dy, z = lt.randn((T, N), BF, 1), lt.randn((T, N), BF, 2)
    ws = hb.linear_workspace(T, K, N, "silu")
    want = hb.linear_bwd(dy, z, x, w, act="silu", ws=ws)
    assert hb.device_status(ws) == hb.HSTU_OK
    hb.set_handoff_limit_for_tests(1)
    try:
        hb.linear_bwd(dy, z, x, w, act="silu", ws=ws)
        assert hb.device_status(ws) == 6
    finally:
        hb.set_handoff_limit_for_tests(0)
    for a, c in zip(want, hb.linear_bwd(dy, z, x, w, act="silu", ws=ws)):
        assert torch.equal(a, c)
    assert hb.device_status(ws) == hb.HSTU_OK


def test_refusals():
    x, w, b, r = _inputs(4, 64, 72, BF)
    q, qw = hb.quantise_rows(x), hb.quantise_rows(w)
    for call, what in (
            (lambda: hb.linear(x, w, act="tanh"), "act"), (lambda: hb.linear(x.half(), w), "w"),
            (lambda: hb.linear(x, w[:, :32]), "w"), (lambda: hb.linear(x, w, bias=b[:8]), "bias"),
            (lambda: hb.linear(x, w, residual=r[:2]), "residual"), (lambda: hb.linear(q, w), "quantised"),
            (lambda: hb.linear(x, qw), "quantised"), (lambda: hb.linear(x, w, out=x), "out"),
            (lambda: hb.linear(x, w, dtype=F16), "x"), (lambda: hb.linear(q, qw, dtype=torch.float32), "dtype"),
            (lambda: hb.linear(q, qw, bias=b, dtype=F16), "bias"), (lambda: hb.linear(x.cpu(), w), "x"),
            (lambda: hb.linear_bwd(r, None, x, w, act="silu"), "z"), (lambda: hb.linear_bwd(r[:3], None, x, w), "x"),
            (lambda: hb.linear_bwd(r.half(), None, x, w), "x")):
        with pytest.raises(ValueError, match=what):
            call()
    y = torch.empty((4, 72), device="cuda", dtype=BF)
    sq = lt.randn((64, 64), BF, 1)
    for call, status in (
            (lambda: hb.linear(x[:, :12], w[:, :12].contiguous()), 2), (lambda: hb.linear(x, w[:70]), 2),
            (lambda: hb.linear(x, w, residual=y, out=y), 1), (lambda: hb.linear(sq, w[:64], out=sq), 1),
            (lambda: hb.linear(lt.randn((4, 68), BF, 1)[:, :64], w), 1),
            (lambda: hb.linear(hb.QuantisedRows(q.codes[:, :24].contiguous(), q.scale), hb.QuantisedRows(qw.codes[:, :24].contiguous(), qw.scale)), 2),
            (lambda: hb.linear(x, w, ws=torch.empty(128, dtype=torch.uint8, device="cuda")), 3),
            (lambda: hb.linear_bwd(y, None, x, w, ws=torch.empty(256, dtype=torch.uint8, device="cuda")), 3)):
        with pytest.raises(hb.HstuError) as e:
            call()
        assert e.value.status == status
