"""Root-mean-square norms, their 8-bit output and gradients against plain 64-bit
forms."""
import numpy as np
import pytest
import torch

from jagged_hstu_attention_gb300 import binding as hb
import layer_testutil as lt

pytestmark = pytest.mark.gpu
BF, F16 = torch.bfloat16, torch.float16
# each way of laying a row out (threads a row, chunks a thread), at its ends
WIDTHS = [8, 64, 72, 128, 136, 256, 264, 512, 520, 1024, 1032, 2048, 2056, 4096, 4104, 8192]


def _inputs(T, D, dtype, residual, gate, seed=0, strided=False):
    pad = 40 if strided else 0
    x = lt.randn((T, D + pad), dtype, seed + 1)[:, :D]
    w = (1 + lt.randn((D,), torch.float32, seed + 2, 0.2)).to(dtype)
    r = lt.randn((T, 2 * D + pad), dtype, seed + 3, 3.0)[:, D:2 * D] if residual else None
    g = lt.randn((T, 4 * D), dtype, seed + 4)[:, :D] if gate else None
    return x, w, r, g


def _check_forward(x, w, r, g, eps=1e-6):
    dtype, D = x.dtype, x.shape[1]
    y, h, rstd = hb.rms_norm(x, w, residual=r, gate=g, eps=eps)
    if r is None:
        assert h is None
        kept = x
    else:
        assert torch.equal(h, (x.float() + r.float()).to(dtype))
        kept = h
    ref, ref_rstd = lt.norm(lt.f64(kept), lt.f64(w), None if g is None else lt.f64(g), eps)
    assert lt.worst(lt.f64(rstd), ref_rstd, lt.NORM_ERR * ref_rstd) <= 1.0
    tol = (lt.half_step(dtype) + lt.NORM_ERR) * np.abs(ref) + lt.smallest_half_step(dtype)
    assert lt.worst(lt.f64(y), ref, tol) <= 1.0
    return y, kept, rstd


@pytest.mark.parametrize("D", WIDTHS)
@pytest.mark.parametrize("dtype,T,residual,gate", [(BF, 5, True, False), (F16, 19, False, True), (BF, 1, True, True),
                                                   (F16, 34, False, False)])
def test_forward(D, dtype, T, residual, gate):
    x, w, r, g = _inputs(T, D, dtype, residual, gate, strided=T == 19)
    _check_forward(x, w, r, g)


@pytest.mark.parametrize("D", WIDTHS)
@pytest.mark.parametrize("dtype,T,gate,dh", [(BF, 37, False, True), (F16, 6, True, False), (BF, 1, True, True),
                                             (F16, 1300, False, False)])
def test_gradients(D, dtype, T, gate, dh):
    if D > 2056 and T > 1000:
        T = 700  # every block still takes two rows
    x, w, _, g = _inputs(T, D, dtype, False, gate, seed=7, strided=True)
    dy = lt.randn((T, D + 8), dtype, 20)[:, :D]
    e = lt.randn((T, D), dtype, 21) if dh else None
    _, _, rstd = hb.rms_norm(x, w, gate=g)
    dx, dw, dg = hb.rms_norm_bwd(dy, x, rstd, w, gate=g, dh=e)
    opt = lambda t: None if t is None else lt.f64(t)  # noqa: E731
    (rx, mag), (rw, wmag), rg = lt.norm_bwd(lt.f64(dy), lt.f64(x), lt.f64(rstd), lt.f64(w), opt(g), opt(e))
    half, tiny = lt.half_step(dtype), lt.smallest_half_step(dtype)
    # the mean's sum as rstd's; each value a few products: below 2^-18 of what is subtracted
    assert lt.worst(lt.f64(dx), rx, half * np.abs(rx) + lt.NORM_ERR * mag + tiny) <= 1.0
    # three products a term, and T sums
    assert lt.worst(lt.f64(dw), rw, half * np.abs(rw) + (T + 4) * lt.STEP32 * wmag + tiny) <= 1.0
    if gate:
        assert lt.worst(lt.f64(dg), rg, (half + 4 * lt.STEP32) * np.abs(rg) + tiny) <= 1.0
    else:
        assert dg is None
    again = hb.rms_norm_bwd(dy, x, rstd, w, gate=g, dh=e)
    assert torch.equal(dx, again[0]) and torch.equal(dw, again[1])


def test_gradients_are_those_of_the_sum():
    """Against central differences of the 64-bit norm along random directions."""
    T, D, eps = 9, 72, 1e-3
    x, w, _, g = _inputs(T, D, F16, False, True, seed=5)
    dy = lt.randn((T, D), F16, 6)
    _, _, rstd = hb.rms_norm(x, w, gate=g, eps=eps)
    dx, dw, dg = hb.rms_norm_bwd(dy, x, rstd, w, gate=g)
    r = np.random.default_rng(0)
    X, W, G, DY = (lt.f64(t) for t in (x, w, g, dy))
    (_, mag), (_, wmag), rg = lt.norm_bwd(DY, X, lt.f64(rstd), W, G)
    half = lt.half_step(F16)
    s = 1e-5
    for got, shape, f, bound in (
            (dx, X.shape, lambda v: lt.norm(X + v, W, G, eps)[0], half * np.abs(lt.f64(dx)) + lt.NORM_ERR * mag),
            (dw, W.shape, lambda v: lt.norm(X, W + v, G, eps)[0], half * np.abs(lt.f64(dw)) + 16 * lt.STEP32 * wmag),
            (dg, G.shape, lambda v: lt.norm(X, W, G + v, eps)[0], (half + 4 * lt.STEP32) * np.abs(rg))):
        v = r.standard_normal(shape)
        slope = ((f(s * v) - f(-s * v)) * DY).sum() / (2 * s)
        # differences: third derivatives times s^2, and 2^-53 of the sums over s
        slack = 1e-8 * np.abs(DY).sum() * 10
        assert abs((lt.f64(got) * v).sum() - slope) <= (1.01 * bound * np.abs(v)).sum() + slack


def _check_codes(codes, scale, ref, slack):
    """Codes and scales of rows `ref` known to a relative `slack`."""
    top = np.abs(ref).max(1)
    with np.errstate(divide="ignore"):
        e = np.where(top > 0, np.ceil(np.log2(np.maximum(top, 1e-300) / 448.0)), -127).clip(-127)
    near = np.abs(top / 448.0 / np.exp2(e) - 1) <= 4 * slack
    near |= np.abs(top / 224.0 / np.exp2(e) - 1) <= 4 * slack
    s = lt.scale_of(scale)
    assert ((s == np.exp2(e)) | near).all()
    got = lt.e4m3(codes) * s[:, None]
    # half a step of four bits, half the smallest step of the codes, and the rows' own error
    tol = (2.0 ** -4 + slack) * np.abs(ref) + 2.0 ** -10 * s[:, None]
    assert lt.worst(got, ref, tol) <= 1.0
    return got


@pytest.mark.parametrize("D", WIDTHS)
@pytest.mark.parametrize("dtype,T,residual,gate", [(BF, 33, True, False), (F16, 4, False, True), (BF, 1, False, False)])
def test_eight_bits(D, dtype, T, residual, gate):
    x, w, r, g = _inputs(T, D, dtype, residual, gate, seed=3)
    x = x * torch.logspace(-3, 3, T, device="cuda")[:, None].to(dtype)
    q, h, rstd = hb.rms_norm(x, w, residual=r, gate=g, quantise=True, want_rstd=True)
    kept = x if r is None else h
    ref, ref_rstd = lt.norm(lt.f64(kept), lt.f64(w), None if g is None else lt.f64(g))
    assert lt.worst(lt.f64(rstd), ref_rstd, lt.NORM_ERR * ref_rstd) <= 1.0
    _check_codes(q.codes, q.scale, ref, lt.NORM_ERR)
    q2, _, none = hb.rms_norm(x, w, residual=r, gate=g, quantise=True)
    assert none is None and torch.equal(q2.codes, q.codes) and torch.equal(q2.scale, q.scale)


@pytest.mark.parametrize("D", WIDTHS)
@pytest.mark.parametrize("dtype", [BF, F16])
def test_quantised_rows(D, dtype):
    T = 17
    x = lt.randn((T, D + 16), dtype, 8)[:, :D].clone()
    x[1] = 0
    x[2] *= 0.001
    x[3] = torch.finfo(dtype).max
    x[4, 0] = 448.0
    x[5] = torch.finfo(dtype).smallest_normal
    q = hb.quantise_rows(x)
    _check_codes(q.codes, q.scale, lt.f64(x), 0.0)
    assert (q.codes[1] == 0).all() and int(q.scale[1]) == 0


def test_values_that_are_not_finite_become_nan_codes():
    x = lt.randn((3, 136), BF, 1)
    x[0, 5], x[1, 9] = float("inf"), float("nan")
    q = hb.quantise_rows(x)
    v = q.codes.view(torch.float8_e4m3fn).float()
    assert torch.isnan(v[0, 5]) and torch.isnan(v[1, 9]) and int(torch.isnan(v).sum()) == 2
    clean = x.clone()
    clean[0, 5] = clean[1, 9] = 0
    assert torch.equal(q.scale, hb.quantise_rows(clean).scale)
    # a row that is not finite leaves its neighbours alone
    w = torch.ones(136, device="cuda", dtype=BF)
    y = hb.rms_norm(x, w)[0]
    assert torch.equal(y[2:], hb.rms_norm(x[2:], w)[0]) and not torch.isfinite(y[1].float()).any()


def test_zero_rows_and_large_rows():
    w = torch.ones(512, device="cuda", dtype=F16)
    x = torch.zeros((3, 512), device="cuda", dtype=F16)
    x[1] = 60000.0  # squares far past fp16
    x[2, 3] = 6e-8
    _check_forward(x, w, None, None)
    y, _, rstd = hb.rms_norm(x, w, eps=0.0)
    assert torch.isinf(rstd[0]) and (y[1] == 1).all()


def test_the_stream_updated_in_place():
    x, w, r, _ = _inputs(70, 520, BF, True, False)
    r = r.contiguous()
    y, h, _ = hb.rms_norm(x, w, residual=r)
    r2, x2 = r.clone(), x.contiguous().clone()
    y2, h2, _ = hb.rms_norm(x, w, residual=r2, outs=(None, r2))
    assert h2 is not None and torch.equal(r2, h) and torch.equal(y2, y)
    y3, _, none = hb.rms_norm(x2, w, residual=r, outs=(None, x2), want_rstd=False)
    assert none is None and torch.equal(x2, h) and torch.equal(y3, y)


def test_rows_past_two_to_the_31_values():
    T, D = 540000, 4096
    x, w = lt.randn((T, D), BF, 1), lt.randn((D,), BF, 2)
    y, h, rstd = hb.rms_norm(x, w, residual=x)
    dx, _, _ = hb.rms_norm_bwd(y, h, rstd, w)
    q = hb.quantise_rows(x)
    for r in (slice(0, 9), slice(T - 9, T)):
        a, b, c = hb.rms_norm(x[r], w, residual=x[r])
        assert torch.equal(y[r], a) and torch.equal(h[r], b) and torch.equal(rstd[r], c)
        assert torch.equal(dx[r], hb.rms_norm_bwd(a, b, c, w)[0])
        assert torch.equal(q.codes[r], hb.quantise_rows(x[r]).codes) and torch.equal(q.scale[r], hb.quantise_rows(x[r]).scale)


def test_no_rows():
    x, w = lt.randn((0, 64), BF, 1), lt.randn((64,), BF, 2)
    y, h, rstd = hb.rms_norm(x, w)
    assert y.shape == (0, 64) and rstd.shape == (0,)
    dx, dw, _ = hb.rms_norm_bwd(x, x, rstd, w)
    assert dx.shape == (0, 64) and (dw == 0).all()
    assert hb.quantise_rows(x).codes.shape == (0, 64)


def test_refusals():
    x, w, r, g = _inputs(4, 64, BF, True, True)
    rstd = torch.ones(4, device="cuda")
    for call, what in (
            (lambda: hb.rms_norm(x.float(), w), "x"), (lambda: hb.rms_norm(x, w.half()), "weight"),
            (lambda: hb.rms_norm(x, w[:32]), "weight"), (lambda: hb.rms_norm(x, w, residual=r[:3]), "residual"),
            (lambda: hb.rms_norm(x, w, gate=g.half()), "gate"), (lambda: hb.rms_norm(x[0], w), "x"),
            (lambda: hb.rms_norm(x, w, outs=(None, torch.empty_like(w.expand(4, 64)))), "outs"),
            (lambda: hb.rms_norm(x, w, quantise=True, outs=(torch.empty_like(x), None)), "outs"),
            (lambda: hb.rms_norm_bwd(x, x, rstd.double(), w), "rstd"), (lambda: hb.rms_norm_bwd(x, x[:2], rstd, w), "h"),
            (lambda: hb.rms_norm(x.cpu(), w), "x"), (lambda: hb.quantise_rows(x.float()), "x"),
            (lambda: hb.QuantisedRows(x, rstd), "codes")):
        with pytest.raises(ValueError, match=what):
            call()
    big = torch.zeros((2, 8200), device="cuda", dtype=BF)
    y = torch.empty_like(x)
    for call, status in (
            (lambda: hb.rms_norm(big, big[0].contiguous()), 2), (lambda: hb.rms_norm(big[:, :12], big[0, :12].contiguous()), 2),
            (lambda: hb.rms_norm(x, w, eps=-1.0), 1), (lambda: hb.rms_norm(x, w, eps=float("nan")), 1),
            (lambda: hb.rms_norm(x, w, outs=(x.contiguous().copy_(x), None)) and hb.rms_norm(y, w, outs=(y, None)), 1),
            (lambda: hb.rms_norm(x, w, residual=y, outs=(y, None)), 1),
            (lambda: hb.rms_norm_bwd(x, x, rstd, w, ws=torch.empty(256, dtype=torch.uint8, device="cuda")), 3)):
        with pytest.raises(hb.HstuError) as e:
            call()
        assert e.value.status == status


def test_codes_and_scales_outlive_each_other():
    """They share a piece of memory, which either keeps; a later call's lie elsewhere."""
    x = lt.randn((37, 48), BF, 5)
    q = hb.quantise_rows(x)
    codes, scale = q.codes.clone(), q.scale.clone()
    later = [hb.quantise_rows(-x) for _ in range(20)]
    assert torch.equal(q.codes, codes) and torch.equal(q.scale, scale)
    assert q.codes.is_contiguous() and q.scale.is_contiguous() and q.scale.data_ptr() % 16 == 0
    only_scale, only_codes = q.scale, later[0].codes
    want = only_codes.clone()
    del q, later
    filler = [torch.full((n,), 255, dtype=torch.uint8, device="cuda") for n in (100, 37, 2000, 4000)]
    assert torch.equal(only_scale, scale) and torch.equal(only_codes, want) and len(filler) == 4
