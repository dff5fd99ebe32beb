"""Sums of the linear maps' gradients: the bias gradient against sums of terms that no rounding
to 16 bits touched, and whole numbers, whose sums are exact."""
import numpy as np
import pytest
import torch

from jagged_hstu_attention_gb300 import binding as hb
import layer_testutil as lt

pytestmark = pytest.mark.gpu
BF, F16 = torch.bfloat16, torch.float16


@pytest.mark.parametrize("T,N", [(300, 264), (61, 2584), (1200, 8)])
@pytest.mark.parametrize("act,dtype", [("silu", BF), ("gelu", F16), ("gelu", BF), ("silu", F16)])
def test_bias_gradient_sums_before_the_rounding_to_16_bits(T, N, act, dtype):
    x, w = lt.randn((T, 16), dtype, 1), lt.randn((N, 16), dtype, 2)
    z, dy = lt.randn((T, N), dtype, 3, 2.0), lt.randn((T, N), dtype, 4)
    db = hb.linear_bwd(dy, z, x, w, act=act)[2]
    Z, DY = lt.f64(z), lt.f64(dy)
    g = DY * lt.act_grad(Z, act)
    eg = np.abs(DY) * lt.act_grad_err(Z, act) + 2 * lt.STEP32 * np.abs(g)
    # a thread's chain of rows (at most T / 152 + 4 of these sizes), halves of 256 threads, 152 / 32
    # chunks a warp, 32 warps: below 64 sums behind one another, an fp32 rounding each
    err = eg.sum(0) + 64 * lt.STEP32 * (np.abs(g) + eg).sum(0)
    ref = g.sum(0)
    tol = err + lt.half_step(dtype) * (np.abs(ref) + err) + lt.smallest_half_step(dtype)
    assert lt.worst(lt.f64(db), ref, tol) <= 1.0


def test_bias_gradient_of_terms_below_the_smallest_half():
    """Each term would round to zero in fp16; their sum does not."""
    T, N = 4096, 64
    x, w = lt.randn((T, 16), F16, 1), lt.randn((N, 16), F16, 2)
    dy = torch.full((T, N), 2.0 ** -24, dtype=F16, device="cuda")  # the smallest subnormal
    z = torch.full((T, N), -0.5, dtype=F16, device="cuda")
    db = lt.f64(hb.linear_bwd(dy, z, x, w, act="silu")[2])
    ref = T * 2.0 ** -24 * float(lt.act_grad(np.float64(-0.5), "silu"))  # 6.3e-5, a normal fp16 number
    assert np.abs(db - ref).max() <= 2.0 ** -11 * ref + 1e-5 * ref


def _whole(shape, top, dtype, seed, stride=None):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    wide = torch.randint(-top, top + 1, (shape[0], stride or shape[1]), generator=g, device="cuda").to(dtype)
    return wide[:, :shape[1]]


# rows, d_in, d_out: splits of dw's K from 1 to 65 and slices of the fold from 1 to 16, chunks of the bias
# gradient from 1 to 608, K blocks and tiles that are not full; few rows and many.
WHOLE = [(41000, 256, 136), (20000, 40, 8), (9001, 512, 200), (5000, 72, 1032), (4500, 520, 96), (4097, 504, 328),
         (81920, 64, 64), (61, 72, 2584), (700, 16, 1056), (64, 512, 2048), (1, 8, 8), (65, 4096, 264)]


@pytest.mark.parametrize("T,K,N", WHOLE)
@pytest.mark.parametrize("act,dtype", [("none", BF), ("relu", F16), ("relu", BF)])
def test_gradients_of_whole_numbers(T, K, N, act, dtype):
    """Every sum is below 2^24 in magnitude, term by term, and so exact in fp32 in any order: one
    rounding, the output's, is all that may differ, and a lost or doubled row shows."""
    x, w = _whole((T, K), 2, dtype, 1, K + 8), _whole((N, K), 2, dtype, 2)
    dy, z = _whole((T, N), 2, dtype, 3, N + 16), _whole((T, N), 1, dtype, 4)
    assert 4 * max(T, N) < 1 << 24
    dx, dw, db = hb.linear_bwd(dy, z, x, w, act=act)
    g = dy.double() * (z > 0) if act == "relu" else dy.double()
    assert torch.equal(dx, (g @ w.double()).to(dtype))
    assert torch.equal(dw, (g.t() @ x.double()).to(dtype))
    assert torch.equal(db, g.sum(0).to(dtype))


@pytest.mark.parametrize("T,K,N", [(1, 8, 8), (64, 512, 2048), (7, 8192, 264), (64, 4096, 1032), (300, 1032, 1000),
                                   (5000, 72, 1032), (1000, 8192, 520), (40000, 264, 136)])
@pytest.mark.parametrize("dtype", [BF, F16])
def test_products_of_whole_numbers(T, K, N, dtype):
    x, w, b, r = _whole((T, K), 2, dtype, 5, K + 8), _whole((N, K), 2, dtype, 6), _whole((1, N), 9, dtype, 7)[0], \
        _whole((T, N), 9, dtype, 8, N + 8)
    y, z = hb.linear(x, w, bias=b, act="relu", residual=r, want_z=True)
    ref = x.double() @ w.double().t() + b.double()
    assert torch.equal(z, ref.to(dtype)) and torch.equal(y, (ref.clamp(min=0) + r.double()).to(dtype))


def test_gradients_of_whole_numbers_past_two_to_the_31_values():
    """With an activation, whose g and column sums have offsets past 32 bits too."""
    T, K, N = 1100000, 16, 2048
    g = torch.Generator(device="cuda").manual_seed(9)
    dy = torch.randint(-1, 2, (T, N), generator=g, device="cuda", dtype=torch.int8).to(BF)
    z = torch.randint(-1, 2, (T, N), generator=g, device="cuda", dtype=torch.int8).to(BF)
    x, w = _whole((T, K), 1, BF, 10), _whole((N, K), 2, BF, 11)
    dx, dw, db = hb.linear_bwd(dy, z, x, w, act="relu")
    sums, products = torch.zeros(N, dtype=torch.float64, device="cuda"), torch.zeros((N, K), dtype=torch.float64, device="cuda")
    for t in range(0, T, 100000):
        part = slice(t, t + 100000)
        d = dy[part].double() * (z[part] > 0)
        sums += d.sum(0)
        products += d.t() @ x[part].double()
        assert torch.equal(dx[part], (d @ w.double()).to(BF))
    assert torch.equal(db, sums.to(BF)) and torch.equal(dw, products.to(BF))


@pytest.mark.parametrize("T,K,N", [(1, 16, 8), (64, 512, 2048), (7, 8192, 264), (300, 1040, 1000), (1000, 8192, 520),
                                   (20000, 2064, 136)])
def test_eight_bit_products_of_whole_numbers(T, K, N):
    """Under scales of powers of two that differ from row to row."""
    codes = lambda shape, seed: _whole(shape, 8, F16, seed).to(torch.float8_e4m3fn).view(torch.uint8)  # noqa: E731
    g = torch.Generator(device="cuda").manual_seed(12)
    scale = lambda n: torch.randint(120, 135, (n,), generator=g, device="cuda", dtype=torch.uint8)  # noqa: E731
    qx, qw = hb.QuantisedRows(codes((T, K), 13), scale(T)), hb.QuantisedRows(codes((N, K), 14), scale(N))
    value = lambda q: q.codes.view(torch.float8_e4m3fn).double() * torch.exp2(q.scale.double() - 127)[:, None]  # noqa: E731
    y, _ = hb.linear(qx, qw, dtype=BF)
    assert torch.equal(y, (value(qx) @ value(qw).t()).float().to(BF))
