"""Embedding rows and the table's gradient against plain 64-bit forms."""
import numpy as np
import pytest
import torch

from jagged_hstu_attention_gb300 import binding as hb
import layer_testutil as lt

pytestmark = pytest.mark.gpu
BF, F16, F32 = torch.bfloat16, torch.float16, torch.float32


def _ids(T, V, seed, kind, dtype=torch.int32):
    r = np.random.default_rng(seed)
    if kind == "even":
        i = r.integers(0, V, T)
    elif kind == "skewed":
        i = np.minimum((V + 1.0) ** r.random(T) - 1, V - 1).astype(np.int64)
    elif kind == "one":
        i = np.full(T, V // 2)
    elif kind == "runs":  # two ids, runs that cross every chunk
        i = np.where(np.arange(T) < T // 3, 1 % V, V - 1)
    else:  # padding and ids past the table among the others
        i = r.integers(-2, V + 2, T)
    return torch.tensor(i, dtype=dtype, device="cuda")


def _bwd_case(T, V, D, dtype, grad, kind, idt=torch.int32, stride=None, seed=0, scale=1.25):
    wide = lt.randn((T, stride or D), dtype, seed + 1)
    dy, ids = wide[:, :D], _ids(T, V, seed, kind, idt)
    ws = hb.embed_workspace(T, V, D)
    got = hb.embed_bwd(dy, ids, V, scale, dtype=grad, ws=ws)
    ref, mag, n = lt.embed_bwd(lt.f64(dy), ids.cpu().numpy(), V, scale)
    # n terms, n - 1 sums and the scale: a rounding of 2^-24 of at most the magnitudes' sum each
    tol = (n[:, None] + 1) * lt.STEP32 * mag + lt.half_step(grad) * np.abs(ref) + lt.smallest_half_step(grad)
    assert lt.worst(lt.f64(got), ref, tol) <= 1.0
    bad = bool(((ids >= V)).any())
    assert hb.device_status(ws) == (5 if bad else 0)
    assert torch.equal(got, hb.embed_bwd(dy, ids, V, scale, dtype=grad))
    return dy, ids, got


@pytest.mark.parametrize("T,V,D", [(1, 1, 8), (1, 7, 512), (3, 5, 24), (64, 1000, 512), (257, 33, 520), (5, 3, 2056),
                                   (1000, 70000, 64)])
@pytest.mark.parametrize("table,dtype,idt", [(BF, BF, torch.int32), (F16, F16, torch.int64), (F32, BF, torch.int64),
                                             (F32, F16, torch.int32)])
def test_rows(T, V, D, table, dtype, idt):
    t = lt.randn((V, D), table, 3)
    ids = _ids(T, V, 4, "bad", idt)
    ws = torch.empty(256, dtype=torch.uint8, device="cuda")
    y = hb.embed(t, ids, 22.6, dtype=dtype, ws=ws)
    assert y.dtype == dtype and y.shape == (T, D)
    ref = lt.embed(lt.f64(t), ids.cpu().numpy(), 22.6)
    tol = (lt.half_step(dtype) + lt.STEP32 * 2) * np.abs(ref) + lt.smallest_half_step(dtype)
    assert lt.worst(lt.f64(y), ref, tol) <= 1.0
    assert hb.device_status(ws) == (5 if bool((ids >= V).any()) else 0)
    assert torch.equal(y, hb.embed(t, ids, 22.6, dtype=dtype))


def test_rows_enough_for_four_chunks_a_thread():
    T, V, D = 41000, 5003, 256
    t, ids = lt.randn((V, D), BF, 5), _ids(41000, 5003, 6, "skewed")
    y = hb.embed(t, ids)
    assert torch.equal(y, t[ids.long()])


@pytest.mark.parametrize("kind", ["even", "skewed", "one", "runs", "bad"])
@pytest.mark.parametrize("T,V,D", [(1, 3, 8), (15, 4, 16), (16, 4, 16), (17, 40, 8), (33, 2, 64), (600, 50, 72),
                                   (2000, 3000, 136), (1025, 513, 8)])
def test_gradient(kind, T, V, D):
    _bwd_case(T, V, D, BF, F32, kind)


@pytest.mark.parametrize("dtype,grad", [(F16, F32), (F16, F16), (BF, BF)])
@pytest.mark.parametrize("T,V,D,kind", [(700, 90, 64, "skewed"), (97, 1000, 520, "bad"), (64, 64, 8, "one")])
def test_gradient_types(dtype, grad, T, V, D, kind):
    _bwd_case(T, V, D, dtype, grad, kind, torch.int64, stride=D + 24)


@pytest.mark.parametrize("T,V,D", [(3000, 300000, 8), (2500, 20000000, 8), (500, 511, 2056), (80000, 7, 8),
                                   (4096, 4096, 16), (4097, 300, 1128), (4500, 300000, 8), (5000, 20000000, 8),
                                   (9000, 3, 520)])
def test_gradient_digits_and_wide_rows(T, V, D):
    """One block's sort and one to three digits, rows wider than a block, long runs that a block joins."""
    _bwd_case(T, V, D, BF, F32 if V < 1000000 else BF, "skewed")


def test_tables_past_two_to_the_32_values():
    """Rows whose offsets pass 32 bits, in values and in bytes."""
    V, D = 34000003, 128
    table = torch.zeros((V, D), dtype=BF, device="cuda")
    ids = torch.tensor([V - 1, 7, V - 2, V - 1, 20000001, V], dtype=torch.int64, device="cuda")
    rows = lt.randn((6, D), BF, 3)
    table[ids[:5]] = rows[:5]
    y = hb.embed(table, ids, 2.0)
    assert torch.equal(y[:5], 2 * table[ids[:5]]) and (y[5] == 0).all()
    del table
    d = hb.embed_bwd(rows, ids, V, dtype=BF)
    assert torch.equal(d[V - 1], (rows[0].float() + rows[3].float()).to(BF)) and torch.equal(d[V - 2], rows[2])
    assert torch.equal(d[20000001], rows[4]) and torch.equal(d[7], rows[1])
    d[ids[:5]] = 0
    assert int(torch.count_nonzero(d[V // 2:])) == 0 and int(torch.count_nonzero(d[:V // 2])) == 0


def test_gradient_is_that_of_the_sum():
    """Along a random direction of the table, against differences of the 64-bit sum."""
    T, V, D, scale = 400, 60, 40, 1.5
    dy, ids, got = _bwd_case(T, V, D, F16, F32, "skewed", seed=9, scale=scale)
    r = np.random.default_rng(1)
    table, v = r.standard_normal((V, D)), r.standard_normal((V, D))
    f = lambda e: (lt.embed(table + e * v, ids.cpu().numpy(), scale) * lt.f64(dy)).sum()  # noqa: E731
    slope = (f(0.5) - f(-0.5))  # linear in the table
    _, mag, n = lt.embed_bwd(lt.f64(dy), ids.cpu().numpy(), V, scale)
    assert abs((lt.f64(got) * v).sum() - slope) <= ((n[:, None] + 1) * lt.STEP32 * mag * np.abs(v)).sum() + 1e-9


@pytest.mark.parametrize("kind", ["even", "one", "bad"])
def test_accumulation_leaves_other_rows(kind):
    T, V, D = 300, 200, 48
    dy, ids = lt.randn((T, D), BF, 1), _ids(T, V, 2, kind)
    base = lt.randn((V, D), F32, 3)
    out = base.clone()
    assert hb.embed_bwd(dy, ids, V, 0.5, out=out, accumulate=True) is out
    ref, mag, n = lt.embed_bwd(lt.f64(dy), ids.cpu().numpy(), V, 0.5)
    ref += lt.f64(base)
    tol = (n[:, None] + 2) * lt.STEP32 * (mag + np.abs(lt.f64(base)))
    assert lt.worst(lt.f64(out), ref, np.where(n[:, None] > 0, tol, 0.0) + 1e-300) <= 1.0


def test_no_tokens():
    dy, ids = lt.randn((0, 16), BF, 1), torch.empty(0, dtype=torch.int32, device="cuda")
    out = torch.full((9, 16), 3.0, device="cuda")
    hb.embed_bwd(dy, ids, 9, out=out, accumulate=True)
    assert (out == 3.0).all()
    assert (hb.embed_bwd(dy, ids, 9) == 0).all() and hb.embed_bwd(dy, ids, 9, dtype=BF).dtype == BF
    assert hb.embed(lt.randn((9, 16), BF, 1), ids).shape == (0, 16)


def test_refusals():
    t, ids = lt.randn((10, 16), BF, 1), torch.zeros(4, dtype=torch.int32, device="cuda")
    dy = lt.randn((4, 16), BF, 2)
    for call, what in (
            (lambda: hb.embed(t, ids.float()), "ids"), (lambda: hb.embed(t, ids.cpu()), "ids"),
            (lambda: hb.embed(t.cpu(), ids), "table"), (lambda: hb.embed(t, ids.view(2, 2)), "ids"),
            (lambda: hb.embed(t, ids, dtype=F16), "table"), (lambda: hb.embed(t.double(), ids, dtype=BF), "table"),
            (lambda: hb.embed(t.t(), ids), "table"), (lambda: hb.embed(t, ids, out=dy[:3]), "out"),
            (lambda: hb.embed(t, ids, dtype=F32), "dtype"), (lambda: hb.embed(t, ids, ws=torch.empty(0, dtype=torch.uint8, device="cuda")), "ws"),
            (lambda: hb.embed_bwd(dy, ids[:3], 10), "dy"), (lambda: hb.embed_bwd(dy.float(), ids, 10), "dy"),
            (lambda: hb.embed_bwd(dy, ids, 0), "table"), (lambda: hb.embed_bwd(dy, ids, 10, accumulate=True), "accumulate"),
            (lambda: hb.embed_bwd(dy, ids, 10, out=torch.empty(9, 16, device="cuda")), "out"),
            (lambda: hb.embed_bwd(dy.t().contiguous().t(), ids, 10), "columns")):
        with pytest.raises(ValueError, match=what):
            call()
    for call, status in (
            (lambda: hb.embed(lt.randn((10, 12), BF, 1), ids), 2), (lambda: hb.embed_bwd(dy, ids, 10, dtype=F16), 2),
            (lambda: hb.embed_bwd(dy, ids, 10, dtype=BF, out=lt.randn((10, 16), BF, 1), accumulate=True), 2),
            (lambda: hb.embed(t, ids, out=t[:4]), 1), (lambda: hb.embed_bwd(dy, ids, 10, ws=torch.empty(512, dtype=torch.uint8, device="cuda")), 3),
            (lambda: hb.embed_bwd(dy, ids, 4, dtype=BF, out=dy), 1),
            (lambda: hb.embed_bwd(lt.randn((4, 20), BF, 1)[:, :16], ids, 10), 1)):
        with pytest.raises(hb.HstuError) as e:
            call()
        assert e.value.status == status
