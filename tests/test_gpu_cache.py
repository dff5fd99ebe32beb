"""The paged K/V cache on the GPU: written, quantised, read back."""
import numpy as np
import pytest
import torch

from jagged_hstu_attention_gb300 import binding as hb
import serving_testutil as su

pytestmark = pytest.mark.gpu


def _offsets(counts):
    return torch.tensor(np.concatenate([[0], np.cumsum(counts)]), dtype=torch.int32, device="cuda")


def _setup(hist, new, H, D, Dv, page, dtype, quantised, seed=0):
    pages = su.Pages([h + n for h, n in zip(hist, new)], H, D, Dv, page, dtype, quantised, seed)
    g = torch.Generator().manual_seed(seed)
    T = int(np.sum(new))
    return pages, su.rows_of((T, H, D), g, dtype), su.rows_of((T, H, Dv), g, dtype)


def _lens(hist):
    return torch.tensor(hist, dtype=torch.int32, device="cuda")


CASES = [
    # hist, new, H, D, Dv, page
    ([0], [1], 1, 32, 32, 16),
    ([0, 5, 31, 100], [1, 1, 1, 1], 4, 128, 128, 32),
    ([0, 15, 16, 17, 0], [33, 0, 1, 64, 7], 3, 64, 128, 16),
    ([250, 0, 3], [300, 513, 0], 2, 128, 32, 256),
    ([63, 1], [2, 700], 5, 32, 64, 64),
    ([0, 40, 0, 1000], [3001, 1999, 0, 2503], 5, 64, 128, 128),  # enough rows for four heads a thread
]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("hist,new,H,D,Dv,page", CASES)
def test_16_bit_rows_come_back_as_they_were(hist, new, H, D, Dv, page, dtype):
    pages, k, v = _setup(hist, new, H, D, Dv, page, dtype, False)
    c, off = pages.cache, _offsets(new)
    ws = torch.empty(256, dtype=torch.uint8, device="cuda")
    hb.cache_write(c, k, v, off, _lens(hist), pages.d_table, ws=ws)
    assert hb.device_status(ws) == hb.HSTU_OK
    at = 0
    written = torch.zeros((pages.num_pages, page), dtype=torch.bool)
    for b, (h, n) in enumerate(zip(hist, new)):
        page_i, slot = pages.places(b, h, n)
        assert torch.equal(c.k[page_i, :, slot], k[at:at + n]) and torch.equal(c.v[page_i, :, slot], v[at:at + n])
        written[page_i, slot] = True
        at += n
    rest = ~written.cuda()
    assert torch.isnan(c.k.transpose(1, 2)[rest]).all() and torch.isnan(c.v.transpose(1, 2)[rest]).all()
    k2, v2 = hb.cache_read(c, off, k.shape[0], pages.d_table, starts=_lens(hist), ws=ws)
    assert hb.device_status(ws) == hb.HSTU_OK
    assert torch.equal(k2, k) and torch.equal(v2, v)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("hist,new,H,D,Dv,page", CASES)
def test_8_bit_rows_are_the_nearest_codes(hist, new, H, D, Dv, page, dtype):
    pages, k, v = _setup(hist, new, H, D, Dv, page, dtype, True)
    for x in (k, v):  # rows of very different sizes, among them zeros and a row below every scale
        x *= torch.exp2(torch.randint(-9, 5, x.shape[:2], generator=torch.Generator().manual_seed(1)).cuda())[..., None].to(dtype)
    if k.shape[0] > 3:
        k[1] = 0
        v[2] = 1e-7
        k[3, 0, 0], v[3, 0, :2] = float("inf"), torch.tensor([float("nan"), -float("inf")], dtype=dtype)
    off = _offsets(new)
    hb.cache_write(pages.cache, k, v, off, _lens(hist), pages.d_table)
    k2, v2 = hb.cache_read(pages.cache, off, k.shape[0], pages.d_table, starts=_lens(hist))
    at = 0
    for x, got, scale in ((k, k2, pages.cache.k_scale), (v, v2, pages.cache.v_scale)):
        want, e = su.quantise(su.f64(x))
        # codes have 4 significant bits, so a power-of-two multiple is exact in
        # bf16; fp16 has the exponents down to 2^-24
        want = torch.tensor(want).to(dtype)
        assert torch.equal(torch.nan_to_num(got.cpu(), nan=12345.0), torch.nan_to_num(want, nan=12345.0))
        at = 0
        for b, (h, n) in enumerate(zip(hist, new)):
            page_i, slot = pages.places(b, h, n)
            assert np.array_equal(scale[page_i, :, slot].cpu().numpy().astype(np.float64) - 127, e[at:at + n])
            at += n


@pytest.mark.parametrize("quantised", [False, True])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("D,R", [(128, 128), (64, 32), (32, 16), (128, 48)])
@pytest.mark.parametrize("hist,new,H", [([100, 0, 7], [3, 150, 40], 3), ([5, 0, 300], [5000, 1, 2999], 6)])
def test_rotation_on_the_way_in(hist, new, H, D, R, interleaved, quantised):
    dtype = torch.bfloat16
    pages, k, v = _setup(hist, new, H, D, 64, 32, dtype, quantised, seed=R)
    off, table = _offsets(new), hb.rope_table(R, interleaved=interleaved)
    f, m = su.frequencies(R)
    own = np.concatenate([np.arange(h, h + n) for h, n in zip(hist, new)])
    given = np.random.default_rng(0).integers(0, 100000, size=k.shape[0]).astype(np.int32)
    for pos, arg in ((own, None), (given, torch.tensor(given, device="cuda"))):
        hb.cache_write(pages.cache, k, v, off, _lens(hist), pages.d_table, rope=table, positions=arg)
        k2, v2 = hb.cache_read(pages.cache, off, k.shape[0], pages.d_table, starts=_lens(hist))
        want = su.rotate(su.f64(k), pos, f, m, interleaved)
        tol = su.rotate_slack(su.f64(k), f, m, interleaved)
        if quantised:
            # half a step of a code (2^-4 of the value, or of the smallest
            # normal code 2^-6 below that) under the scale, which may come out
            # twice as large where the row's top is at a power's border
            top = np.abs(want).max(-1, keepdims=True)
            tol = 2.0 ** -4 * np.abs(want) + 2.0 ** -10 * 2 * (top * 2 / su.E4M3_MAX) + 1.1 * tol
        else:
            tol = tol + su.half_step(dtype) * np.abs(want) * 1.01
        assert np.all(np.abs(su.f64(k2) - want) <= tol)
        want_v = torch.tensor(su.quantise(su.f64(v))[0]).to(dtype) if quantised else v.cpu()
        assert torch.equal(v2.cpu(), want_v)


def test_rows_of_a_wider_projection():
    hist, new, H, D, Dv = [4, 9], [30, 21], 2, 64, 128
    pages, k, v = _setup(hist, new, H, D, Dv, 16, torch.bfloat16, True)
    wide = torch.randn((51, H * (D + Dv) + 64), device="cuda").bfloat16()
    k2, v2 = wide[:, 64:64 + H * D].unflatten(1, (H, D)), wide[:, 64 + H * D:].unflatten(1, (H, Dv))
    k2.copy_(k)
    v2.copy_(v)
    off = _offsets(new)
    hb.cache_write(pages.cache, k, v, off, _lens(hist), pages.d_table)
    want = [t.clone() for t in (pages.cache.k, pages.cache.v, pages.cache.k_scale, pages.cache.v_scale)]
    pages.poison()
    hb.cache_write(pages.cache, k2, v2, off, _lens(hist), pages.d_table)
    for t, w in zip((pages.cache.k, pages.cache.v, pages.cache.k_scale, pages.cache.v_scale), want):
        assert torch.equal(t, w)


def test_rows_without_a_valid_place_are_skipped_and_reported():
    hist, new, H, D = [0, 16, 0], [20, 10, 5], 2, 32
    pages, k, v = _setup(hist, new, H, D, D, 16, torch.bfloat16, False, seed=4)
    off = _offsets(new)
    ws = torch.empty(256, dtype=torch.uint8, device="cuda")

    def write(table=None, lens=None, offsets=None):
        pages.poison()
        hb.cache_write(pages.cache, k, v, off if offsets is None else offsets,
                       _lens(hist) if lens is None else lens, pages.d_table if table is None else table, ws=ws)
        return hb.device_status(ws)

    assert write() == hb.HSTU_OK
    good = pages.cache.k.clone()
    for bad in (-1, pages.num_pages, 1 << 30):
        table = pages.d_table.clone()
        table[0, 1] = bad  # rows 16..19 of sequence 0
        assert write(table=table) == 5
        page_i, slot = pages.places(0, 16, 4)
        want = good.clone()
        want[page_i, :, slot] = float("nan")
        assert torch.equal(torch.nan_to_num(pages.cache.k, nan=99.0), torch.nan_to_num(want, nan=99.0))
        out = torch.full((35, H, D), 7.0, dtype=torch.bfloat16, device="cuda")
        hb.cache_read(pages.cache, off, 35, table, starts=_lens(hist), outs=(out, out.clone()), ws=ws)
        assert hb.device_status(ws) == 5
        assert torch.equal(out[16:20], torch.full_like(out[16:20], 7.0)) and torch.equal(out[:16], k[:16])
    assert write(lens=_lens([0, -1, 0])) == 5
    assert write(lens=_lens([0, 16, 32 * 16])) == 5  # past the table's width
    assert write(lens=_lens([0, 2**31 - 1, 0])) == 5
    assert write(offsets=torch.tensor([0, 20, 30, 34], dtype=torch.int32, device="cuda")) == 5
    assert write(offsets=torch.tensor([1, 20, 30, 35], dtype=torch.int32, device="cuda")) == 5
    assert write(offsets=torch.tensor([0, 25, 20, 35], dtype=torch.int32, device="cuda")) == 5
    assert write() == hb.HSTU_OK  # the error word is the last call's


def test_a_cache_past_32_bits():
    """Element offsets of the last pages are above 2^32."""
    H, D, page = 8, 128, 256
    n = (1 << 32) // (H * D * page) + 3
    cache = hb.alloc_cache(n, page, H, D, dtype=torch.bfloat16)
    g = torch.Generator().manual_seed(0)
    k, v = su.rows_of((300, H, D), g, torch.bfloat16), su.rows_of((300, H, D), g, torch.bfloat16)
    table = torch.tensor([[n - 1, n - 2]], dtype=torch.int32, device="cuda")
    cache.k[2].fill_(0)
    hb.cache_write(cache, k, v, _offsets([300]), _lens([0]), table)
    assert torch.equal(cache.k[n - 1].transpose(0, 1), k[:256]) and torch.equal(cache.v[n - 2, :, :44].transpose(0, 1), v[256:])
    assert (cache.k[2] == 0).all()
    k2, v2 = hb.cache_read(cache, _offsets([300]), 300, table)
    assert torch.equal(k2, k) and torch.equal(v2, v)
    o = hb.fwd_paged(k[-1:].contiguous(), cache, _lens([300]), table, 300)
    want, tol = su.paged_reference(su.f64(k[-1:]), [(su.f64(k), su.f64(v))], [1], None, 300, D ** -0.5, torch.bfloat16)
    assert np.all(np.abs(su.f64(o) - want) <= tol)


def test_captured_and_replayed():
    """A decode step in a graph: one row a sequence, lengths advanced by the caller."""
    hist, H, D = [10, 40], 2, 64
    pages = su.Pages([h + 8 for h in hist], H, D, D, 16, torch.bfloat16, True)
    k, v = (torch.zeros((2, H, D), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    off, lens = _offsets([1, 1]), _lens(hist)
    hb.cache_write(pages.cache, k, v, off, lens, pages.d_table)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        hb.cache_write(pages.cache, k, v, off, lens, pages.d_table)
        lens.add_(1)
    g = torch.Generator().manual_seed(0)
    steps = [su.rows_of((2, H, D), g, torch.bfloat16) for _ in range(3)]
    for x in steps:
        k.copy_(x)
        v.copy_(-x)
        graph.replay()
    k2, v2 = hb.cache_read(pages.cache, _offsets([3, 3]), 6, pages.d_table, starts=_lens(hist))
    want = torch.tensor(su.quantise(np.stack([su.f64(x) for x in steps], 1).reshape(6, H, D))[0]).bfloat16()
    assert torch.equal(k2.cpu(), want) and torch.equal(v2.cpu(), -want)
