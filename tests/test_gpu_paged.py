"""Candidate rows against the paged cache on the GPU, against the 64-bit form."""
import math

import numpy as np
import pytest
import torch

import oracle.hstu_oracle as orc
from jagged_hstu_attention_gb300 import binding as hb
from jagged_hstu_attention_gb300 import workloads as wl
import serving_testutil as su

pytestmark = pytest.mark.gpu


def _int32(v):
    return torch.tensor(np.ascontiguousarray(v), dtype=torch.int32, device="cuda")


def _offsets(counts):
    return np.concatenate([[0], np.cumsum(counts)])


def _run(pages, rows, counts, func, N, seed=0, single=False, alpha=None):
    g = torch.Generator().manual_seed(seed)
    C = int(np.sum(counts))
    q = su.rows_of((C, pages.heads, pages.dim), g, pages.dtype)
    out = torch.full((C, pages.heads, pages.dim_v), 99.0, dtype=pages.dtype, device="cuda")
    ws = hb.paged_workspace(pages.cache, len(counts), C, N)
    o = hb.fwd_paged(q, pages.cache, pages.d_lens, pages.d_table, N, alpha=alpha,
                     cand_offsets=None if single else _int32(_offsets(counts)),
                     func_c=None if func is None else _int32(func), ws=ws, out=out)
    assert hb.device_status(ws) == hb.HSTU_OK
    alpha = alpha if alpha is not None else 1 / math.sqrt(pages.dim)
    want, tol = su.paged_reference(su.f64(q), rows, counts, func, N, alpha, pages.dtype)
    got = su.f64(o)
    assert np.all(np.abs(got - want) <= tol), np.max(np.abs(got - want) / tol)
    return q, o


SIZES = [
    # lens, H, D, Dv, page
    ([1], 1, 32, 32, 16),
    ([16, 64, 33], 2, 32, 32, 16),
    ([0, 1, 15, 16, 17, 255, 256, 257], 3, 64, 128, 32),
    ([1000, 3], 2, 128, 128, 64),
    ([513], 4, 128, 32, 256),
    ([700, 0, 129], 1, 32, 128, 128),
    ([5000], 2, 128, 64, 16),
    ([311, 64], 2, 64, 64, 64),
]


@pytest.mark.parametrize("quantised", [False, True])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("lens,H,D,Dv,page", SIZES)
def test_one_new_token_a_sequence(lens, H, D, Dv, page, dtype, quantised):
    pages = su.Pages(lens, H, D, Dv, page, dtype, quantised)
    rows = pages.fill(np.random.default_rng(len(lens) + D))
    _run(pages, rows, [1] * len(lens), None, max(lens) or 1, single=True)
    _run(pages, rows, [1] * len(lens), None, 2 * max(lens) + 1000)  # N above every length; given offsets


@pytest.mark.parametrize("quantised", [False, True])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("D,Dv", [(128, 128), (64, 32), (32, 128)])
def test_more_ctas_than_sms(D, Dv, dtype, quantised):
    """One row for each of many sequences: four warps a CTA, one split and several."""
    rng = np.random.default_rng(D + Dv)
    lens = rng.integers(0, 700, size=90).tolist()
    pages = su.Pages(lens, 2, D, Dv, 32, dtype, quantised)
    rows = pages.fill(rng)
    _run(pages, rows, [1] * 90, None, 700, single=True)
    func = np.array([(min(60, n), max(0, n - 33), n) for n in lens]).T
    _run(pages, rows, [1] * 90, func, 700, single=True)
    _run(pages, rows, [1] * 90, None, 400000, single=True)  # N far above the lengths


@pytest.mark.parametrize("quantised", [False, True])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("nfunc", [1, 3, 5, 9])
@pytest.mark.parametrize("D,Dv", [(128, 128), (32, 64)])
def test_several_candidates_with_masks(nfunc, D, Dv, dtype, quantised):
    lens, counts = [700, 33, 260, 0, 1, 1300], [10, 0, 3, 2, 1, 25]
    pages = su.Pages(lens, 2, D, Dv, 32, dtype, quantised, seed=nfunc)
    rng = np.random.default_rng(nfunc)
    rows = pages.fill(rng)
    C = sum(counts)
    func = np.zeros((nfunc, C), dtype=np.int32)
    for b, L in enumerate(lens):
        for c in range(sum(counts[:b]), sum(counts[:b + 1])):
            func[0, c] = rng.integers(0, L + 1) if c % 3 else 0
            for i in range(1, nfunc):
                func[i, c] = rng.integers(-5, L + 6)
    func[:, 4] = 0  # a candidate that sees nothing
    _, o = _run(pages, rows, counts, func, 1300)
    assert (o[4] == 0).all()


def test_a_candidate_sees_the_history_and_itself():
    lens, counts, H, D = [600, 130, 2000], [17, 1, 9], 4, 128
    full = [n + c for n, c in zip(lens, counts)]
    pages = su.Pages(full, H, D, D, 64, torch.bfloat16, False)
    rows = pages.fill(np.random.default_rng(7))
    func = np.array([(n, n + j, n + j + 1) for n, c in zip(lens, counts) for j in range(c)]).T
    _run(pages, rows, counts, func, max(full))


@pytest.mark.parametrize("quantised", [False, True])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_what_is_not_seen_may_hold_anything(dtype, quantised):
    """NaN and infinities where a candidate does not look, in tiles that it and
    its neighbours do read."""
    lens, counts, H, D = [300, 40], [3, 9], 2, 64
    pages = su.Pages(lens, H, D, D, 16, dtype, quantised)
    rows = pages.fill(np.random.default_rng(3))
    c = pages.cache
    for b, pos, what in ((0, 5, "nan"), (0, 17, "inf"), (0, 250, "nan"), (1, 38, "nan")):
        page, slot = (int(x[0]) for x in pages.places(b, pos, 1))
        if quantised:  # a NaN code; infinity as the largest code under an infinite scale
            c.k[page, :, slot], c.v[page, :, slot] = (0x7f, 0x7f) if what == "nan" else (0x7e, 0x7e)
            if what == "inf":
                c.k_scale[page, :, slot] = c.v_scale[page, :, slot] = 255
        else:
            c.k[page, :, slot] = c.v[page, :, slot] = float(what)
        for x in rows[b]:
            x[pos] = float(what)
    # sequence 0: candidates see around the poisoned rows; sequence 1: all but the last two rows
    func = np.zeros((5, 12), dtype=np.int32)
    func[:, :3] = np.array([[5, 6, 17, 18, 250], [0, 18, 200, 251, 300], [5, 18, 100, 0, 0]]).T
    func[:, 3:] = np.array([[38, 39, 40, 0, 0]] * 9).T
    _run(pages, rows, counts, func, 300)
    # a candidate that does see one gets what the formula gives; its neighbours are not touched
    func[:, 1] = [300, 0, 0, 0, 0]
    q = su.rows_of((12, H, D), torch.Generator().manual_seed(0), dtype)
    o = hb.fwd_paged(q, c, pages.d_lens, pages.d_table, 300, cand_offsets=_int32(_offsets(counts)),
                     func_c=_int32(func))
    func[:, 1] = 0
    want, tol = su.paged_reference(su.f64(q), rows, counts, func, 300, D ** -0.5, dtype)
    keep = np.arange(12) != 1
    assert np.all(np.abs(su.f64(o) - want)[keep] <= tol[keep])
    assert not torch.isfinite(o[1]).any()


def test_large_scores_and_scales():
    """Scores in the thousands and value scales far from one: fp16 products keep the range."""
    H, D = 2, 64
    for dtype, quantised in ((torch.float16, False), (torch.float16, True), (torch.bfloat16, True)):
        pages = su.Pages([333, 80], H, D, D, 32, dtype, quantised)
        rows = pages.fill(np.random.default_rng(9))
        _run(pages, rows, [2, 1], None, 333, alpha=900.0)
        _run(pages, rows, [2, 1], None, 333, alpha=-900.0)
        _run(pages, rows, [2, 1], None, 333, alpha=1e-6)
        if quantised:
            up = [100, 30] if dtype == torch.bfloat16 else [10, 3]
            for b, by in enumerate(up):
                for t, x in ((pages.cache.v_scale, rows[b][1]), (pages.cache.k_scale, rows[b][0])):
                    sign = 1 if t is pages.cache.v_scale else -1
                    page, slot = pages.places(b, 0, x.shape[0])
                    t[page, :, slot] = (t[page, :, slot].int() + sign * by).to(torch.uint8)
                    x *= 2.0 ** (sign * by)
            _run(pages, rows, [2, 1], None, 333)


def test_rows_equal_those_of_the_contiguous_kernels_inputs():
    """The same rows through the targets-only kernel and the paged one agree
    with the oracle within the framework's bounds."""
    lens, counts, H, D, N = [400, 77, 256], [4, 2, 3], 2, 128, 400
    pages = su.Pages(lens, H, D, D, 64, torch.bfloat16, False)
    rows = pages.fill(np.random.default_rng(11))
    off = _offsets(lens)
    k, v = hb.cache_read(pages.cache, _int32(off), int(off[-1]), pages.d_table)
    func = np.array([[int(n)] for n, c in zip(lens, counts) for _ in range(c)]).T
    q, o = _run(pages, rows, counts, func, N)
    contiguous = hb.fwd_targets(q, k, v, _int32(off), _int32(_offsets(counts)), _int32(func), N)
    want = orc.fwd_targets(su.f64(q), su.f64(k), su.f64(v), off, _offsets(counts), func, 1, N, D ** -0.5)
    for got in (o, contiguous):
        assert np.linalg.norm(su.f64(got) - want) <= 5e-3 * np.linalg.norm(want)


def test_repeatable_and_on_another_stream():
    pages = su.Pages([3000, 2100], 2, 128, 128, 64, torch.bfloat16, True)
    pages.fill(np.random.default_rng(0))
    q = su.rows_of((2, 2, 128), torch.Generator().manual_seed(0), torch.bfloat16)
    first = hb.fwd_paged(q, pages.cache, pages.d_lens, pages.d_table, 3000)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for _ in range(20):
        again = hb.fwd_paged(q, pages.cache, pages.d_lens, pages.d_table, 3000, stream=side)
        side.synchronize()
        assert torch.equal(again, first)


def _stream_of(t):
    """The stream whose memory the tensor lies in."""
    for seg in torch.cuda.memory_snapshot():
        if seg["address"] <= t.data_ptr() < seg["address"] + seg["total_size"]:
            return seg["stream"]
    return None


def test_outputs_belong_to_the_stream_of_the_call():
    """Memory of another stream could still be in use there."""
    pages = su.Pages([3000, 2100], 2, 128, 128, 64, torch.bfloat16, True)
    pages.fill(np.random.default_rng(0))
    q = su.rows_of((2, 2, 128), torch.Generator().manual_seed(0), torch.bfloat16)
    off, pos, table = _int32([0, 3000, 5100]), _int32([5, 7]), hb.rope_table(128)
    side = torch.cuda.Stream()
    first = hb.fwd_paged(q, pages.cache, pages.d_lens, pages.d_table, 3000)
    turned = hb.rope(q, None, pos, table)[0]
    k, v = hb.cache_read(pages.cache, off, 5100, pages.d_table)
    torch.cuda.synchronize()
    outs = [hb.fwd_paged(q, pages.cache, pages.d_lens, pages.d_table, 3000, stream=side),
            hb.rope(q, None, pos, table, stream=side)[0],
            *hb.cache_read(pages.cache, off, 5100, pages.d_table, stream=side)]
    torch.cuda.synchronize()
    for got, want in zip(outs, (first, turned, k, v)):
        assert torch.equal(got, want)
        assert _stream_of(got) == side.cuda_stream and _stream_of(want) != side.cuda_stream
    with pytest.raises(ValueError):  # a refusal leaves the current stream as it was
        hb.rope(q.cpu(), None, pos, table, stream=side)
    assert torch.cuda.current_stream() != side


def test_bad_sequences_are_left_as_they_were():
    lens, counts, H, D = [600, 50, 90], [2, 1, 3], 2, 32
    pages = su.Pages(lens, H, D, D, 16, torch.bfloat16, False, extra_pages=1)
    pages.fill(np.random.default_rng(1))
    q = su.rows_of((6, H, D), torch.Generator().manual_seed(1), torch.bfloat16)
    good = hb.fwd_paged(q, pages.cache, pages.d_lens, pages.d_table, 600, cand_offsets=_int32(_offsets(counts)))

    def run(lens=None, table=None, offsets=None, N=600):
        out = torch.full_like(good, 55.0)
        ws = hb.paged_workspace(pages.cache, 3, 6, N)
        hb.fwd_paged(q, pages.cache, pages.d_lens if lens is None else _int32(lens),
                     pages.d_table if table is None else table, N,
                     cand_offsets=_int32(_offsets(counts) if offsets is None else offsets), ws=ws, out=out)
        return hb.device_status(ws), out

    def left(out, which):
        rows = torch.tensor([c for b in which for c in range(int(_offsets(counts)[b]), int(_offsets(counts)[b + 1]))],
                            dtype=torch.long, device="cuda")
        rest = torch.ones(6, dtype=torch.bool, device="cuda")
        rest[rows] = False
        assert (out[rows] == 55.0).all() and torch.equal(out[rest], good[rest])

    for b, at in ((0, 0), (0, 37), (2, 5)):
        for bad in (-7, pages.num_pages):
            table = pages.d_table.clone()
            table[b, at] = bad
            st, out = run(table=table)
            assert st == 5
            left(out, [b])
    for bad in (-1, 601, 2**31 - 1):
        st, out = run(lens=[600, bad, 90])
        assert st == 5
        left(out, [1])
    for offsets in ([1, 2, 3, 6], [0, 2, 3, 5], [0, 2, 3, 7]):
        st, out = run(offsets=offsets)
        assert st == 5
        left(out, [0, 1, 2])
    st, out = run(offsets=[0, 4, 3, 6])
    assert st == 5
    st, out = run()
    assert st == hb.HSTU_OK and torch.equal(out, good)


def test_bad_offsets_of_long_sequences_leave_their_rows():
    """Sequences of several splits: a refused one wrote no sums to join, and the
    workspace may hold those of an earlier call."""
    lens, counts, H, D, N = [100, 1500, 1400], [2, 1, 3], 2, 64, 1500
    pages = su.Pages(lens, H, D, D, 32, torch.bfloat16, False)
    pages.fill(np.random.default_rng(2))
    q = su.rows_of((6, H, D), torch.Generator().manual_seed(2), torch.bfloat16)
    ws = hb.paged_workspace(pages.cache, 3, 6, N)
    assert ws.numel() > 256  # several splits

    def run(offsets, table=None):
        out = torch.full((6, H, D), 55.0, dtype=torch.bfloat16, device="cuda")
        hb.fwd_paged(q, pages.cache, pages.d_lens, pages.d_table if table is None else table, N,
                     cand_offsets=_int32(offsets), ws=ws, out=out)
        return hb.device_status(ws), out

    st, good = run(_offsets(counts))
    assert st == hb.HSTU_OK
    st, out = run([0, 2, 9, 6])  # sequence 1 ends past the candidates, sequence 2 before it begins
    assert st == 5 and torch.equal(out[:2], good[:2]) and (out[2:] == 55.0).all()
    st, out = run([0, 2, 3, 5])
    assert st == 5 and (out == 55.0).all()
    table = pages.d_table.clone()
    table[1, 40] = -1  # in the third split of sequence 1
    st, out = run(_offsets(counts), table)
    assert st == 5 and (out[2] == 55.0).all() and torch.equal(out[:2], good[:2]) and torch.equal(out[3:], good[3:])
    st, out = run(_offsets(counts))
    assert st == hb.HSTU_OK and torch.equal(out, good)


def test_captured_and_replayed_with_longer_histories():
    """One graph serves every length up to its N; two graphs with workspaces of
    their own may share the cache."""
    H, D, N = 2, 64, 2000
    pages = su.Pages([2000, 2000], H, D, D, 64, torch.float16, True)
    rows = pages.fill(np.random.default_rng(5))
    q = su.rows_of((2, H, D), torch.Generator().manual_seed(5), torch.float16)
    lens, out = _int32([0, 0]), torch.empty((2, H, D), dtype=torch.float16, device="cuda")
    ws = hb.paged_workspace(pages.cache, 2, 2, N)
    hb.fwd_paged(q, pages.cache, lens, pages.d_table, N, ws=ws, out=out)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        hb.fwd_paged(q, pages.cache, lens, pages.d_table, N, ws=ws, out=out)
    for a, b in ((1, 0), (2000, 999), (17, 2000), (0, 0)):
        lens.copy_(_int32([a, b]))
        graph.replay()
        cut = [(rows[i][0][:n], rows[i][1][:n]) for i, n in enumerate((a, b))]
        want, tol = su.paged_reference(su.f64(q), cut, [1, 1], None, N, D ** -0.5, torch.float16)
        assert np.all(np.abs(su.f64(out) - want) <= tol)


def test_serving_steps_together():
    """A session as a server runs it: a prompt, then requests of new rows and
    candidates; projections, rotation, cache and attention of this package,
    against the formulas in 64 bits on the rows that the cache holds."""
    torch.manual_seed(0)
    H, D, din, N, page, dtype = 4, 64, 256, 512, 32, torch.bfloat16
    table = hb.rope_table(D)
    f, m = su.frequencies(D)
    w = {n: (torch.randn((H * D, din), device="cuda") / 16).to(dtype) for n in "qkv"}
    prompts, steps = [100, 37, 250], 3
    pages = su.Pages([n + steps for n in prompts], H, D, D, page, dtype, True)
    lens = _int32([0, 0, 0])

    def append(x, counts):
        k, v = (hb.project_rows(x, w[n], want_z=False)[0].unflatten(1, (H, D)) for n in "kv")
        hb.cache_write(pages.cache, k, v, _int32(_offsets(counts)), lens, pages.d_table, rope=table)
        lens.add_(_int32(counts))

    append(torch.randn((sum(prompts), din), device="cuda").to(dtype), prompts)
    for step in range(steps):
        x = torch.randn((3, din), device="cuda").to(dtype)
        append(x, [1, 1, 1])
        q = hb.project_rows(x, w["q"], want_z=False)[0].unflatten(1, (H, D))
        pos = lens - 1
        qr, _ = hb.rope(q, None, pos, table)
        o = hb.fwd_paged(qr, pages.cache, lens, pages.d_table, N)
        n = [p + step + 1 for p in prompts]
        off = _offsets(n)
        k, v = hb.cache_read(pages.cache, _int32(off), int(off[-1]), pages.d_table)
        rows = [(su.f64(k)[off[b]:off[b + 1]], su.f64(v)[off[b]:off[b + 1]]) for b in range(3)]
        turned = su.rotate(su.f64(q), pos.cpu().numpy(), f, m)
        assert np.all(np.abs(su.f64(qr) - turned) <= su.half_step(dtype) * np.abs(turned) * 1.01 +
                      su.rotate_slack(su.f64(q), f, m))
        want, tol = su.paged_reference(su.f64(qr), rows, [1, 1, 1], None, N, D ** -0.5, dtype)
        assert np.all(np.abs(su.f64(o) - want) <= tol)
        func = _int32(np.array([n]))
        o2 = hb.fwd_targets_only(qr, k, v, _int32(off), func, N)
        assert np.linalg.norm(su.f64(o2) - su.f64(o)) <= 5e-3 * np.linalg.norm(su.f64(o))
    assert lens.cpu().tolist() == [p + steps for p in prompts]


def test_a_history_past_the_contiguous_kernels_limit():
    H, D, L = 1, 32, 70001
    pages = su.Pages([L, 40], H, D, D, 256, torch.float16, True)
    rows = pages.fill(np.random.default_rng(4))
    _run(pages, rows, [1, 1], None, 1 << 20, single=True)
    func = np.array([[20000, 39999, 70000], [3, 50, 60]]).T
    _run(pages, rows, [1, 1], func, 1 << 17, single=True)


def test_many_candidates_take_several_passes():
    """More than one pass (64 candidates), and every way of sharing tiles."""
    lens, counts = [700, 1100, 90, 300, 40], [130, 65, 33, 17, 9]
    full = [n + c for n, c in zip(lens, counts)]
    func = np.array([(n, n + j, n + j + 1) for n, c in zip(lens, counts) for j in range(c)]).T
    for dtype, quantised in ((torch.bfloat16, True), (torch.float16, False)):
        pages = su.Pages(full, 2, 64, 64, 64, dtype, quantised)
        rows = pages.fill(np.random.default_rng(8))
        _run(pages, rows, counts, func, max(full))
        _run(pages, rows, counts, None, max(full))


# More than 16 candidates a sequence on average, widths of 128, N above 256: the kernel whose
# products are tcgen05's (bf16 and 8-bit pages).
MANY_TYPES = [(torch.bfloat16, False), (torch.bfloat16, True), (torch.float16, True), (torch.float16, False)]
MANY_SIZES = [
    # lens, counts, H, page
    ([300, 0, 1, 129, 2100], [40, 5, 17, 33, 70], 2, 64),
    ([15, 16, 17, 700], [20, 16, 64, 65], 3, 16),
    ([1537], [17], 1, 256),
    ([128, 127, 640], [200, 0, 1], 1, 32),
]


@pytest.mark.parametrize("dtype,quantised", MANY_TYPES)
@pytest.mark.parametrize("nfunc", [0, 1, 3, 9])
@pytest.mark.parametrize("lens,counts,H,page", MANY_SIZES)
def test_crowds_of_candidates(lens, counts, H, page, nfunc, dtype, quantised):
    pages = su.Pages(lens, H, 128, 128, page, dtype, quantised, seed=nfunc)
    rng = np.random.default_rng(nfunc + H)
    rows = pages.fill(rng)
    C = sum(counts)
    func = None
    if nfunc:
        func = np.zeros((nfunc, C), dtype=np.int32)
        for b, L in enumerate(lens):
            for c in range(sum(counts[:b]), sum(counts[:b + 1])):
                func[0, c] = rng.integers(0, L + 1) if c % 3 else 0
                for i in range(1, nfunc):
                    func[i, c] = rng.integers(-5, L + 6)
        func[:, 4] = 0
    _, o = _run(pages, rows, counts, func, max(lens))
    assert func is None or (o[4] == 0).all()
    if func is None:
        _run(pages, rows, counts, None, max(lens), alpha=-3.0)
        _run(pages, rows, counts, None, 3 * max(lens), alpha=1e-6)


@pytest.mark.parametrize("dtype,quantised", MANY_TYPES)
def test_crowds_of_candidates_and_rows_that_hold_anything(dtype, quantised):
    lens, counts, H, D = [700, 90], [35, 5], 2, 128
    pages = su.Pages(lens, H, D, D, 16, dtype, quantised)
    rows = pages.fill(np.random.default_rng(5))
    c = pages.cache
    for b, pos in ((0, 5), (0, 300), (1, 88)):
        page, slot = (int(x[0]) for x in pages.places(b, pos, 1))
        c.k[page, :, slot] = c.v[page, :, slot] = 0x7f if quantised else float("nan")
        for x in rows[b]:
            x[pos] = float("nan")
    func = np.zeros((3, 40), dtype=np.int32)
    func[:, :35] = np.array([[5, 6, 300], [0, 301, 700], [5, 6, 200], [0, 100, 290], [0, 0, 0]] * 7).T
    func[:, 35:] = np.array([[88, 89, 90]] * 5).T
    _run(pages, rows, counts, func, 700)
    func[:, 33] = [302, 0, 0]  # sees two of them; its neighbours are not touched
    q = su.rows_of((40, H, D), torch.Generator().manual_seed(0), dtype)
    o = hb.fwd_paged(q, c, pages.d_lens, pages.d_table, 700, cand_offsets=_int32(_offsets(counts)), func_c=_int32(func))
    func[:, 33] = 0
    want, tol = su.paged_reference(su.f64(q), rows, counts, func, 700, D ** -0.5, dtype)
    keep = np.arange(40) != 33
    assert np.all(np.abs(su.f64(o) - want)[keep] <= tol[keep])
    assert not torch.isfinite(o[33]).any()


@pytest.mark.parametrize("quantised", [False, True])
def test_crowds_of_candidates_refused_replayed_and_on_two_streams(quantised):
    lens, counts, H, D, N = [100, 1500, 1400], [20, 40, 66], 2, 128, 1500
    pages = su.Pages(lens, H, D, D, 32, torch.bfloat16, quantised)
    pages.fill(np.random.default_rng(2))
    q = su.rows_of((126, H, D), torch.Generator().manual_seed(2), torch.bfloat16)
    off = _int32(_offsets(counts))
    ws = hb.paged_workspace(pages.cache, 3, 126, N)

    def run(offsets, table=None):
        out = torch.full((126, H, D), 55.0, dtype=torch.bfloat16, device="cuda")
        hb.fwd_paged(q, pages.cache, pages.d_lens, pages.d_table if table is None else table, N,
                     cand_offsets=offsets, ws=ws, out=out)
        return hb.device_status(ws), out

    st, good = run(off)
    assert st == hb.HSTU_OK
    table = pages.d_table.clone()
    table[1, 40] = -1
    table[0, 2] = pages.num_pages
    st, out = run(off, table)
    assert st == 5 and (out[:60] == 55.0).all() and torch.equal(out[60:], good[60:])
    for bad in ([0, 20, 60, 125], [1, 20, 60, 126]):
        st, out = run(_int32(bad))
        assert st == 5 and (out == 55.0).all()
    streams = [torch.cuda.Stream() for _ in range(3)]
    torch.cuda.synchronize()
    outs = [hb.fwd_paged(q, pages.cache, pages.d_lens, pages.d_table, N, cand_offsets=off, stream=s)
            for _ in range(10) for s in streams]
    torch.cuda.synchronize()
    assert all(torch.equal(o, good) for o in outs)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = hb.fwd_paged(q, pages.cache, pages.d_lens, pages.d_table, N, cand_offsets=off)
    for _ in range(5):
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, good)


def test_crowds_of_candidates_beside_kernels_that_hold_tensor_memory():
    """The attention and the projection kernels on another stream: all take
    tensor memory, whichever gets an SM first."""
    lens, counts, H, D, N = [900, 1500, 300, 2000] * 8, [20, 30, 17, 40] * 8, 4, 128, 2000
    pages = su.Pages(lens, H, D, D, 64, torch.bfloat16, False)
    pages.fill(np.random.default_rng(4))
    g = torch.Generator().manual_seed(4)
    qc = su.rows_of((sum(counts), H, D), g, torch.bfloat16)
    off = _int32(_offsets(counts))
    n = [700, 1024, 333, 64] * 8
    x = [su.rows_of((sum(n), H, D), g, torch.bfloat16) for _ in range(3)]
    seq = _int32(_offsets(n))
    func = _int32(np.concatenate([np.arange(1, m + 1) for m in n])[None])
    w = su.rows_of((1, 512, H * D), g, torch.bfloat16)[0]

    def paged():
        return hb.fwd_paged(qc, pages.cache, pages.d_lens, pages.d_table, N, cand_offsets=off)

    def others():
        return hb.fwd(*x, seq, func, 1024), hb.project_rows(x[0].view(-1, H * D), w)[0]

    want, want_others = paged(), others()
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(3)]
    got, got_others = [], []
    for _ in range(10):
        for s in streams:
            with torch.cuda.stream(s):
                if s is streams[1]:
                    got_others.append(others())
                else:
                    got.append(paged())
    torch.cuda.synchronize()
    assert all(torch.equal(o, want) for o in got)
    assert all(torch.equal(a, b) for o in got_others for a, b in zip(o, want_others))


def test_a_length_past_the_page_table_is_refused():
    pages = su.Pages([40, 40], 1, 32, 32, 16, torch.bfloat16, False)
    pages.fill(np.random.default_rng(0))
    q = su.rows_of((2, 1, 32), torch.Generator().manual_seed(0), torch.bfloat16)
    out = torch.full((2, 1, 32), 9.0, dtype=torch.bfloat16, device="cuda")
    ws = hb.paged_workspace(pages.cache, 2, 2, 500)
    hb.fwd_paged(q, pages.cache, _int32([49, 40]), pages.d_table, 500, ws=ws, out=out)  # 3 pages of 16
    assert hb.device_status(ws) == 5 and (out[0] == 9.0).all() and (out[1] != 9.0).any()


def test_no_candidates():
    pages = su.Pages([40, 4000], 1, 32, 32, 16, torch.bfloat16, False)
    q = torch.empty((0, 1, 32), dtype=torch.bfloat16, device="cuda")
    o = hb.fwd_paged(q, pages.cache, pages.d_lens, pages.d_table, 4000, cand_offsets=_int32([0, 0, 0]))
    torch.cuda.synchronize()
    assert o.shape == (0, 1, 32)


def test_two_calls_at_once():
    """Calls on two streams, each with its own workspace, over one cache."""
    pages = su.Pages([3000, 2100, 900], 2, 64, 64, 64, torch.bfloat16, False)
    pages.fill(np.random.default_rng(0))
    qs = [su.rows_of((3, 2, 64), torch.Generator().manual_seed(i), torch.bfloat16) for i in range(2)]
    want = [hb.fwd_paged(q, pages.cache, pages.d_lens, pages.d_table, 3000) for q in qs]
    streams = [torch.cuda.Stream() for _ in qs]
    ws = [hb.paged_workspace(pages.cache, 3, 3, 3000) for _ in qs]
    outs = [torch.zeros_like(w) for w in want]
    torch.cuda.synchronize()
    for _ in range(50):
        for q, s, w, o in zip(qs, streams, ws, outs):
            hb.fwd_paged(q, pages.cache, pages.d_lens, pages.d_table, 3000, ws=w, out=o, stream=s)
    torch.cuda.synchronize()
    assert all(torch.equal(o, w) for o, w in zip(outs, want))


def test_the_binding_refuses_what_does_not_fit():
    pages = su.Pages([40], 2, 64, 32, 16, torch.bfloat16, False)
    c, lens, table = pages.cache, pages.d_lens, pages.d_table
    q = torch.zeros((1, 2, 64), dtype=torch.bfloat16, device="cuda")
    for bad in (dict(q_c=q.half()), dict(q_c=q[:, :1]), dict(q_c=q.transpose(1, 2).contiguous().transpose(1, 2)),
                dict(q_c=q.cpu()), dict(cache_lens=lens.long()), dict(page_table=table[:, ::2]),
                dict(page_table=table[0]), dict(cand_offsets=lens), dict(func_c=torch.zeros((3, 2), device="cuda").int()),
                dict(out=torch.zeros((1, 2, 64), dtype=torch.bfloat16, device="cuda")), dict(ws=torch.zeros(512).byte())):
        args = dict(q_c=q, cache=c, cache_lens=lens, page_table=table, max_seqlen=40)
        args.update(bad)
        with pytest.raises(ValueError):
            hb.fwd_paged(**args)
    with pytest.raises(hb.HstuError):  # an even number of interval rows
        hb.fwd_paged(q, c, lens, table, 40, func_c=torch.zeros((2, 1), device="cuda").int())
    k, v = q.new_zeros((3, 2, 64)), q.new_zeros((3, 2, 32))
    off = _int32([0, 3])
    for bad in (dict(k=v), dict(v=v[:2]), dict(k=k.half()), dict(seq_offsets=off.long()), dict(cache_lens=off),
                dict(positions=off), dict(rope=hb.rope_table(64, device="cpu"))):
        args = dict(cache=c, k=k, v=v, seq_offsets=off, cache_lens=lens, page_table=table)
        args.update(bad)
        with pytest.raises(ValueError):
            hb.cache_write(**args)
    with pytest.raises(hb.HstuError):  # the rotation is wider than the head
        hb.cache_write(c, k, v, off, lens, table, rope=hb.rope_table(128))
    with pytest.raises(ValueError):
        hb.cache_read(c, off, 3, table, outs=(k, k))
    elsewhere = hb.alloc_cache(2, 16, 2, 64, 32)
    elsewhere._device = torch.cuda.device_count()  # as if its tensors were on another device
    with pytest.raises(ValueError, match="current device"):
        hb.fwd_paged(q, elsewhere, lens, table, 40)
