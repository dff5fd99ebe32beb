"""The layer's row operators without a GPU: calls that are refused before
anything is enqueued, and sizes of workspaces."""
import ctypes

import pytest

from jagged_hstu_attention_gb300 import binding as hb
from jagged_hstu_attention_gb300 import build_ext

vp = ctypes.c_void_p


@pytest.fixture(scope="module")
def lib():
    build_ext.build()
    return hb.load()


def at(i):
    """An address of its own; never dereferenced: every call fails a host check."""
    return vp((i + 1) << 40)


def test_embed_refusals(lib):
    def status(**kw):
        a = dict(table=at(0), tdt=0, vocab=100, dim=64, ids=at(1), idb=4, tokens=5, scale=1.0, out=at(2), dt=0, ws=None,
                 wsb=0)
        a.update(kw)
        return lib.hstu_attn_embed(*a.values(), None)
    for kw, want in ((dict(tokens=-1), 1), (dict(vocab=0), 1), (dict(dim=0), 1), (dict(dim=12), 2), (dict(dim=65544), 2),
                     (dict(tdt=1), 2), (dict(dt=2), 2), (dict(idb=2), 2), (dict(table=None), 1), (dict(out=None), 1),
                     (dict(ids=None), 1), (dict(ids=vp((2 << 40) + 2)), 1), (dict(table=vp((1 << 40) + 8)), 1),
                     (dict(out=at(0)), 1), (dict(out=vp((1 << 40) + 128 * 99)), 1), (dict(out=at(1)), 1),
                     (dict(ws=vp(8), wsb=256), 3), (dict(ws=at(3), wsb=128), 3), (dict(tokens=1 << 31), 1),
                     (dict(vocab=(1 << 31) - 1), 1)):
        assert status(**kw) == want, kw
    assert status(tokens=0, table=None, ids=None, out=None) == 0


def test_embed_bwd_refusals(lib):
    def status(**kw):
        a = dict(dy=at(0), ds=64, dt=0, ids=at(1), idb=8, tokens=5, scale=1.0, out=at(2), gdt=2, vocab=100, dim=64, acc=0,
                 ws=at(3), wsb=1 << 30)
        a.update(kw)
        return lib.hstu_attn_embed_bwd(*a.values(), None)
    for kw, want in ((dict(ds=56), 1), (dict(ds=68), 1), (dict(dy=None), 1), (dict(out=None), 1), (dict(gdt=1), 2),
                     (dict(dt=2), 2), (dict(acc=2), 1), (dict(acc=1, gdt=0), 2), (dict(out=at(0)), 1),
                     (dict(out=at(1)), 1), (dict(ws=None), 3), (dict(wsb=256), 3), (dict(ws=vp((4 << 40) + 16)), 3),
                     (dict(ids=None), 1), (dict(dim=4), 2)):
        assert status(**kw) == want, kw
    size = lib.hstu_attn_embed_workspace_size
    assert size(-1, 10, 64) == 0 and size(5, 0, 64) == 0 and size(5, 10, 12) == 0
    assert 0 < size(0, 1, 8) <= size(100, 1000, 64) <= size(1 << 20, 1 << 30, 64)


def test_norm_refusals(lib):
    def status(**kw):
        a = dict(x=at(0), xs=64, r=at(1), rs=64, g=at(2), gs=64, w=at(3), rows=5, width=64, dt=0, eps=1e-6, y=at(4),
                 sc=None, h=at(5), rstd=at(6))
        a.update(kw)
        return lib.hstu_attn_rms_norm(*a.values(), None)
    for kw, want in ((dict(rows=-1), 1), (dict(width=0), 1), (dict(width=12), 2), (dict(width=8200), 2), (dict(dt=2), 2),
                     (dict(eps=-1.0), 1), (dict(eps=float("nan")), 1), (dict(eps=float("inf")), 1), (dict(x=None), 1),
                     (dict(xs=56), 1), (dict(gs=66), 1), (dict(h=None), 1), (dict(r=None), 1), (dict(y=None), 1),
                     (dict(w=None), 1), (dict(y=at(0)), 1), (dict(y=at(5)), 1), (dict(rstd=at(4)), 1),
                     (dict(rstd=vp(2)), 1), (dict(h=at(1), rs=72), 1), (dict(h=at(2)), 1), (dict(sc=at(4)), 1),
                     (dict(h=vp((2 << 40) + 128)), 1)):
        assert status(**kw) == want, kw
    assert status(rows=0, x=None, y=None) == 0

    def codes(**kw):
        a = dict(x=at(0), xs=64, rows=5, width=64, dt=0, c=at(1), s=at(2))
        a.update(kw)
        return lib.hstu_attn_quantise_rows(*a.values(), None)
    for kw, want in ((dict(width=20), 2), (dict(x=None), 1), (dict(c=None), 1), (dict(s=None), 1), (dict(c=at(0)), 1),
                     (dict(s=vp((2 << 40) + 8)), 1), (dict(dt=3), 2), (dict(rows=-2), 1)):
        assert codes(**kw) == want, kw


def test_norm_bwd_refusals(lib):
    def status(**kw):
        a = dict(dy=at(0), ds=64, h=at(1), hs=64, rstd=at(2), w=at(3), g=at(4), gs=64, e=at(5), es=64, rows=5, width=64,
                 dt=1, dx=at(6), dw=at(7), dg=at(8), ws=at(9), wsb=1 << 30)
        a.update(kw)
        return lib.hstu_attn_rms_norm_bwd(*a.values(), None)
    for kw, want in ((dict(dw=None), 1), (dict(dx=None), 1), (dict(dg=None), 1), (dict(g=None), 1), (dict(rstd=None), 1),
                     (dict(dx=at(0)), 1), (dict(dg=at(6)), 1), (dict(dw=at(3)), 1), (dict(es=60), 1), (dict(ws=None), 3),
                     (dict(wsb=4), 3), (dict(dt=2), 2), (dict(width=8200), 2)):
        assert status(**kw) == want, kw
    size = lib.hstu_attn_rms_norm_workspace_size
    assert size(-1, 64) == 0 and size(5, 12) == 0 and 0 < size(0, 8) <= size(1 << 30, 8192) < 1 << 26


def test_linear_refusals(lib):
    def status(**kw):
        a = dict(x=at(0), xs=64, xsc=None, w=at(1), wsc=None, b=at(2), r=at(3), rs=72, rows=5, k=64, n=72, dt=0, act=1,
                 y=at(4), z=at(5), ws=None, wsb=0)
        a.update(kw)
        return lib.hstu_attn_linear(*a.values(), None)
    for kw, want in ((dict(rows=-1), 1), (dict(rows=(1 << 31) - 1), 1), (dict(k=0), 1), (dict(k=60), 2), (dict(n=60), 2),
                     (dict(k=65544), 2), (dict(dt=2), 2), (dict(act=4), 2), (dict(act=-1), 2), (dict(x=None), 1),
                     (dict(xs=56), 1), (dict(xs=68), 1), (dict(w=None), 1), (dict(xsc=at(6)), 1), (dict(wsc=at(6)), 1),
                     (dict(xsc=at(6), wsc=at(7), k=72, xs=72), 2), (dict(xsc=at(6), wsc=at(7), xs=72), 1),
                     (dict(rs=64), 1), (dict(b=vp(8)), 1), (dict(y=at(3)), 1), (dict(z=at(4)), 1), (dict(y=at(1)), 1),
                     (dict(y=None), 1), (dict(z=at(0)), 1), (dict(ws=at(8), wsb=8), 3),
                     (dict(rows=1 << 30, n=65536), 2)):
        assert status(**kw) == want, kw


def test_linear_bwd_refusals(lib):
    def status(**kw):
        a = dict(dy=at(0), ds=72, z=at(1), x=at(2), xs=64, w=at(3), rows=5, k=64, n=72, dt=0, act=1, dx=at(4), dw=at(5),
                 db=at(6), ws=at(7), wsb=1 << 30)
        a.update(kw)
        return lib.hstu_attn_linear_bwd(*a.values(), None)
    for kw, want in ((dict(z=None), 1), (dict(dx=None), 1), (dict(dw=None), 1), (dict(ds=64), 1), (dict(xs=60), 1),
                     (dict(dx=at(0)), 1), (dict(dw=at(3)), 1), (dict(db=at(4)), 1), (dict(ws=None), 3), (dict(wsb=256), 3),
                     (dict(k=12), 2), (dict(act=5), 2), (dict(db=vp(4)), 1)):
        assert status(**kw) == want, kw
    size = lib.hstu_attn_linear_workspace_size
    assert size(-1, 64, 64, 0) == 0 and size(5, 60, 64, 0) == 0 and size(5, 64, 64, 7) == 0
    assert 0 < size(0, 8, 8, 0) <= size(1000, 64, 64, 0) < size(1000, 64, 64, 1)


@pytest.mark.parametrize("dims", [(8, 8), (16, 40), (64, 512), (512, 64), (504, 2056), (512, 2048), (1128, 640),
                                  (2048, 2048), (2048, 8192), (8192, 200), (65536, 8), (8, 65536)])
def test_workspaces_of_more_rows_serve_fewer(lib, dims):
    """Sizes never fall as the rows grow, one by one at first and across the larger counts."""
    a, b = dims
    counts = list(range(1, 700)) + sorted({int(700 * 1.013 ** k) + d for k in range(560) for d in (-1, 0, 1)})
    for size in (lambda n: lib.hstu_attn_linear_workspace_size(n, a, b, 1),
                 lambda n: lib.hstu_attn_linear_workspace_size(n, a, b, 0),
                 lambda n: lib.hstu_attn_embed_workspace_size(n, 1000, a),
                 lambda n: lib.hstu_attn_rms_norm_workspace_size(n, min(a, 8192))):
        sizes = [size(n) for n in counts]
        assert sizes[0] > 0 and all(x <= y for x, y in zip(sizes, sizes[1:]))
