"""Serving entry points without a GPU: the frequency table against its
definition, and the calls that are refused before anything is enqueued."""
import ctypes
import math

import numpy as np
import pytest
import torch

from jagged_hstu_attention_gb300 import binding as hb
from jagged_hstu_attention_gb300 import build_ext
import serving_testutil as su


@pytest.fixture(scope="module")
def lib():
    build_ext.build()
    return hb.load()


vp = ctypes.c_void_p
FAKE = vp(1 << 20)  # never dereferenced: every case fails a host check


@pytest.mark.parametrize("R", [16, 48, 64, 128])
@pytest.mark.parametrize("scaling", ["none", "linear", "ntk", "yarn"])
def test_rope_table_is_the_definition(lib, R, scaling):
    t = hb.rope_table(R, base=20000.0, scaling=scaling, factor=4.0, original_len=2048, device="cpu")
    f, m = su.frequencies(R, 20000.0, scaling, 4.0, 2048)
    turns = t.turns.numpy().view(np.uint64).astype(np.float64) / 2.0 ** 64
    # a power, a quotient and a blend of 64-bit values: a few 2^-53 each; and
    # the cut to whole units of 2^-64 turns, 2 pi 2^-64 radians at the most
    assert np.all(np.abs(turns * 2 * math.pi - f) <= 16 * 2.0 ** -53 * f + 2 * math.pi * 2.0 ** -64)
    assert abs(t.magnitude - m) <= 2.0 ** -24 * m and t.rotary_dim == R


def test_rope_table_refusals(lib):
    def status(**kw):
        a = dict(rotary_dim=64, scaling=0, base=1e4, factor=2.0, original_len=100.0, fast=32.0, slow=1.0)
        a.update(kw)
        spec = hb.RopeSpec(a["rotary_dim"], a["scaling"], a["base"], a["factor"], a["original_len"], a["fast"],
                           a["slow"])
        turns, mag = (ctypes.c_uint64 * 64)(), ctypes.c_float()
        return lib.hstu_attn_rope_table(ctypes.byref(spec), turns, ctypes.byref(mag))
    assert status() == 0 and status(scaling=3) == 0
    for kw in (dict(rotary_dim=0), dict(rotary_dim=8), dict(rotary_dim=24), dict(rotary_dim=144), dict(rotary_dim=-16),
               dict(scaling=4), dict(scaling=-1)):
        assert status(**kw) == 2, kw
    nan, inf = float("nan"), float("inf")
    for kw in (dict(base=1.0), dict(base=nan), dict(base=inf), dict(scaling=1, factor=0.5), dict(scaling=2, factor=nan),
               dict(scaling=2, factor=inf), dict(scaling=3, original_len=0.0), dict(scaling=3, fast=1.0),
               dict(scaling=3, slow=0.0), dict(scaling=3, fast=inf), dict(scaling=2, base=1e300, factor=1e300)):
        assert status(**kw) == 1, kw
    assert lib.hstu_attn_rope_table(None, None, None) == 1
    with pytest.raises(ValueError, match="scaling"):
        hb.rope_table(64, scaling="cubic", device="cpu")


def _rope(lib, rope=None, q=vp(1 << 21), qs=256, k=vp(1 << 22), ks=256, qo=vp(1 << 23), qos=256, ko=vp(1 << 24),
          kos=256, pos=FAKE, tokens=5, H=4,
          D=64, dtype=0, R=64, inter=0, mag=1.0, turns=1 << 20):
    r = hb.Rope(turns, R, inter, mag) if rope is None else rope
    return lib.hstu_attn_rope(q, qs, k, ks, qo, qos, ko, kos, pos, tokens, H, D, dtype,
                              ctypes.byref(r) if r else None, 0, None)


def test_rope_refusals(lib):
    for kw in (dict(D=96), dict(D=256), dict(dtype=2), dict(R=24), dict(R=0), dict(R=128), dict(H=70000)):
        assert _rope(lib, **kw) == 2, kw
    for kw in (dict(rope=False), dict(turns=0), dict(turns=(1 << 20) + 4), dict(inter=2), dict(mag=float("nan")),
               dict(q=None), dict(q=vp((1 << 20) + 8)), dict(qs=248), dict(qs=260), dict(qo=None), dict(ko=None),
               dict(kos=128), dict(ks=257), dict(pos=None), dict(pos=vp((1 << 20) + 2)), dict(tokens=-1),
               dict(tokens=1 << 31), dict(H=0), dict(qo=vp(1 << 21), qos=512),
               # outputs that another input or output shares
               dict(ko=vp(1 << 23)), dict(qo=vp(1 << 22)), dict(ko=vp(1 << 21))):
        assert _rope(lib, **kw) == 1, kw
    assert _rope(lib, tokens=0, q=None, qo=None, k=None, pos=None) == 0


def _cache(**kw):
    a = dict(k=1 << 20, v=1 << 20, ks=None, vs=None, pages=10, page=64, H=4, D=64, Dv=0, dtype=0, e4m3=0)
    a.update(kw)
    return hb.Cache(a["k"], a["v"], a["ks"], a["vs"], a["pages"], a["page"], a["H"], a["D"], a["Dv"], a["dtype"],
                    a["e4m3"])


BAD_CACHES = [
    (dict(D=48), 2), (dict(Dv=256), 2), (dict(dtype=3), 2), (dict(page=8), 2), (dict(page=48), 2),
    (dict(page=512), 2), (dict(page=0), 2), (dict(H=0), 1), (dict(H=70000), 2), (dict(pages=0), 1),
    (dict(pages=1 << 31), 1), (dict(k=None), 1), (dict(v=(1 << 20) + 4), 1), (dict(e4m3=1), 1),
    (dict(e4m3=2, ks=1 << 20, vs=1 << 20), 1),
]


def _write(lib, cache=None, k=FAKE, ks=256, v=FAKE, vs=256, off=FAKE, B=3, rows=9, lens=FAKE, table=FAKE, width=4,
           rope=None, pos=None, ws=None, wsb=0):
    c = cache if cache is not None else _cache()
    return lib.hstu_attn_cache_write(ctypes.byref(c), k, ks, v, vs, off, B, rows, lens, table, width,
                                     ctypes.byref(rope) if rope else None, pos, ws, wsb, None)


def test_cache_write_refusals(lib):
    for kw, want in BAD_CACHES:
        assert _write(lib, cache=_cache(**kw)) == want, kw
    rope = hb.Rope(1 << 20, 64, 0, 1.0)
    for kw in (dict(k=None), dict(k=vp((1 << 20) + 2)), dict(ks=255), dict(vs=128), dict(v=None), dict(off=None),
               dict(off=vp((1 << 20) + 1)), dict(B=0), dict(rows=-1), dict(rows=1 << 31), dict(lens=None),
               dict(table=None), dict(width=0), dict(pos=FAKE), dict(rope=rope, pos=vp((1 << 20) + 2)),
               dict(rope=hb.Rope(0, 64, 0, 1.0))):
        assert _write(lib, **kw) == 1, kw
    assert _write(lib, rope=hb.Rope(1 << 20, 128, 0, 1.0)) == 2  # wider than the head
    assert _write(lib, ws=FAKE, wsb=255) == 3 and _write(lib, ws=vp((1 << 20) + 64), wsb=256) == 3
    assert _write(lib, rows=0, k=None, v=None) == 0
    assert lib.hstu_attn_cache_write(None, FAKE, 256, FAKE, 256, FAKE, 1, 1, FAKE, FAKE, 1, None, None, None, 0,
                                     None) == 1


def test_cache_read_refusals(lib):
    def read(cache=None, k=FAKE, v=FAKE, off=FAKE, B=3, rows=9, starts=None, table=FAKE, width=4, ws=None, wsb=0):
        c = cache if cache is not None else _cache()
        return lib.hstu_attn_cache_read(ctypes.byref(c), k, v, off, B, rows, starts, table, width, ws, wsb, None)
    for kw, want in BAD_CACHES:
        assert read(cache=_cache(**kw)) == want, kw
    for kw in (dict(k=None), dict(v=vp((1 << 20) + 8)), dict(off=None), dict(B=0), dict(rows=-1),
               dict(starts=vp((1 << 20) + 2)), dict(table=None), dict(width=0)):
        assert read(**kw) == 1, kw
    assert read(ws=FAKE, wsb=16) == 3
    assert read(rows=0, k=None, v=None) == 0


def test_paged_refusals(lib):
    def paged(cache=None, q=FAKE, qs=256, o=vp(1 << 21), lens=FAKE, B=3, table=FAKE, width=4, coff=FAKE, C=7, func=None,
              nfunc=0, N=1000, alpha=0.1, ws=FAKE, wsb=1 << 30, flags=0):
        c = cache if cache is not None else _cache()
        return lib.hstu_attn_fwd_paged(q, qs, o, ctypes.byref(c), lens, B, table, width, coff, C, func, nfunc, N,
                                       alpha, ws, wsb, flags, None)
    for kw, want in BAD_CACHES:
        assert paged(cache=_cache(**kw)) == want, kw
        assert lib.hstu_attn_paged_workspace_size(ctypes.byref(_cache(**kw)), 3, 7, 1000) == 0
    for kw in (dict(q=vp(1 << 21)), dict(q=None), dict(q=vp((1 << 20) + 8)), dict(qs=254), dict(qs=260), dict(o=None),
               dict(o=vp((1 << 20) + 4)), dict(lens=None), dict(lens=vp((1 << 20) + 2)), dict(B=0), dict(table=None),
               dict(width=0), dict(coff=None), dict(coff=vp((1 << 20) + 2)), dict(C=-1), dict(C=1 << 31),
               dict(func=vp((1 << 20) + 2), nfunc=3), dict(N=0), dict(alpha=float("nan"))):
        assert paged(**kw) == 1, kw
    for kw in (dict(func=FAKE, nfunc=2), dict(func=FAKE, nfunc=11), dict(N=(1 << 24) + 1),
               dict(cache=_cache(H=60000), B=1 << 20)):
        assert paged(**kw) == 2, kw
    assert paged(ws=None, flags=2) == 3 and paged(ws=None, N=100) == 3 and paged(ws=None) == 3 and paged(ws=vp((1 << 20) + 64)) == 3 and paged(wsb=64) == 3
    size = lib.hstu_attn_paged_workspace_size(ctypes.byref(_cache()), 3, 7, 1000)
    assert size > 256 and paged(wsb=size - 1) == 3  # the sums of several splits
    assert lib.hstu_attn_paged_workspace_size(ctypes.byref(_cache()), 3, 7, 100) == 256
    assert lib.hstu_attn_paged_workspace_size(None, 3, 7, 1000) == 0


def test_a_paged_workspace_serves_fewer_candidates(lib):
    for kw in (dict(), dict(D=128, Dv=128), dict(D=128, Dv=128, dtype=1), dict(D=128, Dv=32),
               dict(D=128, e4m3=1, ks=1 << 20, vs=1 << 20, dtype=1)):
        for B in (1, 7, 300):
            for N in (1, 256, 300, 512, 513, 1100, 20000, 1 << 20):
                sizes = [lib.hstu_attn_paged_workspace_size(ctypes.byref(_cache(**kw)), B, C, N)
                         for C in (0, B, 8 * B, 8 * B + 1, 16 * B, 16 * B + 1, 17 * B + 3, 40 * B, 64 * B)]
                assert sizes[0] >= 256 and sizes == sorted(sizes), (kw, B, N, sizes)


def test_binding_checks_its_tensors(lib):
    q = torch.zeros((4, 2, 64), dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA"):
        hb.rope(q, None, torch.zeros(4, dtype=torch.int32), hb.rope_table(64, device="cpu"))
    with pytest.raises(ValueError, match="must be one of"):
        hb.rope(q.float(), None, torch.zeros(4, dtype=torch.int32), hb.rope_table(64, device="cpu"))
    with pytest.raises(ValueError, match="CUDA"):
        hb.PagedCache(torch.zeros((2, 2, 16, 64), dtype=torch.bfloat16), torch.zeros((2, 2, 16, 64), dtype=torch.bfloat16))
