"""Plain 64-bit forms of the serving operators (rotary positions, the paged
cache, candidate rows against it) and the error bounds their tests use."""
import math

import numpy as np
import torch

from jagged_hstu_attention_gb300 import binding as hb
from jagged_hstu_attention_gb300 import workloads as wl

E4M3_MAX = 448.0


def f64(t):
    """A 16- or 32-bit float tensor as a 64-bit host array."""
    return t.detach().float().cpu().numpy().astype(np.float64)


def half_step(dtype):
    """Relative error of one rounding to nearest."""
    return torch.finfo(dtype).eps / 2


def smallest_half_step(dtype):
    """Absolute error of one rounding below the normal range."""
    return torch.finfo(dtype).smallest_normal * torch.finfo(dtype).eps / 2


def frequencies(rotary, base=10000.0, scaling="none", factor=1.0, original_len=0, fast=32.0, slow=1.0):
    """(radians a position of each pair, magnitude), from the definition."""
    if scaling == "ntk":
        base = base * factor ** (rotary / (rotary - 2))
    f = np.array([base ** (-2.0 * i / rotary) for i in range(rotary // 2)])
    if scaling == "linear":
        f = f / factor
    if scaling == "yarn":
        r = original_len * f / (2 * math.pi)
        keep = np.clip((r - slow) / (fast - slow), 0.0, 1.0)
        return f * keep + f / factor * (1 - keep), 0.1 * math.log(factor) + 1.0
    return f, 1.0


def rotate(x, positions, f, magnitude=1.0, interleaved=False, backward=False):
    """(rows, H, D) 64-bit rows rotated pair by pair."""
    y = np.array(x, dtype=np.float64)
    n = len(f)
    a = np.arange(0, 2 * n, 2) if interleaved else np.arange(n)
    b = a + (1 if interleaved else n)
    angle = np.outer(np.asarray(positions, dtype=np.float64), f)[:, None, :]
    c, s = magnitude * np.cos(angle), magnitude * np.sin(angle) * (-1.0 if backward else 1.0)
    u, v = x[..., a], x[..., b]
    y[..., a], y[..., b] = u * c - v * s, v * c + u * s
    return y


def rotate_slack(x, f, magnitude=1.0, interleaved=False):
    """Error of the rotation in fp32 before its rounding: cosine and sine are
    within 2^-23 (series and argument rounding 2^-24 each, phase 2^-32 turns),
    the two products and their sum add 2^-24 each, so 2^-21 of |x| + |y|
    covers all of it."""
    n = len(f)
    a = np.arange(0, 2 * n, 2) if interleaved else np.arange(n)
    b = a + (1 if interleaved else n)
    out = np.zeros(x.shape)
    both = np.abs(x[..., a]) + np.abs(x[..., b])
    out[..., a] = out[..., b] = magnitude * 2.0 ** -21 * both
    return out


def e4m3_round(y):
    """64-bit values to the nearest 8-bit float (ties to even), |y| <= 448."""
    e = np.floor(np.log2(np.maximum(np.abs(y), 2.0 ** -6)))
    step = 2.0 ** (e - 3)
    return np.rint(y / step) * step


def quantise(x):
    """(values the codes stand for, scale exponents) of 64-bit rows (..., width)."""
    fine = np.isfinite(x)
    top = np.where(fine, np.abs(x), 0.0).max(-1)
    e = np.full(top.shape, -127.0)
    some = top > 0
    e[some] = np.ceil(np.log2(top[some] / E4M3_MAX))
    # log2 rounds: settle the power by comparing
    e = np.where(some & (top > E4M3_MAX * 2.0 ** e), e + 1, e)
    e = np.where(some & (top <= E4M3_MAX * 2.0 ** (e - 1)), e - 1, e)
    e = np.maximum(e, -127.0)
    scale = 2.0 ** e[..., None]
    with np.errstate(invalid="ignore"):
        v = e4m3_round(np.where(fine, x, 0.0) / scale) * scale
    return np.where(fine, v, np.nan), e


class Pages:
    """A paged cache with poisoned slots, its page table and host copies."""

    def __init__(self, lens, heads, dim, dim_v, page, dtype, quantised, seed=0, spare=3, extra_pages=0):
        self.lens = [int(n) for n in lens]
        need = [(n + page - 1) // page for n in self.lens]
        self.max_pages = max(1, max(need) + extra_pages)
        rng = np.random.default_rng(seed)
        order = rng.permutation(sum(need) + spare + extra_pages * len(need))
        table = np.full((len(need), self.max_pages), -1, dtype=np.int32)  # entries past the end are never read
        at = 0
        for b, n in enumerate(need):
            table[b, :n + extra_pages] = order[at:at + n + extra_pages]
            at += n + extra_pages
        self.table = table
        self.page, self.heads, self.dim, self.dim_v, self.dtype, self.quantised = page, heads, dim, dim_v, dtype, quantised
        self.num_pages = len(order)
        self.cache = hb.alloc_cache(self.num_pages, page, heads, dim, dim_v, dtype=dtype, quantised=quantised)
        self.poison()
        self.d_table = torch.tensor(table, device="cuda")
        self.d_lens = torch.tensor(self.lens, dtype=torch.int32, device="cuda")

    def poison(self):
        """Every slot NaN, every scale infinite."""
        c = self.cache
        for t in (c.k, c.v):
            t.fill_(0x7f if self.quantised else float("nan"))
        if self.quantised:
            c.k_scale.fill_(255)
            c.v_scale.fill_(255)

    def places(self, b, first, n):
        pos = np.arange(first, first + n)
        return self.table[b, pos // self.page], pos % self.page

    def fill(self, rng):
        """N(0, 1) rows at every cached position, put there from the host; returns
        the 64-bit values (k, v) of each sequence."""
        out = []
        c = self.cache
        for b, n in enumerate(self.lens):
            page, slot = self.places(b, 0, n)
            got = []
            for t, scale, w in ((c.k, c.k_scale, self.dim), (c.v, c.v_scale, self.dim_v)):
                x = rng.standard_normal((n, self.heads, w))
                if self.quantised:
                    e = rng.integers(-9, -5, size=(n, self.heads))
                    codes = torch.tensor(np.clip(x * 2.0 ** 7, -448, 448), dtype=torch.float32).to(torch.float8_e4m3fn)
                    val = codes.double().numpy() * 2.0 ** e[..., None]
                    t[page, :, slot] = codes.view(torch.uint8).cuda()
                    scale[page, :, slot] = torch.tensor(e + 127, dtype=torch.uint8).cuda()
                else:
                    rows = torch.tensor(x).to(self.dtype)
                    val = f64(rows)
                    t[page, :, slot] = rows.cuda()
                got.append(val)
            out.append(tuple(got))
        return out


def silu(x):
    with np.errstate(over="ignore"):
        return x / (1.0 + np.exp(-x))


def visible(func_col, n):
    m = np.zeros(n, dtype=bool)
    if func_col is None:
        return ~m
    for i in range((len(func_col) + 1) // 2):
        lo, hi = (0 if i == 0 else int(func_col[2 * i - 1])), int(func_col[2 * i])
        m[max(lo, 0):max(min(hi, n), 0)] = True
    return m


def paged_reference(q, rows, counts, func, max_seqlen, alpha, dtype):
    """(o, bound) for candidate rows q (C, H, D) against per-sequence (k, v)
    rows; ``func`` is (nfunc, C) or None.

    The bound, element by element: the output's rounding; the scores' sums of D
    products in fp32 (blocks of 16 terms, each addition within 2^-22 of the
    sum of magnitudes), which silu, of slope at most 1.1, passes on; the
    weights' relative error (their two 16-bit parts hold 18 bits, the
    exponential and the quotient are within 2^-19 for the scores met here);
    and the additions of the weighted rows."""
    o, tol, c = [], [], 0
    for (k, v), n in zip(rows, counts):
        L = k.shape[0]
        for _ in range(n):
            see = visible(None if func is None else func[:, c], L)
            kk, vv = k[see], v[see]
            x = alpha * np.einsum("hd,lhd->lh", q[c], kk)
            mag = abs(alpha) * np.einsum("hd,lhd->lh", np.abs(q[c]), np.abs(kk))
            p = silu(x)
            o.append(np.einsum("lh,lhd->hd", p, vv) / max_seqlen)
            c1 = 2.0 ** -17 + (L / 64 + 16) * 2.0 ** -22
            c2 = 1.1 * (q.shape[2] / 16 + 4) * 2.0 ** -22
            tol.append(np.einsum("lh,lhd->hd", c1 * np.abs(p) + c2 * mag, np.abs(vv)) / max_seqlen)
            c += 1
    o, tol = np.array(o), np.array(tol)
    return o, tol + half_step(dtype) * np.abs(o) * 1.01 + smallest_half_step(dtype)


def rows_of(shape, g, dtype):
    return wl.randn(shape, g, dtype=dtype).cuda()
