"""Cases that measure the serving-side operators: rotary positions, the paged
K/V cache (written, quantised and read back) and the attention of candidate
rows over it.

Each case names one operator (``op``) and its sizes; ``run`` is one pass of it,
in elementary torch operations or, where ``own`` is set, through the calls that
a program makes of this package. The lengths of a case's sequences follow from
the case alone, its tensors from the case and a seed.

  rope   rotates q and k by their positions (and, for training, the gradients
         back).
  cache  appends new K/V rows to the pages of their sequences: 16-bit pages
         (the buffers come back), or 8-bit pages with a power-of-two scale for
         each row and head, of which rows are then read back.
  paged  pointwise-SiLU attention of each sequence's candidate rows over its
         cached rows.
"""
import math
import random

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16}
CHUNK_NEW = 256


def _dev():
    return "cuda" if torch.cuda.is_available() else "cpu"


# ------------------------------------------------------------------- cases


def listed():
    return [
        # One new token for each of 64 users: q and k of a single decode step.
        {"name": "rope_step", "op": "rope", "tokens": 64, "heads": 4, "dim": 128, "rotary": 128, "layout": "half",
         "scaling": "none", "dtype": "bf16", "far": 2048, "train": False, "fused": False},
        # A training batch of the OneRank shape (64 sequences of 512 to 2048 rows): forward and backward.
        {"name": "rope_train", "op": "rope", "tokens": 81920, "heads": 4, "dim": 128, "rotary": 128, "layout": "half",
         "scaling": "none", "dtype": "bf16", "far": 2048, "train": True, "fused": False},
        # A long prompt, fp16, half of each head rotated in interleaved pairs, positions far past the trained
        # length (scaled frequencies), q and k as slices of one projection's output rows.
        {"name": "rope_long_f16", "op": "rope", "tokens": 32749, "heads": 8, "dim": 128, "rotary": 64,
         "layout": "interleaved", "scaling": "yarn", "dtype": "f16", "far": 1 << 20, "train": False, "fused": True},
        # One new token for each of 64 users into 8-bit pages, the new rows read back.
        {"name": "cache_step_e4m3", "op": "cache", "batch": 64, "hist_lo": 512, "hist_hi": 2048, "new_lo": 1, "new_hi": 1,
         "heads": 4, "dim": 128, "dim_v": 128, "page": 64, "dtype": "bf16", "quantised": True, "rotary": 0,
         "back": "new"},
        # Prompts of the OneRank lengths into 16-bit pages, k rotated on its way.
        {"name": "cache_prompt_bf16", "op": "cache", "batch": 64, "hist_lo": 0, "hist_hi": 0, "new_lo": 512,
         "new_hi": 2048, "heads": 4, "dim": 128, "dim_v": 128, "page": 64, "dtype": "bf16", "quantised": False,
         "rotary": 128, "back": "none"},
        # A chunk of new rows behind histories of the DLRM lengths, 8-bit pages; the whole sequences are read
        # back for the contiguous attention kernels.
        {"name": "cache_chunk_e4m3", "op": "cache", "batch": 32, "hist_lo": 1332, "hist_hi": 3994, "new_lo": 1,
         "new_hi": CHUNK_NEW, "heads": 4, "dim": 128, "dim_v": 128, "page": 128, "dtype": "bf16", "quantised": True,
         "rotary": 0, "back": "all"},
        # The smallest service call: four short sequences, narrow heads.
        {"name": "paged_tiny", "op": "paged", "batch": 4, "len_lo": 16, "len_hi": 64, "cand_lo": 1, "cand_hi": 1,
         "heads": 2, "dim": 32, "dim_v": 32, "page": 16, "dtype": "bf16", "quantised": False, "mask": "none"},
        # One new token for each of 256 users with histories of the DLRM lengths, 16-bit pages.
        {"name": "paged_dlrm_bf16", "op": "paged", "batch": 256, "len_lo": 1332, "len_hi": 3994, "cand_lo": 1,
         "cand_hi": 1, "heads": 4, "dim": 128, "dim_v": 128, "page": 64, "dtype": "bf16", "quantised": False,
         "mask": "none"},
        # The same over 8-bit pages.
        {"name": "paged_dlrm_e4m3", "op": "paged", "batch": 256, "len_lo": 1332, "len_hi": 3994, "cand_lo": 1,
         "cand_hi": 1, "heads": 4, "dim": 128, "dim_v": 128, "page": 64, "dtype": "bf16", "quantised": True,
         "mask": "none"},
        # One user with a very long history: the cache's length is all there is to split.
        {"name": "paged_long_e4m3", "op": "paged", "batch": 1, "len_lo": 32749, "len_hi": 32749, "cand_lo": 1,
         "cand_hi": 1, "heads": 4, "dim": 128, "dim_v": 128, "page": 256, "dtype": "f16", "quantised": True,
         "mask": "none"},
        # Ranking: up to 48 candidates for each of 64 users; a candidate sees the history and itself.
        {"name": "paged_cands_bf16", "op": "paged", "batch": 64, "len_lo": 512, "len_hi": 2048, "cand_lo": 0,
         "cand_hi": 48, "heads": 4, "dim": 128, "dim_v": 128, "page": 64, "dtype": "bf16", "quantised": False,
         "mask": "self"},
        # The SLA mask (256 columns of prefix, a window of 32) at a single new row: most pages are not read.
        {"name": "paged_sla_f16", "op": "paged", "batch": 128, "len_lo": 1024, "len_hi": 2048, "cand_lo": 1,
         "cand_hi": 1, "heads": 8, "dim": 64, "dim_v": 128, "page": 32, "dtype": "f16", "quantised": False,
         "mask": "sla"},
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    heads, dim, dim_v = rng.choice([1, 2, 3, 4, 8]), rng.choice([32, 64, 128, 128]), rng.choice([32, 64, 128, 128])
    dtype, page = rng.choice(["bf16", "f16"]), rng.choice([16, 32, 64, 128, 256])
    op = rng.choice(["rope", "cache", "paged", "paged"])
    if op == "rope":
        c = {"op": op, "tokens": _log_int(rng, 1, 131072), "heads": heads, "dim": dim,
             "rotary": rng.choice([r for r in range(16, dim + 1, 16)] + [dim]),
             "layout": rng.choice(["half", "interleaved"]), "scaling": rng.choice(["none", "linear", "ntk", "yarn"]),
             "dtype": dtype, "far": _log_int(rng, 64, 1 << 20), "train": rng.random() < 0.5,
             "fused": rng.random() < 0.5}
        grow = "tokens"
    elif op == "cache":
        quantised = rng.random() < 0.5
        hist, new = rng.choice([0, _log_int(rng, 1, 4096)]), _log_int(rng, 1, 2048)
        c = {"op": op, "batch": _log_int(rng, 1, 128), "hist_lo": hist // 2, "hist_hi": hist,
             "new_lo": rng.choice([0, 1, (new + 1) // 2]), "new_hi": new, "heads": heads, "dim": dim, "dim_v": dim_v,
             "page": page, "dtype": dtype, "quantised": quantised,
             "rotary": 0 if quantised else rng.choice([0, 16, dim]), "back": rng.choice(["new", "all"]) if quantised else "none"}
        c["new_lo"] = max(1, min(c["new_lo"], new)) if c["batch"] == 1 else min(c["new_lo"], new)
        grow = "batch"
    else:
        length, cands = _log_int(rng, 1, 32768), rng.choice([1, 1, _log_int(rng, 2, 48)])
        c = {"op": op, "batch": _log_int(rng, 1, 256), "len_lo": rng.choice([(length + 1) // 2, length]),
             "len_hi": length, "cand_lo": 1 if cands == 1 else rng.choice([0, 1, cands]), "cand_hi": cands,
             "heads": heads, "dim": dim, "dim_v": dim_v, "page": page, "dtype": dtype,
             "quantised": rng.random() < 0.5, "mask": "self" if cands > 1 else rng.choice(["none", "none", "sla"])}
        if c["batch"] == 1:
            c["cand_lo"] = max(1, c["cand_lo"])
        grow = "batch"
    while c[grow] > 1 and _cost(c) > 1.0e9:
        c[grow] = (c[grow] + 1) // 2
    return c


def _cost(c):
    """Bytes that bound a case from above, whatever its mask."""
    if c["op"] == "rope":
        return c["tokens"] * c["heads"] * c["dim"] * 8 * (2 if c["train"] else 1)
    rows = c["batch"] * (c["hist_hi"] + c["new_hi"] if c["op"] == "cache" else c["len_hi"] + c["cand_hi"])
    return rows * c["heads"] * (c["dim"] + c["dim_v"]) * (4 if c["op"] == "cache" else 2)


def _between(c, what, lo, hi, n):
    """n whole numbers from lo to hi that follow from the case alone."""
    r = random.Random("%s %d %d %d" % (what, lo, hi, c["batch"]))
    return [r.randint(lo, hi) for _ in range(n)]


def _lengths(c):
    """(rows before, rows added) of each sequence of a cache case; (history, candidates) of a paged one."""
    if c["op"] == "cache":
        first, second = ("hist_lo", "hist_hi"), ("new_lo", "new_hi")
    else:
        first, second = ("len_lo", "len_hi"), ("cand_lo", "cand_hi")
    a = _between(c, "rows", c[first[0]], c[first[1]], c["batch"])
    b = _between(c, "added", c[second[0]], c[second[1]], c["batch"])
    if not any(b):
        b[-1] = c[second[1]]
    return a, b


def _cached(c):
    """Rows in the cache of each sequence when a paged case runs: candidates that see themselves have a row there."""
    hist, cands = _lengths(c)
    return [h + n for h, n in zip(hist, cands)] if c["mask"] == "self" else hist


def work(case):
    c = case
    e = 2
    if c["op"] == "rope":
        n = c["tokens"] * c["heads"] * c["dim"]
        passes = 2 if c["train"] else 1
        return {"bytes": passes * (4 * n * e + 4 * c["tokens"]),
                "flops": passes * 6 * c["tokens"] * c["heads"] * c["rotary"]}
    width = c["dim"] + c["dim_v"]
    row = c["heads"] * (width + 2 if c["quantised"] else width * e)  # bytes of a cached row, its scales among them
    if c["op"] == "cache":
        hist, new = _lengths(c)
        n = sum(new)
        total = n * c["heads"] * width * e + n * row
        if c["back"] != "none":
            back = n if c["back"] == "new" else n + sum(hist)
            total += back * c["heads"] * width * e + (back - n) * row
        return {"bytes": total, "flops": n * c["heads"] * (3 * width + 3 * c["rotary"])}
    hist, cands = _lengths(c)
    read = pairs = 0
    for full, h, n in zip(_cached(c), hist, cands):
        if c["mask"] == "sla":
            seen = min(256, full) + min(32, max(0, full - 256))
            read, pairs = read + (seen if n else 0), pairs + n * seen
        elif c["mask"] == "self":
            read, pairs = read + (full if n else 0), pairs + n * (h + 1)
        else:
            read, pairs = read + (full if n else 0), pairs + n * full
    return {"bytes": read * row + sum(cands) * c["heads"] * width * e, "flops": 2 * pairs * c["heads"] * width}


# ------------------------------------------------------------------ inputs


def _frequencies(rotary, scaling):
    """(radians a position for each pair in 64 bits, factor on the rotated values): base 10000, eight times the trained
    length of 4096 where the frequencies are scaled."""
    i = torch.arange(rotary // 2, dtype=torch.float64)
    base, by, trained = 10000.0, 8.0, 4096.0
    if scaling == "ntk":
        base = base * by ** (rotary / (rotary - 2))
    f = base ** (-2.0 * i / rotary)
    if scaling == "linear":
        return f / by, 1.0
    if scaling == "yarn":
        turns = trained * f / (2 * math.pi)
        keep = ((turns - 1.0) / 31.0).clamp(0.0, 1.0)
        return f * (keep + (1 - keep) / by), 0.1 * math.log(by) + 1.0
    return f, 1.0


def _own_table(hb, rotary, layout, scaling, dev):
    return hb.rope_table(rotary, base=10000.0, scaling=scaling, factor=8.0 if scaling != "none" else 1.0,
                         original_len=4096, interleaved=layout == "interleaved", device=dev)


def _randn(g, shape, dtype, dev):
    return torch.randn(shape, generator=g, device=dev, dtype=torch.float32).to(dtype)


def _int32(v, dev):
    return torch.tensor(v, dtype=torch.int32, device=dev)


def _offsets(v, dev):
    return _int32([0] + torch.tensor(v, dtype=torch.int64).cumsum(0).tolist(), dev)


def _quantise(x):
    """8-bit codes of x, (..., width), and the exponent of each row's scale: the smallest power of two, 2^-127 at the
    least, that brings the row's finite values to 448 or below. A value that is not finite becomes NaN."""
    x = x.float()
    fine = x.isfinite()
    top = torch.where(fine, x.abs(), 0.0).amax(-1)
    m, e = torch.frexp(top)
    e = torch.where(top > 0, e - 9 + (m > 0.875).int(), -127).clamp(min=-127)
    x = torch.where(fine, torch.ldexp(x, -e[..., None]), math.nan)
    return x.to(torch.float8_e4m3fn), (e + 127).to(torch.uint8)


def _pages(c, lens, g, dev):
    """A page table with room for `lens` rows of each sequence, pages in any order, and the number of pages."""
    need = [(n + c["page"] - 1) // c["page"] for n in lens]
    order = torch.randperm(sum(need) + 3, generator=g, device=dev).int()
    width = max(1, max(need))
    need = torch.tensor(need, device=dev)
    at = torch.arange(width, device=dev)[None, :]
    first = (need.cumsum(0) - need)[:, None]
    table = torch.where(at < need[:, None], order[(first + at).clamp(max=order.numel() - 1)], -1)
    return table.int().contiguous(), int(order.numel())


def prepare(case, seed):
    c, dev = case, _dev()
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    dtype, H, D = DTYPES[c["dtype"]], c["heads"], c["dim"]
    s = {"c": c}
    if own:
        from jagged_hstu_attention_gb300 import binding as hb
        s["hb"] = hb
    if c["op"] == "rope":
        T = c["tokens"]
        if c["fused"]:  # rows of a projection that holds u, v, q and k of a token side by side
            both = _randn(g, (T, 4 * H * D), dtype, dev)
            s["q"], s["k"] = (both[:, i * H * D:(i + 1) * H * D].unflatten(1, (H, D)) for i in (2, 3))
        else:
            s["q"], s["k"] = _randn(g, (T, H, D), dtype, dev), _randn(g, (T, H, D), dtype, dev)
        s["positions"] = torch.randint(0, c["far"], (T,), generator=g, device=dev).int()
        if c["train"]:
            s["dq"], s["dk"] = _randn(g, (T, H, D), dtype, dev), _randn(g, (T, H, D), dtype, dev)
        f, s["factor"] = _frequencies(c["rotary"], c["scaling"])
        s["f"] = f.to(dev)
        if own:
            s["table"] = _own_table(hb, c["rotary"], c["layout"], c["scaling"], dev)
        return s
    Dv, P = c["dim_v"], c["page"]
    hist, added = _lengths(c)
    after = [h + n for h, n in zip(hist, added)] if c["op"] == "cache" else _cached(c)
    s["page_table"], pages = _pages(c, after, g, dev)
    for name, width in (("k", D), ("v", Dv)):
        rows = _randn(g, (pages, H, P, width), dtype, dev)
        if c["quantised"]:
            codes, s[name + "_scale"] = _quantise(rows)
            rows = codes.view(torch.uint8)
        s[name + "_pages"] = rows
    if c["op"] == "cache":
        T = sum(added)
        s["k"], s["v"] = _randn(g, (T, H, D), dtype, dev), _randn(g, (T, H, Dv), dtype, dev)
        s["offsets"], s["lens"], s["rows"] = _offsets(added, dev), _int32(hist, dev), T
        if c["back"] == "all":
            s["back"], s["back_rows"], s["starts"] = _offsets(after, dev), sum(after), None
        elif c["back"] == "new":
            s["back"], s["back_rows"], s["starts"] = s["offsets"], T, s["lens"]
        if c["rotary"]:
            f, s["factor"] = _frequencies(c["rotary"], "none")
            s["f"] = f.to(dev)
            s["table"] = _own_table(hb, c["rotary"], "half", "none", dev) if own else None
    else:
        s["q"] = _randn(g, (sum(added), H, D), dtype, dev)
        s["lens"], s["cand_offsets"] = _int32(after, dev), _offsets(added, dev)
        s["most"], s["most_cands"], s["cands"] = max(after), max(added), sum(added)
        s["func"] = None
        if c["mask"] == "self":
            at = [(h, h + j, h + j + 1) for h, n in zip(hist, added) for j in range(n)]
            s["func"] = _int32(at, dev).t().contiguous()
        elif c["mask"] == "sla":
            at = [(min(256, n), max(0, n - 32), n) for n in after]
            s["func"] = _int32(at, dev).t().contiguous()
        if own:
            s["single"] = c["cand_lo"] == 1 and c["cand_hi"] == 1
    if own:
        s["cache"] = hb.PagedCache(s["k_pages"], s["v_pages"], s.get("k_scale"), s.get("v_scale"), dtype=dtype)
    return s


# ------------------------------------------------------------- plain forms


def _rotate(x, positions, f, factor, layout, sign):
    """x (T, H, D) with the first 2 len(f) values of each head turned by sign * position * f."""
    half = f.numel()
    angle = positions.double()[:, None] * f
    cos, sin = (factor * angle.cos()).float()[:, None], (sign * factor * angle.sin()).float()[:, None]
    y = x.float().clone()
    if layout == "half":
        a, b = y[..., :half], y[..., half:2 * half]
    else:
        a, b = y[..., 0:2 * half:2], y[..., 1:2 * half:2]
    turned = a * cos - b * sin, b * cos + a * sin
    a.copy_(turned[0])
    b.copy_(turned[1])
    return y.to(x.dtype)


def _places(offsets, rows, starts, page_table, page):
    """(page, slot) of each row of a jagged batch whose sequence b begins at starts[b] of its pages."""
    counts = (offsets[1:] - offsets[:-1]).long()
    b = torch.repeat_interleave(torch.arange(counts.numel(), device=offsets.device), counts, output_size=rows)
    pos = torch.arange(rows, device=offsets.device) - offsets[:-1].long()[b]
    if starts is not None:
        pos = pos + starts.long()[b]
    return page_table[b, pos // page].long(), pos % page, pos


def _plain_cache(s, c):
    page, slot, pos = _places(s["offsets"], s["rows"], s["lens"], s["page_table"], c["page"])
    k = _rotate(s["k"], pos, s["f"], s["factor"], "half", 1.0) if c["rotary"] else s["k"]
    for name, x in (("k", k), ("v", s["v"])):
        if c["quantised"]:
            codes, scale = _quantise(x)
            s[name + "_pages"][page, :, slot] = codes.view(torch.uint8)
            s[name + "_scale"][page, :, slot] = scale
        else:
            s[name + "_pages"][page, :, slot] = x
    if c["back"] == "none":
        return {"k": s["k_pages"], "v": s["v_pages"]}
    page, slot, _ = _places(s["back"], s["back_rows"], s["starts"], s["page_table"], c["page"])
    return {name: _values(s, name, page, slot).to(DTYPES[c["dtype"]]) for name in ("k", "v")}


def _values(s, name, page, slot):
    """The cached rows at (page, slot), (..., H, width) in 32 bits."""
    rows = s[name + "_pages"][page, :, slot]
    if name + "_scale" not in s:
        return rows.float()
    e = s[name + "_scale"][page, :, slot].int() - 127
    return torch.ldexp(rows.view(torch.float8_e4m3fn).float(), e[..., None])


def _plain_paged(s, c):
    B, dev = c["batch"], s["q"].device
    pos = torch.arange(s["most"], device=dev)
    page, slot = s["page_table"].clamp(min=0)[:, pos // c["page"]].long(), (pos % c["page"]).expand(B, -1)
    offsets = s["cand_offsets"].long()
    k, v = _values(s, "k", page, slot), _values(s, "v", page, slot)  # (B, L, H, width)
    at = offsets[:-1, None] + torch.arange(s["most_cands"], device=dev)  # (B, C): a sequence's candidates
    real = at < offsets[1:, None]
    at = at.clamp(max=s["cands"] - 1)
    seen = pos < s["lens"][:, None, None]
    if s["func"] is not None:
        f = s["func"][:, at][..., None]  # (3, B, C, 1)
        seen = seen & ((pos < f[0]) | ((pos >= f[1]) & (pos < f[2])))
    x = torch.einsum("bchd,blhd->bhcl", s["q"].float()[at], k) / math.sqrt(c["dim"])
    p = torch.where(seen[:, None], x / (1 + torch.exp(-x)) / s["most"], 0.0)
    o = torch.einsum("bhcl,blhd->bchd", p, v)
    return torch.zeros((s["cands"],) + o.shape[2:], device=dev).index_put((at[real],), o[real]).to(s["q"].dtype)


def run(state):
    s, c = state, state["c"]
    if own:
        return _run_own(s, c)
    if c["op"] == "rope":
        turn = lambda x, sign: _rotate(x, s["positions"], s["f"], s["factor"], c["layout"], sign)  # noqa: E731
        out = {"q": turn(s["q"], 1.0), "k": turn(s["k"], 1.0)}
        if c["train"]:
            out["dq"], out["dk"] = turn(s["dq"], -1.0), turn(s["dk"], -1.0)
        return out
    return _plain_cache(s, c) if c["op"] == "cache" else {"o": _plain_paged(s, c)}


def _run_own(s, c):
    hb = s["hb"]
    if c["op"] == "rope":
        q, k = hb.rope(s["q"], s["k"], s["positions"], s["table"])
        if not c["train"]:
            return {"q": q, "k": k}
        dq, dk = hb.rope(s["dq"], s["dk"], s["positions"], s["table"], backward=True)
        return {"q": q, "k": k, "dq": dq, "dk": dk}
    if c["op"] == "cache":
        hb.cache_write(s["cache"], s["k"], s["v"], s["offsets"], s["lens"], s["page_table"], rope=s.get("table"))
        if c["back"] == "none":
            return {"k": s["k_pages"], "v": s["v_pages"]}
        k, v = hb.cache_read(s["cache"], s["back"], s["back_rows"], s["page_table"], starts=s["starts"])
        return {"k": k, "v": v}
    return {"o": hb.fwd_paged(s["q"], s["cache"], s["lens"], s["page_table"], s["most"], func_c=s["func"],
                              cand_offsets=None if s["single"] else s["cand_offsets"])}


# ------------------------------------------------------- values in 64 bits


def exact(case, seed):
    c, s = case, prepare(case, seed)
    if c["op"] == "rope":
        names = ("q", "k", "dq", "dk") if c["train"] else ("q", "k")
        return {n: _turned(s[n], s["positions"], s["f"], s["factor"], c["layout"], n in ("dq", "dk")) for n in names}
    return _exact_cache(s, c) if c["op"] == "cache" else {"o": _exact_paged(s, c)}


def _turned(x, positions, f, factor, layout, back):
    """The rotation as a product of complex numbers, backwards by the conjugate."""
    n = f.numel()
    x = x.double()
    head = x[..., :2 * n]
    pairs = head.unflatten(-1, (2, n)).transpose(-1, -2) if layout == "half" else head.unflatten(-1, (n, 2))
    angle = torch.outer(positions.double(), -f if back else f)
    z = torch.view_as_complex(pairs.contiguous()) * torch.polar(torch.full_like(angle, factor), angle)[:, None, :]
    z = torch.view_as_real(z)
    z = z.transpose(-1, -2) if layout == "half" else z
    return torch.cat([z.reshape(head.shape), x[..., 2 * n:]], -1)


def _rows_of(s, c, name, b, n, start=0):
    """Rows [start, start + n) of sequence b as (n, H, width) in 64 bits, page by page."""
    first, last = start // c["page"], (start + n + c["page"] - 1) // c["page"]
    which = s["page_table"][b, first:last].long()
    rows = s[name + "_pages"][which]
    if c["quantised"]:
        e = s[name + "_scale"][which].double() - 127
        rows = rows.view(torch.float8_e4m3fn).double() * torch.exp2(e)[..., None]
    rows = rows.double().transpose(1, 2).flatten(0, 1)
    return rows[start - first * c["page"]:][:n]


def _through_codes(x):
    """x after a trip through 8 bits: mantissas of four bits below the row's power-of-two scale."""
    x = x.double()
    top = x.abs().amax(-1, keepdim=True)
    scale = torch.exp2(torch.ceil(torch.log2(top / 448.0).nan_to_num(neginf=-127.0)).clamp(min=-127.0))
    scale = torch.where(top > 448.0 * scale, 2 * scale, torch.where(top <= 224.0 * scale, scale / 2, scale))
    y = x / scale
    step = torch.exp2(torch.floor(torch.log2(y.abs().clamp(min=2.0 ** -6))) - 3)
    return torch.round(y / step) * step * scale


def _exact_cache(s, c):
    hist, new = _lengths(c)
    if not c["quantised"]:
        out = {n: s[n + "_pages"].double() for n in ("k", "v")}
        k = s["k"].double()
        at = 0
        for b, (h, n) in enumerate(zip(hist, new)):
            pos = torch.arange(h, h + n, device=k.device)
            page, slot = s["page_table"][b].long()[pos // c["page"]], pos % c["page"]
            rows = s["k"][at:at + n]
            rows = _turned(rows, pos, s["f"], s["factor"], "half", False) if c["rotary"] else rows.double()
            out["k"][page, :, slot] = rows
            out["v"][page, :, slot] = s["v"][at:at + n].double()
            at += n
        return out
    out = {}
    for name in ("k", "v"):
        fresh = _through_codes(s[name])
        parts, at = [], 0
        for b, (h, n) in enumerate(zip(hist, new)):
            if c["back"] == "all":
                parts.append(_rows_of(s, c, name, b, h))
            parts.append(fresh[at:at + n])
            at += n
        out[name] = torch.cat(parts)
    return out


def _exact_paged(s, c):
    out, at = [], 0
    hist, cands = _lengths(c)
    for b, (full, n) in enumerate(zip(_cached(c), cands)):
        if n == 0:
            continue
        k, v = _rows_of(s, c, "k", b, full), _rows_of(s, c, "v", b, full)
        x = torch.matmul(s["q"][at:at + n].double().transpose(0, 1), k.permute(1, 2, 0)) * c["dim"] ** -0.5  # (H, n, L)
        p = x * torch.sigmoid(x) / s["most"]
        if c["mask"] == "self":
            see = torch.zeros((n, full), dtype=torch.bool, device=p.device)
            see[:, :hist[b]] = True
            see[torch.arange(n), hist[b] + torch.arange(n)] = True
            p = p * see
        elif c["mask"] == "sla":
            see = torch.zeros(full, dtype=torch.bool, device=p.device)
            see[:256] = True
            see[-32:] = True
            p = p * see
        out.append(torch.matmul(p, v.transpose(0, 1)).transpose(0, 1))
        at += n
    return torch.cat(out)
