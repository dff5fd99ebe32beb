"""Cases that measure the operators around the attention of a layer: embedding
rows and their gradient, root-mean-square norms, matrix products with an
epilogue, and the two chained through 8 bits.

Each case names one operator (``op``) and its sizes; ``run`` is one pass of it,
in elementary torch operations or, where ``own`` is set, through the calls that
a program makes of this package.

  embed   rows of a table by id, scaled (and, for training, the table's
          gradient).
  norm    h = x + residual, y = h / rms(h) * weight * gate (and, for training,
          the gradients).
  linear  y = act(x w^T + bias) + residual (and, for training, the gradients).
  chain8  a norm whose output is 8-bit codes with a power-of-two scale a row,
          and a product of those codes with a weight held in 8 bits.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
EPS = 1e-6


def _dev():
    return "cuda" if torch.cuda.is_available() else "cpu"


# ------------------------------------------------------------------- cases


def listed():
    return [
        # The newest item of each of 64 users: a decode step's lookup in a table of 200003 items.
        {"name": "embed_step", "op": "embed", "tokens": 64, "vocab": 200003, "dim": 512, "table": "bf16", "dtype": "bf16",
         "ids": "i32", "padding": 0.0, "train": False, "grad": "f32"},
        # A training batch of the OneRank shape (64 sequences of 512 to 2048 rows): lookup and gradient.
        {"name": "embed_train", "op": "embed", "tokens": 81920, "vocab": 200003, "dim": 512, "table": "bf16",
         "dtype": "bf16", "ids": "i32", "padding": 0.0, "train": True, "grad": "f32"},
        # A large table of narrow rows held in 32 bits, ids in 64 bits, a tenth of them padding.
        {"name": "embed_large", "op": "embed", "tokens": 524287, "vocab": 4000037, "dim": 64, "table": "f32",
         "dtype": "f16", "ids": "i64", "padding": 0.1, "train": True, "grad": "f32"},
        # The norm in front of a layer at a decode step of 64 users, residual added on the way.
        {"name": "norm_step", "op": "norm", "tokens": 64, "dim": 512, "dtype": "bf16", "residual": True, "gate": False,
         "train": False},
        # The same norm over a training batch of the OneRank shape, forward and backward.
        {"name": "norm_train", "op": "norm", "tokens": 81920, "dim": 512, "dtype": "bf16", "residual": True,
         "gate": False, "train": True},
        # The norm behind the attention: its output normed and gated by u, a slice of the input projection's rows.
        {"name": "norm_gate_f16", "op": "norm", "tokens": 32749, "dim": 1024, "dtype": "f16", "residual": False,
         "gate": True, "train": True},
        # The input projection (u, v, q and k of four heads of 128) at a decode step of 64 users.
        {"name": "linear_step", "op": "linear", "tokens": 64, "d_in": 512, "d_out": 2048, "dtype": "bf16",
         "act": "silu", "bias": True, "residual": False, "train": False},
        # The output projection of a long batch with the layer's input added.
        {"name": "linear_out_f16", "op": "linear", "tokens": 81920, "d_in": 512, "d_out": 512, "dtype": "f16",
         "act": "none", "bias": False, "residual": True, "train": False},
        # The input projection over a training batch, forward and backward.
        {"name": "linear_train", "op": "linear", "tokens": 81920, "d_in": 512, "d_out": 2048, "dtype": "bf16",
         "act": "silu", "bias": True, "residual": False, "train": True},
        # A wide feed-forward product, ragged in its rows.
        {"name": "linear_wide", "op": "linear", "tokens": 8179, "d_in": 2048, "d_out": 8192, "dtype": "bf16",
         "act": "gelu", "bias": True, "residual": False, "train": False},
        # Norm and input projection through 8 bits at a decode step of 64 users.
        {"name": "chain8_step", "op": "chain8", "tokens": 64, "d_in": 512, "d_out": 2048, "dtype": "bf16",
         "act": "silu", "bias": True, "residual": True},
        # The same for a long prompt and a wide layer.
        {"name": "chain8_wide", "op": "chain8", "tokens": 16381, "d_in": 2048, "d_out": 8192, "dtype": "bf16",
         "act": "silu", "bias": True, "residual": True},
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def _width(rng, lo, hi, step):
    return step * _log_int(rng, lo // step, hi // step)


def draw(rng):
    op, dtype = rng.choice(["embed", "norm", "linear", "chain8"]), rng.choice(["bf16", "f16"])
    if op == "embed":
        c = {"op": op, "tokens": _log_int(rng, 1, 524287), "vocab": _log_int(rng, 2, 4000000),
             "dim": _width(rng, 8, 2048, 8), "table": rng.choice([dtype, "f32"]), "dtype": dtype,
             "ids": rng.choice(["i32", "i64"]), "padding": rng.choice([0.0, 0.2]), "train": rng.random() < 0.6,
             "grad": rng.choice([dtype, "f32"])}
        while c["vocab"] > 2 and c["vocab"] * c["dim"] > 1 << 28:
            c["vocab"] = (c["vocab"] + 1) // 2
        while c["tokens"] > 1 and c["tokens"] * c["dim"] > 1 << 26:
            c["tokens"] = (c["tokens"] + 1) // 2
    elif op == "norm":
        c = {"op": op, "tokens": _log_int(rng, 1, 131072), "dim": _width(rng, 8, 8192, 8), "dtype": dtype,
             "residual": rng.random() < 0.6, "gate": rng.random() < 0.4, "train": rng.random() < 0.5}
        while c["tokens"] > 1 and c["tokens"] * c["dim"] > 1 << 26:
            c["tokens"] = (c["tokens"] + 1) // 2
    else:
        step = 16 if op == "chain8" else 8
        c = {"op": op, "tokens": _log_int(rng, 1, 81920), "d_in": _width(rng, 16, 8192, step),
             "d_out": _width(rng, 16, 8192, step), "dtype": dtype, "act": rng.choice(["none", "silu", "gelu", "relu"]),
             "bias": rng.random() < 0.6, "residual": rng.random() < 0.5}
        if op == "linear":
            c["train"] = rng.random() < 0.5
        # A quarter of the largest case's multiplications at the most, and no more rows than it writes.
        while c["tokens"] > 1 and (c["tokens"] * c["d_in"] * c["d_out"] > 1 << 36
                                   or c["tokens"] * max(c["d_in"], c["d_out"]) > 1 << 27):
            c["tokens"] = (c["tokens"] + 1) // 2
    return c


def _shares(c):
    """Of the vocabulary's ids, how likely a token names each: Zipf's law, floor(vocab^u) of a uniform u."""
    edges = torch.arange(1, c["vocab"] + 2, dtype=torch.float64).log() / math.log(c["vocab"] + 1)
    return edges.diff()


def work(case):
    c = case
    T = c["tokens"]
    if c["op"] == "embed":
        real = T * (1.0 - c["padding"])
        # rows named at least once: 1 - (1 - p)^n of each
        named = float((1.0 - (1.0 - _shares(c)).clamp(min=0.0).pow(real)).sum())
        e, size = 2, 4 if c["table"] == "f32" else 2
        idb = 8 if c["ids"] == "i64" else 4
        total, flops = T * idb + named * c["dim"] * size + T * c["dim"] * e, T * c["dim"]
        if c["train"]:
            total += T * idb + real * c["dim"] * e + c["vocab"] * c["dim"] * (4 if c["grad"] == "f32" else 2)
            flops += 2 * T * c["dim"]
        return {"bytes": total, "flops": flops}
    if c["op"] == "norm":
        n = T * c["dim"] * 2
        passes = 2 + (2 if c["residual"] else 0) + (1 if c["gate"] else 0)  # x, y; residual, h; gate
        flops = 6 * T * c["dim"]
        if c["train"]:
            passes += 3 + (1 if c["residual"] else 0) + (2 if c["gate"] else 0)  # dy, h, dx; dh; gate, its gradient
            flops += 12 * T * c["dim"]
        return {"bytes": passes * n + 2 * c["dim"] + (8 * T + 4 * c["dim"] if c["train"] else 4 * T), "flops": flops}
    K, N = c["d_in"], c["d_out"]
    flops = 2 * T * K * N
    if c["op"] == "chain8":
        # x, residual and h; the codes out and in again; codes of the weight; y
        return {"bytes": T * K * (6 if c["residual"] else 2) + 2 * T * (K + 1) + N * (K + 1) + 2 * T * N,
                "flops": flops + 8 * T * K}
    total = 2 * (T * K + N * K + T * N) + (2 * T * N if c["residual"] else 0)
    if c["train"]:
        z = 0 if c["act"] == "none" else 2 * T * N
        total += z + (z + 2 * T * N) + 2 * T * K + 2 * N * K + 2 * T * K + 2 * N * K
        flops *= 3
    return {"bytes": total, "flops": flops}


# ------------------------------------------------------------------ inputs


def _randn(g, shape, dtype, dev, scale=1.0):
    return (torch.randn(shape, generator=g, device=dev, dtype=torch.float32) * scale).to(dtype)


def _codes(x):
    """8-bit codes of x, (rows, width) in 32 bits, and the exponent byte of each row's scale: the smallest power of two,
    2^-127 at the least, that brings the row to 448 or below."""
    m, e = torch.frexp(x.abs().amax(-1))
    e = torch.where(m > 0, e - 9 + (m > 0.875).int(), -127).clamp(min=-127)
    return torch.ldexp(x, -e[:, None]).to(torch.float8_e4m3fn), (e + 127).to(torch.uint8)


def prepare(case, seed):
    c, dev = case, _dev()
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    dtype, T = DTYPES[c["dtype"]], c["tokens"]
    s = {"c": c}
    if own:
        from jagged_hstu_attention_gb300 import binding as hb
        s["hb"] = hb
    if c["op"] == "embed":
        V, D = c["vocab"], c["dim"]
        s["table"] = _randn(g, (V, D), DTYPES[c["table"]], dev, D ** -0.5)
        u = torch.rand(T, generator=g, device=dev, dtype=torch.float64)
        ids = (torch.exp(u * math.log(V + 1)).long() - 1).clamp(0, V - 1)
        ids = ids * 7919 % V  # neighbours by frequency are no neighbours in the table
        if c["padding"]:
            ids = torch.where(torch.rand(T, generator=g, device=dev) < c["padding"], -1, ids)
        s["ids"] = ids if c["ids"] == "i64" else ids.int()
        if c["train"]:
            s["dy"] = _randn(g, (T, D), dtype, dev)
        return s
    if c["op"] == "norm":
        D = c["dim"]
        s["x"] = _randn(g, (T, D), dtype, dev)
        s["w"] = (1.0 + 0.1 * torch.randn(D, generator=g, device=dev)).to(dtype)
        s["r"] = _randn(g, (T, D), dtype, dev, 3.0) if c["residual"] else None
        # u lies in front of v, q and k in the rows of a projection
        s["gate"] = _randn(g, (T, 4 * D), dtype, dev)[:, :D] if c["gate"] else None
        if c["train"]:
            s["dy"] = _randn(g, (T, D), dtype, dev)
            s["dh"] = _randn(g, (T, D), dtype, dev) if c["residual"] else None
        return s
    K, N = c["d_in"], c["d_out"]
    s["x"] = _randn(g, (T, K), dtype, dev)
    w = torch.randn((N, K), generator=g, device=dev, dtype=torch.float32) * K ** -0.5
    s["b"] = _randn(g, (N,), dtype, dev, 0.1) if c["bias"] else None
    if c["op"] == "chain8":
        s["r"] = _randn(g, (T, K), dtype, dev, 3.0) if c["residual"] else None
        s["nw"] = (1.0 + 0.1 * torch.randn(K, generator=g, device=dev)).to(dtype)
        s["w_codes"], s["w_scale"] = _codes(w)
        if own:
            s["w8"] = hb.QuantisedRows(s["w_codes"].view(torch.uint8), s["w_scale"])
        return s
    s["w"] = w.to(dtype)
    s["r"] = _randn(g, (T, N), dtype, dev) if c["residual"] else None
    if c["train"]:
        s["dy"] = _randn(g, (T, N), dtype, dev)
    return s


# ------------------------------------------------------------- plain forms


def _plain_embed(s, c):
    keep = (s["ids"] >= 0)[:, None]
    at = s["ids"].clamp(min=0).long()
    scale = math.sqrt(c["dim"])
    out = {"y": torch.where(keep, s["table"][at].float() * scale, 0.0).to(DTYPES[c["dtype"]])}
    if c["train"]:
        d = torch.zeros(s["table"].shape, device=at.device).index_add_(0, at, torch.where(keep, s["dy"].float() * scale, 0.0))
        out["dtable"] = d.to(DTYPES[c["grad"]])
    return out


def _plain_norm(x, r, w, gate):
    """(y in 32 bits, h, 1 / rms): the norm is that of h as it is kept, in the rows' type."""
    h = x if r is None else (x.float() + r.float()).to(x.dtype)
    h32 = h.float()
    rstd = 1 / torch.sqrt((h32 * h32).mean(-1) + EPS)
    y = h32 * rstd[:, None] * w.float()
    return y if gate is None else y * gate.float(), h, rstd


def _plain_norm_bwd(dy, h, rstd, w, gate, dh):
    hat = h.float() * rstd[:, None]
    a = dy.float() if gate is None else dy.float() * gate.float()
    t = a * w.float()
    dx = rstd[:, None] * (t - hat * (t * hat).mean(-1, keepdim=True))
    if dh is not None:
        dx = dx + dh.float()
    dgate = None if gate is None else (dy.float() * hat * w.float()).to(h.dtype)
    return dx.to(h.dtype), (a * hat).sum(0).to(h.dtype), dgate


def _act(z, act):
    if act == "silu":
        return z / (1 + torch.exp(-z))
    if act == "gelu":
        return z / (1 + torch.exp(-2 * math.sqrt(2 / math.pi) * (z + 0.044715 * z * z * z)))
    return z * (z > 0) if act == "relu" else z


def _act_grad(z, act):
    if act == "silu":
        p = 1 / (1 + torch.exp(-z))
        return p * (1 + z * (1 - p))
    if act == "gelu":
        k = 2 * math.sqrt(2 / math.pi)
        p = 1 / (1 + torch.exp(-k * (z + 0.044715 * z * z * z)))
        return p * (1 + z * (1 - p) * k * (1 + 3 * 0.044715 * z * z))
    return (z > 0).float()


def _plain_linear(s, c):
    dtype = s["x"].dtype
    z = s["x"].float() @ s["w"].float().t()
    if c["bias"]:
        z = z + s["b"].float()
    y = _act(z, c["act"])
    out = {"y": (y + s["r"].float() if c["residual"] else y).to(dtype)}
    if c["train"]:
        d = s["dy"].float()
        if c["act"] != "none":
            out["z"] = z.to(dtype)
            d = d * _act_grad(out["z"].float(), c["act"])
        out["dx"], out["dw"] = (d @ s["w"].float()).to(dtype), (d.t() @ s["x"].float()).to(dtype)
        if c["bias"]:
            out["db"] = d.sum(0).to(dtype)
    return out


def _plain_chain8(s, c):
    y, h, _ = _plain_norm(s["x"], s["r"], s["nw"], None)
    codes, scale = _codes(y)
    a = torch.ldexp(codes.float(), scale[:, None].int() - 127)
    w = torch.ldexp(s["w_codes"].float(), s["w_scale"][:, None].int() - 127)
    z = a @ w.t()
    if c["bias"]:
        z = z + s["b"].float()
    out = {"y": _act(z, c["act"]).to(h.dtype)}
    return {**out, "h": h} if c["residual"] else out


def run(state):
    s, c = state, state["c"]
    if own:
        return _run_own(s, c)
    if c["op"] == "embed":
        return _plain_embed(s, c)
    if c["op"] == "norm":
        y, h, rstd = _plain_norm(s["x"], s["r"], s["w"], s["gate"])
        out = {"y": y.to(h.dtype), "rstd": rstd, "h": h if c["residual"] else None}
        if c["train"]:
            out["dx"], out["dw"], out["dgate"] = _plain_norm_bwd(s["dy"], h, rstd, s["w"], s["gate"], s["dh"])
        return out
    return _plain_linear(s, c) if c["op"] == "linear" else _plain_chain8(s, c)


def _run_own(s, c):
    hb = s["hb"]
    if c["op"] == "embed":
        scale = math.sqrt(c["dim"])
        out = {"y": hb.embed(s["table"], s["ids"], scale, dtype=DTYPES[c["dtype"]])}
        if c["train"]:
            out["dtable"] = hb.embed_bwd(s["dy"], s["ids"], c["vocab"], scale, dtype=DTYPES[c["grad"]])
        return out
    if c["op"] == "norm":
        y, h, rstd = hb.rms_norm(s["x"], s["w"], residual=s["r"], gate=s["gate"], eps=EPS)
        out = {"y": y, "rstd": rstd, "h": h}
        if c["train"]:
            out["dx"], out["dw"], out["dgate"] = hb.rms_norm_bwd(s["dy"], s["x"] if h is None else h, rstd, s["w"],
                                                                 gate=s["gate"], dh=s["dh"])
        return out
    if c["op"] == "chain8":
        y8, h, _ = hb.rms_norm(s["x"], s["nw"], residual=s["r"], eps=EPS, quantise=True)
        y, _ = hb.linear(y8, s["w8"], bias=s["b"], act=c["act"], dtype=DTYPES[c["dtype"]])
        return {"y": y, "h": h} if c["residual"] else {"y": y}
    keep = c["train"] and c["act"] != "none"
    y, z = hb.linear(s["x"], s["w"], bias=s["b"], act=c["act"], residual=s["r"], want_z=keep)
    out = {"y": y}
    if c["train"]:
        out["dx"], out["dw"], db = hb.linear_bwd(s["dy"], z, s["x"], s["w"], act=c["act"], want_dbias=c["bias"])
        if keep:
            out["z"] = z
        if c["bias"]:
            out["db"] = db
    return out


# ------------------------------------------------------- values in 64 bits


def exact(case, seed):
    c, s = case, prepare(case, seed)
    if c["op"] == "embed":
        return _exact_embed(s, c)
    if c["op"] == "norm":
        return _exact_norm(s, c)
    return _exact_linear(s, c) if c["op"] == "linear" else _exact_chain8(s, c)


def _exact_embed(s, c):
    root, ids = c["dim"] ** 0.5, s["ids"].long()
    real = torch.nonzero(ids >= 0).squeeze(1)
    y = torch.zeros((c["tokens"], c["dim"]), dtype=torch.float64, device=ids.device)
    y[real] = torch.index_select(s["table"], 0, ids[real]).double() * root
    out = {"y": y}
    if c["train"]:
        d = torch.zeros((c["vocab"], c["dim"]), dtype=torch.float64, device=ids.device)
        out["dtable"] = d.index_put_((ids[real],), s["dy"][real].double() * root, accumulate=True)
    return out


def _kept(s):
    """h in 64 bits, and as it is kept."""
    h = s["x"].double()
    if s["r"] is None:
        return h, h
    h = h + s["r"].double()
    return h, h.to(s["x"].dtype).double()


def _exact_norm(s, c):
    total, h = _kept(s)
    n = h.shape[1]
    rms = (torch.linalg.vector_norm(h, dim=1, keepdim=True) ** 2 / n + EPS).sqrt()
    unit, w = h / rms, s["w"].double()
    through = torch.ones_like(h) if s["gate"] is None else s["gate"].double()
    out = {"y": unit * w * through, "rstd": 1 / rms[:, 0], "h": total if c["residual"] else None}
    if c["train"]:
        dy = s["dy"].double()
        d = dy * through * w
        # the part of d along h does not move a normed row, but for what eps leaves
        out["dx"] = d / rms - h * ((d * h).sum(1, keepdim=True) / (n * rms ** 3))
        if c["residual"]:
            out["dx"] = out["dx"] + s["dh"].double()
        out["dw"] = torch.einsum("td,td->d", dy * through, unit)
        out["dgate"] = None if s["gate"] is None else dy * unit * w
    return out


def _exact_act(z, act):
    """(act(z), its derivative) in 64 bits."""
    if act == "silu":
        p = torch.sigmoid(z)
        return z * p, p + z * p * torch.sigmoid(-z)
    if act == "gelu":
        k = (2 / math.pi) ** 0.5
        t = torch.tanh(k * (z + 0.044715 * z ** 3))
        return 0.5 * z * (1 + t), 0.5 * (1 + t) + 0.5 * z * (1 - t * t) * k * (1 + 0.134145 * z * z)
    if act == "relu":
        return torch.clamp(z, min=0), torch.where(z > 0, 1.0, 0.0).double()
    return z, torch.ones_like(z)


def _exact_linear(s, c):
    x, w = s["x"].double(), s["w"].double()
    z = torch.einsum("tk,nk->tn", x, w)
    if c["bias"]:
        z += s["b"].double()
    y = _exact_act(z, c["act"])[0]
    out = {"y": y + s["r"].double() if c["residual"] else y}
    if c["train"]:
        g = s["dy"].double()
        if c["act"] != "none":
            out["z"] = z
            g = g * _exact_act(z.to(s["x"].dtype).double(), c["act"])[1]  # by z as it is kept
        out["dx"], out["dw"] = torch.einsum("tn,nk->tk", g, w), torch.einsum("tn,tk->nk", g, x)
        if c["bias"]:
            out["db"] = torch.einsum("tn->n", g)
    return out


def _through_codes(x):
    """x, (rows, width) in 64 bits, after a trip through 8 bits: mantissas of four bits below the row's scale."""
    top = x.abs().amax(1, keepdim=True)
    e = torch.ceil(torch.log2(top / 448.0).nan_to_num(neginf=-127.0)).clamp(min=-127.0)
    e = torch.where(top > 448.0 * torch.exp2(e), e + 1, torch.where(top <= 224.0 * torch.exp2(e), e - 1, e)).clamp(min=-127.0)
    v = x * torch.exp2(-e)
    step = torch.exp2(torch.floor(torch.log2(v.abs().clamp(min=2.0 ** -6))) - 3)
    return torch.round(v / step) * step * torch.exp2(e)


def _exact_chain8(s, c):
    total, h = _kept(s)
    unit = h / (torch.linalg.vector_norm(h, dim=1, keepdim=True) ** 2 / h.shape[1] + EPS).sqrt()
    w = s["w_codes"].double() * torch.exp2(s["w_scale"].double() - 127.0)[:, None]
    z = torch.einsum("tk,nk->tn", _through_codes(unit * s["nw"].double()), w)
    if c["bias"]:
        z += s["b"].double()
    y = _exact_act(z, c["act"])[0]
    return {"y": y, "h": total} if c["residual"] else {"y": y}
