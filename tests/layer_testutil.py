"""Plain 64-bit forms of the layer's row operators (embedding rows, norms,
linear maps) and the error bounds their tests use. Rows are numpy arrays."""
import math

import numpy as np
import torch

from serving_testutil import f64, half_step, smallest_half_step  # noqa: F401

STEP32 = 2.0 ** -24  # one rounding in fp32
GELU_A, GELU_B = 2 * math.sqrt(2 / math.pi), 0.044715


def randn(shape, dtype, seed, scale=1.0):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return (torch.randn(shape, generator=g, device="cuda") * scale).to(dtype)


def worst(got, ref, tol):
    """How far past its bound the worst value is (at most 1 where all hold)."""
    d = np.abs(got - ref)
    assert np.isfinite(got).all()
    return float((d / np.maximum(tol, 1e-300)).max()) if d.size else 0.0


# ------------------------------------------------------------------- embed


def embed(table, ids, scale):
    ok = (ids >= 0) & (ids < table.shape[0])
    y = np.zeros((len(ids), table.shape[1]))
    y[ok] = table[ids[ok]] * float(np.float32(scale))
    return y


def embed_bwd(dy, ids, vocab, scale):
    """(gradient, sum of magnitudes, tokens of each row)."""
    ok = (ids >= 0) & (ids < vocab)
    s = float(np.float32(scale))
    d, m, n = np.zeros((vocab, dy.shape[1])), np.zeros((vocab, dy.shape[1])), np.zeros(vocab)
    np.add.at(d, ids[ok], dy[ok] * s)
    np.add.at(m, ids[ok], np.abs(dy[ok] * s))
    np.add.at(n, ids[ok], 1)
    return d, m, n


# -------------------------------------------------------------------- norm


def norm(h, w, gate=None, eps=1e-6):
    """(y, rstd) of kept rows h."""
    rstd = 1 / np.sqrt((h * h).mean(1) + eps)
    y = h * rstd[:, None] * w
    return (y if gate is None else y * gate), rstd


# Relative error of rstd in fp32: a thread's chain of at most 32 squares, then up
# to 8 joins (2^-24 each, terms of one sign), half of which passes the square
# root; mean, eps, root and reciprocal add 2^-24 each: below 32 * 2^-24. A y adds three
# products: below 2^-18 together.
NORM_ERR = 2.0 ** -18


def norm_bwd(dy, h, rstd, w, gate=None, dh=None):
    """dx, dweight, dgate with their magnitudes before cancellation."""
    u = h * rstd[:, None]
    a = dy if gate is None else dy * gate
    t = a * w
    m = (t * u).mean(1, keepdims=True)
    dx = rstd[:, None] * (t - u * m) + (0 if dh is None else dh)
    mag = rstd[:, None] * (np.abs(t) + np.abs(u) * np.abs(t * u).mean(1, keepdims=True))
    mag = mag + (0 if dh is None else np.abs(dh))
    dgate = None if gate is None else dy * u * w
    return (dx, mag), ((a * u).sum(0), np.abs(a * u).sum(0)), dgate


def e4m3(codes):
    """Values of 8-bit codes (a uint8 tensor)."""
    return codes.view(torch.float8_e4m3fn).float().cpu().numpy().astype(np.float64)


def scale_of(byte):
    return np.exp2(byte.cpu().numpy().astype(np.float64) - 127)


# ------------------------------------------------------------------ linear


def gate_arg(z, act):
    """(u, du/dz) of the sigmoid's argument."""
    if act == "gelu":
        return GELU_A * (z + GELU_B * z ** 3), GELU_A * (1 + 3 * GELU_B * z * z)
    return z, np.ones_like(z)


def act(z, name):
    if name == "none":
        return z
    if name == "relu":
        return np.maximum(z, 0)
    return z / (1 + np.exp(-gate_arg(z, name)[0]))


def act_grad(z, name):
    if name == "none":
        return np.ones_like(z)
    if name == "relu":
        return (z > 0) * 1.0
    u, du = gate_arg(z, name)
    s = 1 / (1 + np.exp(-u))
    return s * (1 + z * (1 - s) * du)


def act_rel(z, name):
    """Relative error of the sigmoid: the exponential's argument (three roundings of
    u), 2 + 1.2 |u| units of the exponential, the sum, and 2 units of the division."""
    if name in ("none", "relu"):
        return np.zeros_like(z)
    return (6 + 3 * np.abs(gate_arg(z, name)[0])) * 2 * STEP32


def act_grad_err(z, name):
    """Error of act': that of the sigmoid in each of its three factors."""
    if name in ("none", "relu"):
        return np.zeros_like(z)
    return act_rel(z, name) * (1 + 2 * np.abs(z) * np.abs(gate_arg(z, name)[1]))


def product_err(a, b):
    """Bound of a product's fp32 accumulation: one unit (2^-23, the sum may be cut) a
    term of the sum of magnitudes."""
    return a.shape[1] * 2 * STEP32 * (np.abs(a) @ np.abs(b))
