"""The layer's row operators as they are used together: embedding rows, norm, input
projection, attention, gated norm, output projection with the layer's input
added, and all their gradients; the same through 8 bits; captured into graphs, on
other streams and from several workspaces at once."""
import math
import threading

import numpy as np
import pytest
import torch

import oracle.hstu_oracle as orc
from jagged_hstu_attention_gb300 import binding as hb
from jagged_hstu_attention_gb300 import workloads as wl
import layer_testutil as lt

pytestmark = pytest.mark.gpu
F16, BF = torch.float16, torch.bfloat16
B, H, D, EPS = 3, 2, 32, 1e-6
DM = H * D  # width of the stream


def _layer(dtype, seed=0, vocab=50):
    r = np.random.default_rng(seed)
    lens = r.integers(5, 40, B)
    T, N = int(lens.sum()), int(lens.max())
    dev = "cuda"
    s = dict(T=T, N=N, vocab=vocab, offsets=wl.offsets_from_lengths(lens))
    s["off"] = torch.tensor(s["offsets"], dtype=torch.int32, device=dev)
    s["ids"] = torch.tensor(r.integers(-1, vocab, T), dtype=torch.int32, device=dev)
    s["table"] = lt.randn((vocab, DM), dtype, seed + 1, DM ** -0.5)
    for n, i in (("n1", 2), ("n2", 3)):
        s[n] = (1 + lt.randn((DM,), torch.float32, seed + i, 0.1)).to(dtype)
    s["w1"], s["b1"] = lt.randn((4 * DM, DM), dtype, seed + 4, DM ** -0.5), lt.randn((4 * DM,), dtype, seed + 5, 0.1)
    s["w2"] = lt.randn((DM, DM), dtype, seed + 6, DM ** -0.5)
    s["dy"] = lt.randn((T, DM), dtype, seed + 7)
    s["func"] = hb.build_func("causal", s["off"], T, N, 1)
    return s


def _forward(s):
    T, alpha = s["T"], 1.0 / math.sqrt(D)
    k = {}
    k["h"] = hb.embed(s["table"], s["ids"], math.sqrt(DM))
    k["a"], _, k["r1"] = hb.rms_norm(k["h"], s["n1"], eps=EPS)
    k["p"], k["z"] = hb.linear(k["a"], s["w1"], bias=s["b1"], act="silu", want_z=True)
    u, v, q, kk = (k["p"][:, i * DM:(i + 1) * DM] for i in range(4))
    k["u"] = u
    k["v"], k["q"], k["k"] = (t.contiguous().view(T, H, D) for t in (v, q, kk))
    k["o"] = hb.fwd(k["q"], k["k"], k["v"], s["off"], s["func"], s["N"], alpha).view(T, DM)
    k["g"], _, k["r2"] = hb.rms_norm(k["o"], s["n2"], gate=u, eps=EPS)
    k["y"], _ = hb.linear(k["g"], s["w2"], residual=k["h"])
    return k


def _backward(s, k):
    T, alpha = s["T"], 1.0 / math.sqrt(D)
    out = {}
    dg, out["w2"], _ = hb.linear_bwd(s["dy"], None, k["g"], s["w2"], want_dbias=False)
    do, out["n2"], du = hb.rms_norm_bwd(dg, k["o"], k["r2"], s["n2"], gate=k["u"])
    dq, dk, dv = hb.bwd(do.view(T, H, D), k["q"], k["k"], k["v"], s["off"], s["func"], s["N"], alpha)
    dp = torch.cat([du, dv.view(T, DM), dq.view(T, DM), dk.view(T, DM)], 1)
    da, out["w1"], out["b1"] = hb.linear_bwd(dp, k["z"], k["a"], s["w1"], act="silu")
    dh, out["n1"], _ = hb.rms_norm_bwd(da, k["h"], k["r1"], s["n1"], dh=s["dy"])
    out["table"] = hb.embed_bwd(dh, s["ids"], s["vocab"], math.sqrt(DM))
    return out


def _plain(s, p):
    """The layer in 64 bits, of parameters p (a dict of numpy arrays)."""
    h = lt.embed(p["table"], s["ids"].cpu().numpy(), math.sqrt(DM))
    a, _ = lt.norm(h, p["n1"], eps=EPS)
    z = a @ p["w1"].T + p["b1"]
    x = lt.act(z, "silu")
    u, v, q, k = (x[:, i * DM:(i + 1) * DM] for i in range(4))
    sh = lambda t: t.reshape(-1, H, D)  # noqa: E731
    func = s["func"].cpu().numpy()
    o = orc.fwd_dense(sh(q), sh(k), sh(v), s["offsets"], func, 1, s["N"], 1.0 / math.sqrt(D)).reshape(-1, DM)
    g, _ = lt.norm(o, p["n2"], u, EPS)
    return g @ p["w2"].T + h


def _params(s):
    return {n: lt.f64(s[n]) for n in ("table", "n1", "n2", "w1", "b1", "w2")}


def _rel(a, b):
    return float(np.linalg.norm(a - b) / np.linalg.norm(b))


# Roundings from one operator to the next (rows, projections, q k v, P and O of the
# attention, gated rows, y; as many back): 16 of a relative half step each in the
# 2-norm, each passed on by at most 4 (the attention divides small sums by their own rms).
def _bound(dtype):
    return 16 * 4 * lt.half_step(dtype)


def test_forward():
    s = _layer(F16)
    assert _rel(lt.f64(_forward(s)["y"]), _plain(s, _params(s))) <= _bound(F16)


@pytest.mark.parametrize("name", ["table", "n1", "n2", "w1", "b1", "w2"])
def test_gradients_against_differences(name):
    s = _layer(F16, seed=3)
    got = lt.f64(_backward(s, _forward(s))[name])
    p, dy = _params(s), lt.f64(s["dy"])
    r = np.random.default_rng(1)
    e = 1e-5
    for _ in range(3):
        # along the gradient itself, turned a little: a slope of about its norm
        v = got / np.linalg.norm(got) + 0.2 * r.standard_normal(got.shape) / math.sqrt(got.size)
        f = lambda x: (_plain(s, {**p, name: p[name] + x * v}) * dy).sum()  # noqa: E731
        slope = (f(e) - f(-e)) / (2 * e)
        assert abs((got * v).sum() - slope) <= _bound(F16) * np.linalg.norm(got) * np.linalg.norm(v)


def test_captured_and_replayed():
    """Forward and backward in one graph, replayed on other inputs: what an eager run gives."""
    s, other = _layer(BF, seed=1), _layer(BF, seed=1)
    other["dy"] = lt.randn(tuple(s["dy"].shape), BF, 99)
    other["ids"] = (s["ids"] + 7) % s["vocab"]
    want = {n: _backward(x, _forward(x)) for n, x in (("s", s), ("o", other))}
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        _backward(s, _forward(s))
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = _backward(s, _forward(s))
    for name, x in (("s", {"dy": s["dy"].clone(), "ids": s["ids"].clone()}), ("o", other), ("s", None)):
        if x is None:
            x = first
        elif name == "s":
            first = x
        s["dy"].copy_(x["dy"])
        s["ids"].copy_(x["ids"])
        graph.replay()
        torch.cuda.synchronize()
        for n in want[name]:
            assert torch.equal(got[n], want[name][n]), n


def test_two_streams_at_once():
    layers = [_layer(BF, seed=i) for i in range(2)]
    want = [_backward(s, _forward(s)) for s in layers]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in layers]
    got = []
    for _ in range(5):
        got = []
        for s, st in zip(layers, streams):
            with torch.cuda.stream(st):
                got.append(_backward(s, _forward(s)))
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        for n in b:
            assert torch.equal(a[n], b[n]), n


def test_threads_at_once():
    """Threads with a stream each, whose calls take every kind of product and sort: pairs with whole and half tiles,
    few rows, one block's sort and several."""
    sizes = [(4500, 136, 528), (5000, 72, 1040), (64, 512, 1024), (600, 264, 336)]

    def work(i):
        T, K, N = sizes[i]
        x, w, dy = lt.randn((T, K), BF, i), lt.randn((N, K), BF, 10 + i, K ** -0.5), lt.randn((T, N), BF, 20 + i)
        ids = torch.randint(-1, 500, (T,), generator=torch.Generator("cuda").manual_seed(i), device="cuda")
        q, qw = hb.quantise_rows(dy), hb.quantise_rows(w.t().contiguous())
        nw = lt.randn((K,), BF, 30 + i)
        torch.cuda.current_stream().synchronize()

        def once():
            a, _, rstd = hb.rms_norm(x, nw)
            y, z = hb.linear(a, w, act="silu", want_z=True)
            dx, dw, db = hb.linear_bwd(dy, z, a, w, act="silu")
            back, dn, _ = hb.rms_norm_bwd(dx, x, rstd, nw)
            return [y, dx, dw, db, back, dn, hb.embed_bwd(back, ids, 500), hb.linear(q, qw)[0]]
        return once
    calls = [work(i) for i in range(len(sizes))]
    want = [once() for once in calls]
    torch.cuda.synchronize()
    got, errors = [None] * len(calls), []

    def run(i):
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                for _ in range(20):
                    got[i] = calls[i]()
                torch.cuda.current_stream().synchronize()
        except Exception as e:  # noqa: BLE001
            errors.append(e)
    threads = [threading.Thread(target=run, args=(i,)) for i in range(len(calls))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors, errors
    for a, b in zip(got, want):
        assert all(torch.equal(x, y) for x, y in zip(a, b))


def test_a_stream_given():
    s = _layer(BF)
    want = _forward(s)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    h = hb.embed(s["table"], s["ids"], math.sqrt(DM), stream=st)
    a, _, r = hb.rms_norm(h, s["n1"], eps=EPS, stream=st)
    p, z = hb.linear(a, s["w1"], bias=s["b1"], act="silu", want_z=True, stream=st)
    dx, dw, db = hb.linear_bwd(p, z, a, s["w1"], act="silu", stream=st)
    dh, dn, _ = hb.rms_norm_bwd(dx, h, r, s["n1"], stream=st)
    dt = hb.embed_bwd(dh, s["ids"], s["vocab"], stream=st)
    q = hb.quantise_rows(a, stream=st)
    st.synchronize()
    assert torch.equal(h, want["h"]) and torch.equal(p, want["p"])
    want_dx, want_dw, want_db = hb.linear_bwd(p, z, a, s["w1"], act="silu")
    want_dh, want_dn, _ = hb.rms_norm_bwd(dx, h, r, s["n1"])
    for x, y in ((dx, want_dx), (dw, want_dw), (db, want_db), (dh, want_dh), (dn, want_dn),
                 (dt, hb.embed_bwd(dh, s["ids"], s["vocab"])), (q.codes, hb.quantise_rows(a).codes)):
        assert torch.equal(x, y)


@pytest.mark.parametrize("rows", [1, 64, 300])
def test_through_eight_bits(rows):
    """A decode step's norm and projection: the projection of the codes' values."""
    K, N = 512, 2048
    x, r = lt.randn((rows, K), BF, 1), lt.randn((rows, K), BF, 2)
    w, nw = lt.randn((N, K), BF, 3, K ** -0.5), lt.randn((K,), BF, 4)
    b, qw = lt.randn((N,), BF, 5), hb.quantise_rows(w)
    q, h, _ = hb.rms_norm(x, nw, residual=r, quantise=True)
    y, _ = hb.linear(q, qw, bias=b, act="silu")
    values = lambda t: lt.e4m3(t.codes) * lt.scale_of(t.scale)[:, None]  # noqa: E731
    A, W = values(q), values(qw)
    z = A @ W.T + lt.f64(b)
    err = lt.product_err(A, W.T) + lt.STEP32 * np.abs(z)
    ref = lt.act(z, "silu")
    tol = 1.2 * err + lt.act_rel(z, "silu") * np.abs(ref) + lt.half_step(BF) * (np.abs(ref) + 1.2 * err) + 1e-15
    assert lt.worst(lt.f64(y), ref, tol) <= 1.0
    # and near the layer in 16 bits: codes of both operands, half a step of 2^-4 each, K of them by chance
    # of either sign
    y16, _ = hb.linear(hb.rms_norm(x, nw, residual=r)[0], w, bias=b, act="silu")
    assert _rel(lt.f64(y), lt.f64(y16)) <= 2 * 2.0 ** -4


def test_one_workspace_for_calls_in_turn():
    """A stream's calls share a workspace of the largest one's size."""
    T, V = 700, 900
    big = hb.embed_workspace(T, V, 64)
    for n in (T, 3, 250):
        dy, ids = lt.randn((n, 64), BF, n), torch.randint(0, V, (n,), device="cuda")
        assert torch.equal(hb.embed_bwd(dy, ids, V, ws=big), hb.embed_bwd(dy, ids, V))
    big = hb.linear_workspace(T, 64, 72, "silu")
    for n in (T, 5, 300):
        x, w, dy = lt.randn((n, 64), BF, n), lt.randn((72, 64), BF, 1), lt.randn((n, 72), BF, 2)
        z = hb.linear(x, w, act="silu", want_z=True)[1]
        for a, b in zip(hb.linear_bwd(dy, z, x, w, act="silu", ws=big), hb.linear_bwd(dy, z, x, w, act="silu")):
            assert torch.equal(a, b)


def test_another_current_device_is_refused():
    if torch.cuda.device_count() > 1:
        x = torch.zeros((4, 64), dtype=BF, device="cuda:1")
        with pytest.raises(ValueError, match="current device"):
            hb.quantise_rows(x)
