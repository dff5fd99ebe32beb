"""Thin Python binding of the C ABI in ``include/hstu_attn.h``.

Argument marshalling only: every step of the computation runs in the CUDA
library. Tensors are torch CUDA tensors (torch supplies device memory and the
current stream); the library is loaded with ctypes from this directory and the
binding raises if it is missing -- there is no fallback path.
"""
from __future__ import annotations

import ctypes
import math
import os
from typing import Optional, Tuple

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libhstu_attn.so")
# The same entry points compiled with device-side index checks (see
# hstu_attn.h); select_library() switches the wrappers below to it.
CHECKED_LIB_PATH = os.path.join(_HERE, "libhstu_attn_checked.so")

HSTU_OK = 0
STATUS_NAMES = {
    0: "HSTU_OK", 1: "HSTU_ERR_INVALID_ARG", 2: "HSTU_ERR_UNSUPPORTED", 3: "HSTU_ERR_WORKSPACE",
    4: "HSTU_ERR_CUDA", 5: "HSTU_ERR_DEVICE_INPUT", 6: "HSTU_ERR_TIMEOUT", 7: "HSTU_ERR_DEVICE_CHECK",
}
WS_FULL = 0
WS_TARGETS = 1
FLAG_REUSE_PLAN = 1

EXPORTED = (
    "hstu_attn_nfunc_supported", "hstu_attn_workspace_size", "hstu_attn_plan", "hstu_attn_fwd",
    "hstu_attn_bwd", "hstu_attn_fwd_targets_only", "hstu_attn_bwd_targets_only",
    "hstu_attn_get_device_status", "hstu_status_string", "hstu_attn_fwd_noalloc",
    "hstu_attn_shard_sequences", "hstu_attn_test_wait_timeout", "hstu_attn_build_func",
    "hstu_attn_build_func_candidates", "hstu_attn_targets_workspace_size", "hstu_attn_fwd_targets",
    "hstu_attn_bwd_targets", "hstu_attn_project_workspace_size", "hstu_attn_project_rows",
    "hstu_attn_project_rows_bwd", "hstu_attn_test_set_handoff_limit", "hstu_attn_rope_table", "hstu_attn_rope",
    "hstu_attn_cache_write", "hstu_attn_cache_read", "hstu_attn_paged_workspace_size", "hstu_attn_fwd_paged",
    "hstu_attn_cache_read_zeroed", "hstu_attn_embed", "hstu_attn_embed_workspace_size", "hstu_attn_embed_bwd",
    "hstu_attn_rms_norm", "hstu_attn_quantise_rows", "hstu_attn_rms_norm_workspace_size", "hstu_attn_rms_norm_bwd",
    "hstu_attn_linear", "hstu_attn_linear_workspace_size", "hstu_attn_linear_bwd",
)
FUNC_CAUSAL, FUNC_SLA, FUNC_ONERANK = 0, 1, 2
NOALLOC_SCRATCH_BYTES = 8 << 20


class HstuError(RuntimeError):
    def __init__(self, status: int, what: str):
        self.status = status
        super().__init__(f"{what}: {STATUS_NAMES.get(status, status)} ({status_string(status)})")


class FuncSpec(ctypes.Structure):
    _fields_ = [
        ("kind", ctypes.c_int32),
        ("k1", ctypes.c_int32),
        ("k2", ctypes.c_int32),
        ("groups", ctypes.c_int32),
        ("task_tokens", ctypes.c_int32),
    ]


class Shape(ctypes.Structure):
    _fields_ = [
        ("batch", ctypes.c_int32),
        ("total", ctypes.c_int64),
        ("num_heads", ctypes.c_int32),
        ("head_dim", ctypes.c_int32),
        ("nfunc", ctypes.c_int32),
        ("max_seqlen", ctypes.c_int32),
        ("alpha", ctypes.c_float),
        ("head_dim_v", ctypes.c_int32),
        ("dtype", ctypes.c_int32),
    ]


class RopeSpec(ctypes.Structure):
    _fields_ = [
        ("rotary_dim", ctypes.c_int32),
        ("scaling", ctypes.c_int32),
        ("base", ctypes.c_double),
        ("factor", ctypes.c_double),
        ("original_len", ctypes.c_double),
        ("fast_turns", ctypes.c_double),
        ("slow_turns", ctypes.c_double),
    ]


class Rope(ctypes.Structure):
    _fields_ = [
        ("turns", ctypes.c_void_p),
        ("rotary_dim", ctypes.c_int32),
        ("interleaved", ctypes.c_int32),
        ("magnitude", ctypes.c_float),
    ]


class Cache(ctypes.Structure):
    _fields_ = [
        ("k", ctypes.c_void_p),
        ("v", ctypes.c_void_p),
        ("k_scale", ctypes.c_void_p),
        ("v_scale", ctypes.c_void_p),
        ("num_pages", ctypes.c_int64),
        ("page_size", ctypes.c_int32),
        ("num_heads", ctypes.c_int32),
        ("head_dim", ctypes.c_int32),
        ("head_dim_v", ctypes.c_int32),
        ("dtype", ctypes.c_int32),
        ("e4m3", ctypes.c_int32),
    ]


_libs = {}
_active = LIB_PATH


def select_library(path: str) -> str:
    """Makes the wrappers of this module call the library at ``path`` (the
    release or the checked build); returns the previously selected path."""
    global _active
    prev, _active = _active, path
    return prev


def load(path: str = None) -> ctypes.CDLL:
    """Loads the selected library (once per path). Raises if it has not been
    built."""
    path = _active if path is None else path
    if path in _libs:
        return _libs[path]
    if not os.path.exists(path):
        raise RuntimeError(
            f"CUDA library {path} is missing: build it first "
            "(python -c 'import __graft_entry__ as g; g.build()')")
    lib = ctypes.CDLL(path)
    vp, i32, u32, sz = ctypes.c_void_p, ctypes.c_int32, ctypes.c_uint32, ctypes.c_size_t
    i64, sp = ctypes.c_int64, ctypes.POINTER(Shape)
    sig = {
        "hstu_attn_nfunc_supported": (ctypes.c_int, [i32]),
        "hstu_attn_workspace_size": (sz, [sp, i32]),
        "hstu_attn_plan": (ctypes.c_int, [vp, vp, sp, vp, vp, sz, vp]),
        "hstu_attn_fwd": (ctypes.c_int, [vp, vp, vp, vp, vp, vp, sp, vp, vp, sz, u32, vp]),
        "hstu_attn_bwd": (ctypes.c_int, [vp, vp, vp, vp, vp, vp, vp, vp, vp, sp, vp, sz, u32, vp]),
        "hstu_attn_fwd_targets_only": (ctypes.c_int, [vp, vp, vp, vp, vp, vp, sp, vp, sz, vp]),
        "hstu_attn_bwd_targets_only": (ctypes.c_int, [vp, vp, vp, vp, vp, vp, vp, vp, vp, sp, vp, sz, vp]),
        "hstu_attn_get_device_status": (ctypes.c_int, [vp, vp]),
        "hstu_status_string": (ctypes.c_char_p, [ctypes.c_int]),
        "hstu_attn_fwd_noalloc": (ctypes.c_int, [vp, vp, vp, vp, vp, vp, sp, vp, vp]),
        "hstu_attn_shard_sequences": (ctypes.c_int, [vp, i32, i32, vp, vp]),
        "hstu_attn_test_wait_timeout": (ctypes.c_int, [vp, i32, vp]),
        "hstu_attn_test_set_handoff_limit": (ctypes.c_int, [ctypes.c_uint64]),
        "hstu_attn_build_func": (ctypes.c_int, [ctypes.POINTER(FuncSpec), vp, i32, ctypes.c_int64, i32, i32, vp,
                                                vp]),
        "hstu_attn_build_func_candidates": (ctypes.c_int, [vp, i32, i32, vp, vp]),
        "hstu_attn_targets_workspace_size": (sz, [sp, ctypes.c_int64]),
        "hstu_attn_project_workspace_size": (sz, [ctypes.c_int64, i32, i32, i32]),
        "hstu_attn_project_rows": (ctypes.c_int, [vp, ctypes.c_int64, vp, ctypes.c_int64, vp, vp, i32, i32, i32, vp,
                                                  vp, vp, sz, vp]),
        "hstu_attn_project_rows_bwd": (ctypes.c_int, [vp, vp, vp, ctypes.c_int64, vp, ctypes.c_int64, vp, i32, i32,
                                                      i32, vp, vp, vp, vp, sz, vp]),
        "hstu_attn_fwd_targets": (ctypes.c_int, [vp, vp, vp, vp, vp, vp, ctypes.c_int64, vp, sp, vp, sz, vp]),
        "hstu_attn_bwd_targets": (ctypes.c_int, [vp, vp, vp, vp, vp, vp, vp, vp, vp, ctypes.c_int64, vp, sp, vp,
                                                 sz, vp]),
        "hstu_attn_rope_table": (ctypes.c_int, [ctypes.POINTER(RopeSpec), vp, ctypes.POINTER(ctypes.c_float)]),
        "hstu_attn_rope": (ctypes.c_int, [vp, i64, vp, i64, vp, i64, vp, i64, vp, i64, i32, i32, i32, vp, i32, vp]),
        "hstu_attn_cache_write": (ctypes.c_int, [vp, vp, i64, vp, i64, vp, i32, i64, vp, vp, i32, vp, vp, vp, sz,
                                                 vp]),
        "hstu_attn_cache_read": (ctypes.c_int, [vp, vp, vp, vp, i32, i64, vp, vp, i32, vp, sz, vp]),
        "hstu_attn_cache_read_zeroed": (ctypes.c_int, [vp, vp, vp, vp, i32, i64, vp, vp, i32, vp, sz, vp]),
        "hstu_attn_paged_workspace_size": (sz, [vp, i32, i64, i32]),
        "hstu_attn_fwd_paged": (ctypes.c_int, [vp, i64, vp, vp, vp, i32, vp, i32, vp, i64, vp, i32, i32,
                                               ctypes.c_float, vp, sz, u32, vp]),
        "hstu_attn_embed": (ctypes.c_int, [vp, i32, i64, i32, vp, i32, i64, ctypes.c_float, vp, i32, vp, sz, vp]),
        "hstu_attn_embed_workspace_size": (sz, [i64, i64, i32]),
        "hstu_attn_embed_bwd": (ctypes.c_int, [vp, i64, i32, vp, i32, i64, ctypes.c_float, vp, i32, i64, i32, i32, vp,
                                               sz, vp]),
        "hstu_attn_rms_norm": (ctypes.c_int, [vp, i64, vp, i64, vp, i64, vp, i64, i32, i32, ctypes.c_float, vp, vp, vp,
                                              vp, vp]),
        "hstu_attn_quantise_rows": (ctypes.c_int, [vp, i64, i64, i32, i32, vp, vp, vp]),
        "hstu_attn_rms_norm_workspace_size": (sz, [i64, i32]),
        "hstu_attn_rms_norm_bwd": (ctypes.c_int, [vp, i64, vp, i64, vp, vp, vp, i64, vp, i64, i64, i32, i32, vp, vp,
                                                  vp, vp, sz, vp]),
        "hstu_attn_linear": (ctypes.c_int, [vp, i64, vp, vp, vp, vp, vp, i64, i64, i32, i32, i32, i32, vp, vp, vp, sz,
                                            vp]),
        "hstu_attn_linear_workspace_size": (sz, [i64, i32, i32, i32]),
        "hstu_attn_linear_bwd": (ctypes.c_int, [vp, i64, vp, vp, i64, vp, i64, i32, i32, i32, i32, vp, vp, vp, vp, sz,
                                                vp]),
    }
    for name, (res, args) in sig.items():
        fn = getattr(lib, name)
        fn.restype = res
        fn.argtypes = args
    _libs[path] = lib
    return lib


def status_string(status: int) -> str:
    try:
        return load().hstu_status_string(status).decode()
    except Exception:  # library missing: still format the error
        return STATUS_NAMES.get(status, "unknown")


def _check(status: int, what: str):
    if status != HSTU_OK:
        raise HstuError(status, what)


def _ptr(t: Optional[torch.Tensor]):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream: Optional[torch.cuda.Stream] = None):
    s = stream if stream is not None else torch.cuda.current_stream()
    return ctypes.c_void_p(s.cuda_stream)


def _need(t: torch.Tensor, dtype, name: str):
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if isinstance(dtype, tuple):
        if t.dtype not in dtype:
            raise ValueError(f"{name} must be one of {dtype}, got {t.dtype}")
    elif t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


DTYPES = {torch.bfloat16: 0, torch.float16: 1}
_FLOATS = tuple(DTYPES)


def _same_dtype(*ts):
    d = ts[0].dtype
    for t in ts[1:]:
        if t.dtype != d:
            raise ValueError(f"all tensors must share one dtype, got {d} and {t.dtype}")
    return DTYPES[d]


def make_shape(batch: int, total: int, heads: int, dim: int, nfunc: int, max_seqlen: int,
               alpha: Optional[float] = None, dim_v: int = 0, dtype: int = 0) -> Shape:
    """The C shape struct. ``dim`` is D_qk, ``dim_v`` D_v (0: equal to D_qk),
    ``dtype`` 0 for bf16 and 1 for fp16."""
    if alpha is None:
        alpha = 1.0 / math.sqrt(dim)
    return Shape(batch, total, heads, dim, nfunc, max_seqlen, alpha, dim_v, dtype)


def nfunc_supported(nfunc: int) -> bool:
    return bool(load().hstu_attn_nfunc_supported(nfunc))


def workspace_size(shape: Shape, mode: int = WS_FULL) -> int:
    return int(load().hstu_attn_workspace_size(ctypes.byref(shape), mode))


def alloc_workspace(shape: Shape, mode: int = WS_FULL, device="cuda") -> torch.Tensor:
    n = workspace_size(shape, mode)
    if n == 0:
        raise HstuError(2, "workspace_size")
    return torch.empty(n, dtype=torch.uint8, device=device)


def _shape_full(q, v, seq_offsets, func, max_seqlen, alpha):
    T, H, D = q.shape
    return make_shape(seq_offsets.numel() - 1, T, H, D, func.shape[0], max_seqlen, alpha, dim_v=v.shape[2],
                      dtype=DTYPES[q.dtype])


def plan(seq_offsets, func, shape: Shape, ws: torch.Tensor, row_counts=None, stream=None):
    _need(seq_offsets, torch.int32, "seq_offsets")
    _need(func, torch.int32, "func")
    _check(load().hstu_attn_plan(_ptr(seq_offsets), _ptr(func), ctypes.byref(shape), _ptr(row_counts),
                                 _ptr(ws), ws.numel(), _stream(stream)), "hstu_attn_plan")


def fwd(q, k, v, seq_offsets, func, max_seqlen: int, alpha: Optional[float] = None,
        ws: Optional[torch.Tensor] = None, row_counts: Optional[torch.Tensor] = None,
        reuse_plan: bool = False, out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """o = HSTU attention over the jagged batch (see include/hstu_attn.h).
    q, k are (T, H, D_qk) and v (T, H, D_v), all bf16 or all fp16; o is
    (T, H, D_v)."""
    for t, n in ((q, "q"), (k, "k"), (v, "v")):
        _need(t, _FLOATS, n)
    _same_dtype(q, k, v)
    _need(seq_offsets, torch.int32, "seq_offsets")
    _need(func, torch.int32, "func")
    shape = _shape_full(q, v, seq_offsets, func, max_seqlen, alpha)
    if ws is None:
        ws = alloc_workspace(shape, WS_FULL, q.device)
    o = q.new_empty((q.shape[0], q.shape[1], v.shape[2])) if out is None else out
    flags = FLAG_REUSE_PLAN if reuse_plan else 0
    _check(load().hstu_attn_fwd(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(seq_offsets), _ptr(func),
                                ctypes.byref(shape), _ptr(row_counts), _ptr(ws), ws.numel(), flags,
                                _stream(stream)), "hstu_attn_fwd")
    return o


def bwd(do, q, k, v, seq_offsets, func, max_seqlen: int, alpha: Optional[float] = None,
        ws: Optional[torch.Tensor] = None, reuse_plan: bool = False, outs=None,
        stream=None) -> Tuple[torch.Tensor, torch.Tensor, torch.Tensor]:
    """(dq, dk, dv) of sum(o * do)."""
    for t, n in ((do, "dout"), (q, "q"), (k, "k"), (v, "v")):
        _need(t, _FLOATS, n)
    _same_dtype(do, q, k, v)
    _need(seq_offsets, torch.int32, "seq_offsets")
    _need(func, torch.int32, "func")
    shape = _shape_full(q, v, seq_offsets, func, max_seqlen, alpha)
    if ws is None:
        ws = alloc_workspace(shape, WS_FULL, q.device)
    dq, dk, dv = outs if outs is not None else (torch.empty_like(q), torch.empty_like(k), torch.empty_like(v))
    flags = FLAG_REUSE_PLAN if reuse_plan else 0
    _check(load().hstu_attn_bwd(_ptr(do), _ptr(q), _ptr(k), _ptr(v), _ptr(dq), _ptr(dk), _ptr(dv),
                                _ptr(seq_offsets), _ptr(func), ctypes.byref(shape), _ptr(ws), ws.numel(),
                                flags, _stream(stream)), "hstu_attn_bwd")
    return dq, dk, dv


def _shape_targets(q_c, k, v, seq_offsets, func_c, max_seqlen, alpha):
    B, H, D = q_c.shape
    return make_shape(B, k.shape[0], H, D, func_c.shape[0], max_seqlen, alpha, dim_v=v.shape[2],
                      dtype=DTYPES[q_c.dtype])


def fwd_targets_only(q_c, k, v, seq_offsets, func_c, max_seqlen: int, alpha: Optional[float] = None,
                     ws: Optional[torch.Tensor] = None, out=None, stream=None) -> torch.Tensor:
    for t, n in ((q_c, "q_c"), (k, "k"), (v, "v")):
        _need(t, _FLOATS, n)
    _same_dtype(q_c, k, v)
    _need(seq_offsets, torch.int32, "seq_offsets")
    _need(func_c, torch.int32, "func_c")
    shape = _shape_targets(q_c, k, v, seq_offsets, func_c, max_seqlen, alpha)
    if ws is None:
        ws = alloc_workspace(shape, WS_TARGETS, q_c.device)
    o_c = q_c.new_empty((q_c.shape[0], q_c.shape[1], v.shape[2])) if out is None else out
    _check(load().hstu_attn_fwd_targets_only(_ptr(q_c), _ptr(k), _ptr(v), _ptr(o_c), _ptr(seq_offsets),
                                             _ptr(func_c), ctypes.byref(shape), _ptr(ws), ws.numel(),
                                             _stream(stream)), "hstu_attn_fwd_targets_only")
    return o_c


def bwd_targets_only(do_c, q_c, k, v, seq_offsets, func_c, max_seqlen: int,
                     alpha: Optional[float] = None, ws: Optional[torch.Tensor] = None, outs=None,
                     stream=None):
    for t, n in ((do_c, "dout_c"), (q_c, "q_c"), (k, "k"), (v, "v")):
        _need(t, _FLOATS, n)
    _same_dtype(do_c, q_c, k, v)
    _need(seq_offsets, torch.int32, "seq_offsets")
    _need(func_c, torch.int32, "func_c")
    shape = _shape_targets(q_c, k, v, seq_offsets, func_c, max_seqlen, alpha)
    if ws is None:
        ws = alloc_workspace(shape, WS_TARGETS, q_c.device)
    dq_c, dk, dv = outs if outs is not None else (torch.empty_like(q_c), torch.empty_like(k),
                                                  torch.empty_like(v))
    _check(load().hstu_attn_bwd_targets_only(_ptr(do_c), _ptr(q_c), _ptr(k), _ptr(v), _ptr(dq_c), _ptr(dk),
                                             _ptr(dv), _ptr(seq_offsets), _ptr(func_c), ctypes.byref(shape),
                                             _ptr(ws), ws.numel(), _stream(stream)),
           "hstu_attn_bwd_targets_only")
    return dq_c, dk, dv


def device_status(ws: torch.Tensor, stream=None) -> int:
    """Synchronises the stream and returns the workspace status code."""
    return int(load().hstu_attn_get_device_status(_ptr(ws), _stream(stream)))


def fwd_noalloc(q, k, v, seq_offsets, func, max_seqlen: int, alpha: Optional[float] = None,
                row_counts: Optional[torch.Tensor] = None, out: Optional[torch.Tensor] = None,
                stream=None) -> torch.Tensor:
    """Forward pass for callers that cannot allocate device memory: the plan's
    scratch is a fixed array inside the library (hstu_attn_fwd_noalloc).
    ``out`` lets the caller supply the output buffer too."""
    for t, n in ((q, "q"), (k, "k"), (v, "v")):
        _need(t, _FLOATS, n)
    _same_dtype(q, k, v)
    _need(seq_offsets, torch.int32, "seq_offsets")
    _need(func, torch.int32, "func")
    shape = _shape_full(q, v, seq_offsets, func, max_seqlen, alpha)
    o = q.new_empty((q.shape[0], q.shape[1], v.shape[2])) if out is None else out
    _check(load().hstu_attn_fwd_noalloc(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(seq_offsets), _ptr(func),
                                        ctypes.byref(shape), _ptr(row_counts), _stream(stream)),
           "hstu_attn_fwd_noalloc")
    return o


def shard_sequences(cost, world: int) -> Tuple[torch.Tensor, torch.Tensor]:
    """Splits a batch over ``world`` data-parallel ranks by whole sequences
    (hstu_attn_shard_sequences, host-only). ``cost`` is one non-negative work
    estimate per sequence. Returns (owner, rank_load): the rank of each
    sequence (int32) and each rank's total cost (int64), as CPU tensors."""
    c = torch.as_tensor(cost, dtype=torch.int64).contiguous()
    if c.dim() != 1 or c.is_cuda:
        raise ValueError("cost must be a 1-D host array")
    owner = torch.empty(c.numel(), dtype=torch.int32)
    load_ = torch.empty(max(world, 0), dtype=torch.int64)
    _check(load().hstu_attn_shard_sequences(_ptr(c), c.numel(), world, _ptr(owner), _ptr(load_)),
           "hstu_attn_shard_sequences")
    return owner, load_


def selftest_wait_timeout(ws: torch.Tensor, limit_ms: int, stream=None) -> None:
    """Enqueues the failure-path test of the in-kernel waits
    (hstu_attn_test_wait_timeout): a wait that nothing ends gives up after
    ``limit_ms`` and records HSTU_ERR_TIMEOUT in ``ws``."""
    _check(load().hstu_attn_test_wait_timeout(_ptr(ws), int(limit_ms), _stream(stream)),
           "hstu_attn_test_wait_timeout")


_KINDS = {"causal": FUNC_CAUSAL, "sla": FUNC_SLA, "onerank": FUNC_ONERANK}


def build_func(mask: str, seq_offsets: torch.Tensor, total: int, max_seqlen: int, nfunc: int, k1: int = 0,
               k2: int = 0, groups: int = 8, task_tokens: int = 3, out: Optional[torch.Tensor] = None,
               stream=None) -> torch.Tensor:
    """func (nfunc, total) int32 of a mask family, built on the device
    (hstu_attn_build_func). ``mask`` is "causal", "sla" or "onerank"."""
    _need(seq_offsets, torch.int32, "seq_offsets")
    if mask not in _KINDS:
        raise ValueError(f"mask must be one of {sorted(_KINDS)}")
    spec = FuncSpec(_KINDS[mask], k1, k2, groups, task_tokens)
    func = torch.empty((nfunc, total), dtype=torch.int32, device=seq_offsets.device) if out is None else out
    _check(load().hstu_attn_build_func(ctypes.byref(spec), _ptr(seq_offsets), seq_offsets.numel() - 1, total,
                                       max_seqlen, nfunc, _ptr(func), _stream(stream)), "hstu_attn_build_func")
    return func


def build_func_candidates(seq_offsets: torch.Tensor, nfunc: int = 1, out: Optional[torch.Tensor] = None,
                          stream=None) -> torch.Tensor:
    """func_c (nfunc, batch) int32 of the targets-only entry points (each
    sequence's last row sees the whole sequence), built on the device."""
    _need(seq_offsets, torch.int32, "seq_offsets")
    B = seq_offsets.numel() - 1
    func_c = torch.empty((nfunc, B), dtype=torch.int32, device=seq_offsets.device) if out is None else out
    _check(load().hstu_attn_build_func_candidates(_ptr(seq_offsets), B, nfunc, _ptr(func_c), _stream(stream)),
           "hstu_attn_build_func_candidates")
    return func_c


def targets_workspace(shape: Shape, num_candidates: int, device="cuda") -> torch.Tensor:
    n = int(load().hstu_attn_targets_workspace_size(ctypes.byref(shape), num_candidates))
    if n == 0:
        raise HstuError(2, "hstu_attn_targets_workspace_size")
    return torch.empty(n, dtype=torch.uint8, device=device)


def _shape_multi(q_c, k, v, seq_offsets, func_c, max_seqlen, alpha):
    C, H, D = q_c.shape
    return make_shape(seq_offsets.numel() - 1, k.shape[0], H, D, func_c.shape[0], max_seqlen, alpha,
                      dim_v=v.shape[2], dtype=DTYPES[q_c.dtype])


def fwd_targets(q_c, k, v, seq_offsets, cand_offsets, func_c, max_seqlen: int, alpha: Optional[float] = None,
                ws: Optional[torch.Tensor] = None, out=None, stream=None) -> torch.Tensor:
    """Targets-only forward with any number of candidates per sequence
    (hstu_attn_fwd_targets): rows cand_offsets[b] .. cand_offsets[b+1] of
    q_c belong to sequence b."""
    for t, n in ((q_c, "q_c"), (k, "k"), (v, "v")):
        _need(t, _FLOATS, n)
    _same_dtype(q_c, k, v)
    for t, n in ((seq_offsets, "seq_offsets"), (cand_offsets, "cand_offsets"), (func_c, "func_c")):
        _need(t, torch.int32, n)
    shape = _shape_multi(q_c, k, v, seq_offsets, func_c, max_seqlen, alpha)
    C = q_c.shape[0]
    if ws is None:
        ws = targets_workspace(shape, C, q_c.device)
    o_c = q_c.new_empty((C, q_c.shape[1], v.shape[2])) if out is None else out
    _check(load().hstu_attn_fwd_targets(_ptr(q_c), _ptr(k), _ptr(v), _ptr(o_c), _ptr(seq_offsets),
                                        _ptr(cand_offsets), C, _ptr(func_c), ctypes.byref(shape), _ptr(ws),
                                        ws.numel(), _stream(stream)), "hstu_attn_fwd_targets")
    return o_c


def bwd_targets(do_c, q_c, k, v, seq_offsets, cand_offsets, func_c, max_seqlen: int,
                alpha: Optional[float] = None, ws: Optional[torch.Tensor] = None, outs=None, stream=None):
    """(dq_c, dk, dv) of the multi-candidate targets-only forward."""
    for t, n in ((do_c, "dout_c"), (q_c, "q_c"), (k, "k"), (v, "v")):
        _need(t, _FLOATS, n)
    _same_dtype(do_c, q_c, k, v)
    for t, n in ((seq_offsets, "seq_offsets"), (cand_offsets, "cand_offsets"), (func_c, "func_c")):
        _need(t, torch.int32, n)
    shape = _shape_multi(q_c, k, v, seq_offsets, func_c, max_seqlen, alpha)
    C = q_c.shape[0]
    if ws is None:
        ws = targets_workspace(shape, C, q_c.device)
    dq_c, dk, dv = outs if outs is not None else (torch.empty_like(q_c), torch.empty_like(k), torch.empty_like(v))
    _check(load().hstu_attn_bwd_targets(_ptr(do_c), _ptr(q_c), _ptr(k), _ptr(v), _ptr(dq_c), _ptr(dk), _ptr(dv),
                                        _ptr(seq_offsets), _ptr(cand_offsets), C, _ptr(func_c),
                                        ctypes.byref(shape), _ptr(ws), ws.numel(), _stream(stream)),
           "hstu_attn_bwd_targets")
    return dq_c, dk, dv


def project_workspace(num_rows: int, d_in: int, d_out: int, backward: bool, device="cuda") -> torch.Tensor:
    n = int(load().hstu_attn_project_workspace_size(num_rows, d_in, d_out, 1 if backward else 0))
    if n == 0:
        raise HstuError(2, "hstu_attn_project_workspace_size")
    return torch.empty(n, dtype=torch.uint8, device=device)


def project_rows(x, w, rows=None, bias=None, want_z=True, ws=None, stream=None):
    """(y, z) = (silu(x[rows] w^T + bias), x[rows] w^T + bias) on the
    listed rows of x (all rows if ``rows`` is None, which ``linear`` with act
    "silu" does faster), hstu_attn_project_rows.
    x (T, d_in), w (d_out, d_in), one dtype (bf16 or fp16)."""
    _need(x, _FLOATS, "x")
    _need(w, _FLOATS, "w")
    ts = [x, w] + ([bias] if bias is not None else [])
    dtype = _same_dtype(*ts)
    if rows is not None:
        _need(rows, torch.int32, "rows")
    n = x.shape[0] if rows is None else rows.numel()
    d_out, d_in = w.shape
    if ws is None:
        ws = project_workspace(n if rows is not None else 0, d_in, d_out, False, x.device)
    y = x.new_empty((n, d_out))
    z = x.new_empty((n, d_out)) if want_z else None
    _check(load().hstu_attn_project_rows(_ptr(x), x.shape[0], _ptr(rows), n, _ptr(w), _ptr(bias), d_in, d_out,
                                         dtype, _ptr(y), _ptr(z), _ptr(ws), ws.numel(), _stream(stream)),
           "hstu_attn_project_rows")
    return y, z


def project_rows_bwd(dy, z, x, w, rows=None, want_dbias=True, ws=None, stream=None):
    """(dx_rows, dw, dbias) of sum(y * dy) for project_rows."""
    for t, name in ((dy, "dy"), (z, "z"), (x, "x"), (w, "w")):
        _need(t, _FLOATS, name)
    dtype = _same_dtype(dy, z, x, w)
    if rows is not None:
        _need(rows, torch.int32, "rows")
    n = x.shape[0] if rows is None else rows.numel()
    d_out, d_in = w.shape
    if ws is None:
        ws = project_workspace(n, d_in, d_out, True, x.device)
    dx = x.new_empty((n, d_in))
    dw = torch.empty_like(w)
    db = w.new_empty((d_out,)) if want_dbias else None
    _check(load().hstu_attn_project_rows_bwd(_ptr(dy), _ptr(z), _ptr(x), x.shape[0], _ptr(rows), n, _ptr(w), d_in,
                                             d_out, dtype, _ptr(dx), _ptr(dw), _ptr(db), _ptr(ws), ws.numel(),
                                             _stream(stream)), "hstu_attn_project_rows_bwd")
    return dx, dw, db


def set_handoff_limit_for_tests(limit_ns: int) -> None:
    """Test hook (hstu_attn_test_set_handoff_limit): shortens the attention
    kernels' and the linear maps' accumulator hand-off wait, and with 1 ns makes the
    waits of ``fwd_paged`` and of ``linear`` of few rows on tensor memory give up;
    0 restores the normal limits."""
    _check(load().hstu_attn_test_set_handoff_limit(int(limit_ns)), "hstu_attn_test_set_handoff_limit")


# ---------------------------------------------------------------- serving
# A decode step is a few microseconds on the GPU. The calls below go through
# the extension of csrc/serving_ext.cpp, which checks the tensors, allocates the
# outputs and calls the selected library's entry points; ctypes and checks in
# Python take three times as long as the step. It launches on the current stream
# and allocates from that stream's memory, so a ``stream`` given is made the
# current one: an output of another stream's memory could still be in use there.

EXT_PATH = os.path.join(_HERE, "_serving.so")
_ext_module = None
_ext_library = None  # the library that the extension calls


def load_extension():
    """The extension, bound to the selected library. Raises if it has not been
    built."""
    global _ext_module, _ext_library
    if _ext_library != _active:
        lib = load()
        if _ext_module is None:
            if not os.path.exists(EXT_PATH):
                raise RuntimeError(f"extension {EXT_PATH} is missing: build it first "
                                   "(python -c 'import __graft_entry__ as g; g.build()')")
            from . import _serving
            _ext_module = _serving
        names = ("rope", "cache_write", "cache_read", "paged_workspace_size", "fwd_paged", "cache_read_zeroed")
        address = lambda n: ctypes.cast(getattr(lib, "hstu_attn_" + n), ctypes.c_void_p).value
        _ext_module.bind(*map(address, names))
        layer = ("embed", "embed_workspace_size", "embed_bwd", "rms_norm", "quantise_rows", "rms_norm_workspace_size",
                 "rms_norm_bwd", "linear", "linear_workspace_size", "linear_bwd")
        _ext_module.bind_layer(*map(address, layer))
        _ext_library = _active
    return _ext_module


_ROPE_SCALINGS = {"none": 0, "linear": 1, "ntk": 2, "yarn": 3}


class RopeTable:
    """A rotation of the first ``rotary_dim`` columns of each head: the pairs'
    frequencies on the device, as ``rope`` and ``cache_write`` take it (see
    hstu_rope_t). Made by ``rope_table``."""

    def __init__(self, turns: torch.Tensor, interleaved: bool, magnitude: float):
        self.turns = turns
        self.rotary_dim = 2 * turns.numel()
        self.interleaved = bool(interleaved)
        self.magnitude = magnitude
        self._c = Rope(turns.data_ptr(), self.rotary_dim, int(self.interleaved), magnitude)
        self._addr = ctypes.addressof(self._c)
        self._device = turns.get_device()


def rope_table(rotary_dim: int, base: float = 10000.0, scaling: str = "none", factor: float = 1.0,
               original_len: float = 0.0, fast_turns: float = 32.0, slow_turns: float = 1.0,
               interleaved: bool = False, device="cuda") -> RopeTable:
    """The frequencies of a rotation (hstu_attn_rope_table), made once and
    kept. ``scaling`` is "none", "linear", "ntk" or "yarn"; ``factor`` is how
    many times longer than trained the contexts are, ``original_len`` the
    trained length (yarn only)."""
    if scaling not in _ROPE_SCALINGS:
        raise ValueError(f"scaling must be one of {sorted(_ROPE_SCALINGS)}")
    spec = RopeSpec(int(rotary_dim), _ROPE_SCALINGS[scaling], base, factor, original_len, fast_turns, slow_turns)
    turns = torch.zeros(max(int(rotary_dim) // 2, 1), dtype=torch.int64)
    magnitude = ctypes.c_float()
    _check(load().hstu_attn_rope_table(ctypes.byref(spec), turns.data_ptr(), ctypes.byref(magnitude)),
           "hstu_attn_rope_table")
    return RopeTable(turns.to(device), interleaved, magnitude.value)


def rope(q, k, positions, table: RopeTable, backward: bool = False, outs=None, stream=None):
    """(q', k') with the leading columns of every head rotated by the row's
    position (hstu_attn_rope). q and k are (T, H, D), bf16 or fp16, and may be
    slices of a wider projection; k may be None. ``backward=True`` takes the
    gradients of q' and k' to those of q and k. ``outs`` may be (q, k) itself:
    the rows are then rotated in place."""
    if stream is not None:
        with torch.cuda.stream(stream):
            return rope(q, k, positions, table, backward, outs)
    qo, ko = (None, None) if outs is None else outs
    r = load_extension().rope(q, k, positions, table._addr, table._device, bool(backward), qo, ko)
    if type(r) is int:
        _check(r, "hstu_attn_rope")
    return r


class PagedCache:
    """K/V pages on the device (hstu_cache_t). ``k`` is (pages, H, page, D_qk)
    and ``v`` (pages, H, page, D_v): bf16 or fp16, or uint8 holding 8-bit
    floats under the power-of-two scales ``k_scale`` and ``v_scale`` (uint8,
    (pages, H, page)). ``dtype`` is the type of the rows written, read back
    and multiplied (16-bit pages hold it as it is)."""

    def __init__(self, k, v, k_scale=None, v_scale=None, dtype=None):
        e4m3 = k_scale is not None
        dtype = dtype if dtype is not None else k.dtype
        if dtype not in DTYPES:
            raise ValueError(f"dtype must be one of {_FLOATS}, got {dtype}")
        for t, n in ((k, "k"), (v, "v")):
            _need(t, torch.uint8 if e4m3 else dtype, n)
            if t.dim() != 4:
                raise ValueError(f"{n} must be (pages, heads, page, width), got {tuple(t.shape)}")
        if k.shape[:3] != v.shape[:3]:
            raise ValueError("k and v must have the same pages, heads and page size")
        if (v_scale is not None) != e4m3:
            raise ValueError("k_scale and v_scale come together")
        if e4m3:
            for t, n in ((k_scale, "k_scale"), (v_scale, "v_scale")):
                _need(t, torch.uint8, n)
                if t.shape != k.shape[:3]:
                    raise ValueError(f"{n} must have shape {tuple(k.shape[:3])}, got {tuple(t.shape)}")
        for t in (v, k_scale, v_scale):
            if t is not None and t.device != k.device:
                raise ValueError("the cache's tensors must be on one device")
        self.k, self.v, self.k_scale, self.v_scale = k, v, k_scale, v_scale
        self.dtype, self.device, self.quantised = dtype, k.device, e4m3
        self.num_pages, self.heads, self.page_size, self.dim = k.shape
        self.dim_v = v.shape[3]
        addr = lambda t: None if t is None else t.data_ptr()
        self._c = Cache(addr(k), addr(v), addr(k_scale), addr(v_scale), self.num_pages, self.page_size, self.heads,
                        self.dim, self.dim_v, DTYPES[dtype], int(e4m3))
        self._addr = ctypes.addressof(self._c)
        self._device = k.get_device()


def alloc_cache(num_pages: int, page_size: int, heads: int, dim: int, dim_v: int = 0, dtype=torch.bfloat16,
                quantised: bool = False, device="cuda") -> PagedCache:
    """An empty paged cache; its slots hold anything until rows are written."""
    shape = (num_pages, heads, page_size)
    kind = torch.uint8 if quantised else dtype
    new = lambda *s: torch.empty(s, dtype=kind, device=device)
    k, v = new(*shape, dim), new(*shape, dim_v or dim)
    return PagedCache(k, v, new(*shape) if quantised else None, new(*shape) if quantised else None, dtype=dtype)


def cache_write(cache: PagedCache, k, v, seq_offsets, cache_lens, page_table, rope: Optional[RopeTable] = None,
                positions=None, ws: Optional[torch.Tensor] = None, stream=None) -> None:
    """Appends the jagged rows k (T, H, D_qk) and v (T, H, D_v) to their
    sequences' pages behind the ``cache_lens`` rows already there
    (hstu_attn_cache_write); ``rope`` rotates k on its way, by ``positions``
    or by its place in the cache. ``cache_lens`` is not changed. With a ``ws``
    (256 bytes) skipped rows are reported by ``device_status``."""
    if stream is not None:
        with torch.cuda.stream(stream):
            return cache_write(cache, k, v, seq_offsets, cache_lens, page_table, rope, positions, ws)
    st = load_extension().cache_write(cache._addr, cache._device, k, v, seq_offsets, cache_lens, page_table,
                                      0 if rope is None else rope._addr, 0 if rope is None else rope._device,
                                      positions, ws)
    if st is not None:
        _check(st, "hstu_attn_cache_write")


def cache_read(cache: PagedCache, seq_offsets, rows: int, page_table, starts=None, outs=None,
               ws: Optional[torch.Tensor] = None, stream=None):
    """(k, v) of cached rows, jagged and contiguous, in the cache's dtype
    (hstu_attn_cache_read): ``rows`` rows, those of sequence b from position
    ``starts[b]`` (0 without ``starts``). Rows without a valid place are left
    as they were in ``outs`` and are zeros in new tensors."""
    if stream is not None:
        with torch.cuda.stream(stream):
            return cache_read(cache, seq_offsets, rows, page_table, starts, outs, ws)
    k, v = (None, None) if outs is None else outs
    r = load_extension().cache_read(cache._addr, cache._device, seq_offsets, rows, page_table, starts, k, v, ws)
    if type(r) is int:
        _check(r, "hstu_attn_cache_read")
    return r


def paged_workspace(cache: PagedCache, batch: int, num_candidates: int, max_seqlen: int) -> torch.Tensor:
    """Workspace of ``fwd_paged``."""
    n = load().hstu_attn_paged_workspace_size(cache._addr, batch, num_candidates, max_seqlen)
    if n == 0:
        raise HstuError(2, "hstu_attn_paged_workspace_size")
    return torch.empty(n, dtype=torch.uint8, device=cache.device)


def fwd_paged(q_c, cache: PagedCache, cache_lens, page_table, max_seqlen: int, alpha: Optional[float] = None,
              cand_offsets=None, func_c=None, ws: Optional[torch.Tensor] = None, out=None, stream=None):
    """o_c (C, H, D_v): candidate rows q_c (C, H, D_qk) against the
    ``cache_lens[b]`` cached rows of their sequences (hstu_attn_fwd_paged).
    One candidate a sequence without ``cand_offsets``; all cached rows are
    visible without ``func_c`` (nfunc, C). With a ``ws`` (``paged_workspace``)
    of its own a caller can read ``device_status``. Rows of bad sequences are
    left as they were in ``out`` and are zeros in a new tensor."""
    if stream is not None:
        with torch.cuda.stream(stream):
            return fwd_paged(q_c, cache, cache_lens, page_table, max_seqlen, alpha, cand_offsets, func_c, ws, out)
    r = load_extension().fwd_paged(cache._addr, cache._device, q_c, cache_lens, page_table, max_seqlen,
                                   1.0 / math.sqrt(cache.dim) if alpha is None else alpha, cand_offsets, func_c, ws,
                                   out)
    if type(r) is int:
        _check(r, "hstu_attn_fwd_paged")
    return r


# ------------------------------------------------------- the rest of a layer
# Embedding rows, norms and linear maps of (rows, width) matrices, through the same
# extension. Inputs may be slices of wider rows where the header gives them a
# stride.

_WIDE = {**DTYPES, torch.float32: 2}
_ACTS = {"none": 0, "silu": 1, "gelu": 2, "relu": 3}


def _dtype_code(dtype, codes, name: str) -> int:
    if dtype not in codes:
        raise ValueError(f"{name} must be one of {tuple(codes)}, got {dtype}")
    return codes[dtype]


def _act_code(act: str) -> int:
    if act not in _ACTS:
        raise ValueError(f"act must be one of {sorted(_ACTS)}")
    return _ACTS[act]


def embed(table, ids, scale: float = 1.0, dtype=None, out=None, ws: Optional[torch.Tensor] = None, stream=None):
    """(T, D): ``scale * table[ids]`` (hstu_attn_embed). The table is (V, D), of the
    rows' type or float32 (the rows are then of ``dtype``, bf16 if it is not
    given); ids are int32 or int64, below 0 for padding, whose rows are zeros; the
    scale is finite.
    With a ``ws`` (256 bytes) ids past the table are reported by
    ``device_status``; their rows are zeros too."""
    if stream is not None:
        with torch.cuda.stream(stream):
            return embed(table, ids, scale, dtype, out, ws)
    if dtype is None:
        dtype = torch.bfloat16 if table.dtype == torch.float32 else table.dtype
    r = load_extension().embed(table, ids, scale, _dtype_code(dtype, DTYPES, "dtype"), out, ws)
    if type(r) is int:
        _check(r, "hstu_attn_embed")
    return r


def embed_workspace(tokens: int, vocab: int, dim: int, device="cuda") -> torch.Tensor:
    """Workspace of ``embed_bwd``, for up to so many tokens."""
    n = int(load().hstu_attn_embed_workspace_size(tokens, vocab, dim))
    if n == 0:
        raise HstuError(2, "hstu_attn_embed_workspace_size")
    return torch.empty(n, dtype=torch.uint8, device=device)


def embed_bwd(dy, ids, vocab: int, scale: float = 1.0, dtype=torch.float32, out=None, accumulate: bool = False,
              ws: Optional[torch.Tensor] = None, stream=None):
    """The table's gradient (vocab, D) of sum(embed(table, ids, scale) * dy), of
    ``dtype``: float32 or dy's (hstu_attn_embed_bwd). ``accumulate`` adds it to a
    float32 ``out`` and leaves rows that no id names untouched."""
    if stream is not None:
        with torch.cuda.stream(stream):
            return embed_bwd(dy, ids, vocab, scale, dtype, out, accumulate, ws)
    r = load_extension().embed_bwd(dy, ids, vocab, scale, _dtype_code(dtype, _WIDE, "dtype"), out, bool(accumulate), ws)
    if type(r) is int:
        _check(r, "hstu_attn_embed_bwd")
    return r


class QuantisedRows:
    """Rows of 8-bit floats (e4m3): ``codes`` (rows, width) and the exponent
    bytes of their power-of-two scales, ``scale`` (rows,), both uint8. Made by
    ``quantise_rows`` or ``rms_norm(..., quantise=True)``, taken by ``linear``."""

    __slots__ = ("codes", "scale")

    def __init__(self, codes: torch.Tensor, scale: torch.Tensor):
        if codes.dtype != torch.uint8 or codes.dim() != 2:
            raise ValueError(f"codes must be (rows, width) of torch.uint8, got {tuple(codes.shape)} of {codes.dtype}")
        if scale.dtype != torch.uint8 or tuple(scale.shape) != (codes.shape[0],):
            raise ValueError(f"scale must be ({codes.shape[0]},) of torch.uint8, got {tuple(scale.shape)} of "
                             f"{scale.dtype}")
        self.codes, self.scale = codes, scale


def _quantised(codes, scale) -> QuantisedRows:
    """One of the extension's own outputs, which need no checks."""
    q = object.__new__(QuantisedRows)
    q.codes, q.scale = codes, scale
    return q


def quantise_rows(x, stream=None) -> QuantisedRows:
    """x (rows, width) as 8-bit floats under a power of two for each row
    (hstu_attn_quantise_rows); a weight of ``linear`` once, before it is used."""
    if stream is not None:
        with torch.cuda.stream(stream):
            return quantise_rows(x)
    r = load_extension().quantise_rows(x)
    if type(r) is int:
        _check(r, "hstu_attn_quantise_rows")
    return _quantised(*r)


def rms_norm(x, weight, residual=None, gate=None, eps: float = 1e-6, quantise: bool = False,
             want_rstd: Optional[bool] = None, outs=None, stream=None):
    """(y, h, rstd): h = x + residual (None without one), rstd = 1 / rms(h) and
    y = h * rstd * weight * gate (hstu_attn_rms_norm). y is QuantisedRows with
    ``quantise``; rstd, which the backward reads, is then None unless asked for.
    ``outs`` may be (y, h), either None; h may be the residual
    itself, which is then updated in place."""
    if stream is not None:
        with torch.cuda.stream(stream):
            return rms_norm(x, weight, residual, gate, eps, quantise, want_rstd, outs)
    y, h = (None, None) if outs is None else outs
    if type(y) is QuantisedRows:
        y, s = y.codes, y.scale
    else:
        s = None
    rstd = not quantise if want_rstd is None else bool(want_rstd)
    r = load_extension().rms_norm(x, weight, residual, gate, eps, bool(quantise), rstd, y, s, h)
    if type(r) is int:
        _check(r, "hstu_attn_rms_norm")
    y, s, h, rstd = r
    return (y if s is None else _quantised(y, s)), h, rstd


def rms_norm_workspace(rows: int, width: int, device="cuda") -> torch.Tensor:
    """Workspace of ``rms_norm_bwd``, for up to so many rows."""
    n = int(load().hstu_attn_rms_norm_workspace_size(rows, width))
    if n == 0:
        raise HstuError(2, "hstu_attn_rms_norm_workspace_size")
    return torch.empty(n, dtype=torch.uint8, device=device)


def rms_norm_bwd(dy, h, rstd, weight, gate=None, dh=None, ws: Optional[torch.Tensor] = None, stream=None):
    """(dx, dweight, dgate) of sum(y * dy) for rms_norm, h and rstd those of the
    forward (h is x where there was no residual; dx is the residual's gradient
    too). ``dh``, the gradient of h's other uses, is added to dx; dgate is None
    without a gate (hstu_attn_rms_norm_bwd)."""
    if stream is not None:
        with torch.cuda.stream(stream):
            return rms_norm_bwd(dy, h, rstd, weight, gate, dh, ws)
    r = load_extension().rms_norm_bwd(dy, h, rstd, weight, gate, dh, ws)
    if type(r) is int:
        _check(r, "hstu_attn_rms_norm_bwd")
    return r


def linear(x, w, bias=None, act: str = "none", residual=None, want_z: bool = False, dtype=None, out=None,
           ws: Optional[torch.Tensor] = None, stream=None):
    """(y, z): z = x w^T + bias, y = act(z) + residual (hstu_attn_linear). x (T,
    d_in) and w (d_out, d_in) are both bf16, both fp16, or both QuantisedRows (y
    is then of ``dtype``, bf16 if it is not given). ``act`` is "none", "silu",
    "gelu" (the tanh form) or "relu". z is None without ``want_z``; ``linear_bwd``
    needs it where there is an activation. With a ``ws`` (256 bytes) a wait that
    gave up is reported by ``device_status``."""
    if stream is not None:
        with torch.cuda.stream(stream):
            return linear(x, w, bias, act, residual, want_z, dtype, out, ws)
    xs = ws_ = None
    if type(x) is QuantisedRows:
        x, xs = x.codes, x.scale
    if type(w) is QuantisedRows:
        w, ws_ = w.codes, w.scale
    if dtype is None:
        dtype = x.dtype if xs is None else torch.bfloat16
    r = load_extension().linear(x, xs, w, ws_, bias, _act_code(act), residual, _dtype_code(dtype, DTYPES, "dtype"),
                                bool(want_z), out, ws)
    if type(r) is int:
        _check(r, "hstu_attn_linear")
    return r


def linear_workspace(rows: int, d_in: int, d_out: int, act: str = "none", device="cuda") -> torch.Tensor:
    """Workspace of ``linear_bwd``, for up to so many rows."""
    n = int(load().hstu_attn_linear_workspace_size(rows, d_in, d_out, _act_code(act)))
    if n == 0:
        raise HstuError(2, "hstu_attn_linear_workspace_size")
    return torch.empty(n, dtype=torch.uint8, device=device)


def linear_bwd(dy, z, x, w, act: str = "none", want_dbias: bool = True, ws: Optional[torch.Tensor] = None,
               stream=None):
    """(dx, dw, dbias) of sum(y * dy) for linear with 16-bit operands
    (hstu_attn_linear_bwd); z is not read with act "none", and the residual's
    gradient is dy."""
    if stream is not None:
        with torch.cuda.stream(stream):
            return linear_bwd(dy, z, x, w, act, want_dbias, ws)
    r = load_extension().linear_bwd(dy, z, x, w, _act_code(act), bool(want_dbias), ws)
    if type(r) is int:
        _check(r, "hstu_attn_linear_bwd")
    return r
