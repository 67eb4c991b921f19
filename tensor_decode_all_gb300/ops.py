"""Python binding of include/ar_ops.h: the operators around a decode step's all-reduce.

    plan = kv_plan(lens, new, table, free_pages, free_used, page=, max_tokens=)   # once a step
    kv4_append(k, v, pool, plan.slots)                                            # each layer
    out = kv4_attend(q, pool, table, plan.lens, plan.cu, max_new=)
    ... output projection, Handle.allreduce of the partial sums ...
    y, scales, residual = add_norm_fp8(x, weight, residual=residual)

Tensor checks and marshalling only: every step runs in libtda_ar.so, and there
is no CPU path.  Wrong tensors raise ``ValueError`` before anything is
enqueued, codes of the library ``ArError``.  ``stream`` (a torch stream, a raw
handle, or None for the current stream) is where the call is enqueued; what it
returns without an ``out`` of the caller's is allocated for that stream.
"""
from __future__ import annotations

import ctypes
import threading
from typing import NamedTuple

from . import ar
from .ar import AR_BF16, AR_F16, ArError

_P, _I64, _I32 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32


class KvPlanArgs(ctypes.Structure):
    _fields_ = [("lens", _P), ("new_tokens", _P), ("table", _P), ("free_pages", _P), ("free_used", _P),
                ("lens_out", _P), ("cu", _P), ("slots", _P), ("request", _P), ("position", _P),
                ("free_used_out", _P), ("status", _P), ("table_stride", _I64), ("free_count", _I64),
                ("requests", _I32), ("table_width", _I32), ("page", _I32), ("max_tokens", _I32)]


class Kv4RowsArgs(ctypes.Structure):
    _fields_ = [("k", _P), ("v", _P), ("pool", _P), ("slots", _P),
                ("k_token_stride", _I64), ("k_head_stride", _I64), ("v_token_stride", _I64), ("v_head_stride", _I64),
                ("pages", _I64), ("tokens", _I64),
                ("dtype", _I32), ("kv_heads", _I32), ("head_dim", _I32), ("page", _I32)]


class Kv4AttendArgs(ctypes.Structure):
    _fields_ = [("q", _P), ("out", _P), ("lse", _P), ("pool", _P), ("table", _P), ("lens", _P), ("cu", _P),
                ("workspace", _P),
                ("q_token_stride", _I64), ("q_head_stride", _I64), ("out_token_stride", _I64), ("out_head_stride", _I64),
                ("table_stride", _I64), ("pages", _I64),
                ("dtype", _I32), ("tokens", _I32), ("requests", _I32), ("max_new", _I32), ("q_heads", _I32),
                ("kv_heads", _I32), ("head_dim", _I32), ("page", _I32), ("table_width", _I32), ("window", _I32),
                ("sinks", _I32), ("scale", ctypes.c_float)]


class AddNormFp8Args(ctypes.Structure):
    _fields_ = [("x", _P), ("residual", _P), ("weight", _P), ("out", _P), ("scales", _P), ("residual_out", _P),
                ("x_stride", _I64), ("residual_stride", _I64), ("residual_out_stride", _I64), ("rows", _I64),
                ("dtype", _I32), ("dim", _I32), ("group", _I32), ("eps", ctypes.c_float)]


STRUCTS = {"ar_kv_plan_args": KvPlanArgs, "ar_kv4_rows_args": Kv4RowsArgs, "ar_kv4_attend_args": Kv4AttendArgs,
           "ar_add_norm_fp8_args": AddNormFp8Args}

_lib = None


def _ops():
    """The loaded library, with this header's entry points typed."""
    global _lib
    if _lib is None:
        L = ar.lib()
        for name in ("ar_kv_plan", "ar_kv4_append", "ar_kv4_load", "ar_kv4_attend", "ar_add_norm_fp8"):
            f = getattr(L, name)
            f.argtypes = [_P, _P]
            f.restype = ctypes.c_int
        L.ar_kv4_workspace_bytes.argtypes = []
        L.ar_kv4_workspace_bytes.restype = ctypes.c_size_t
        L.ar_kv4_workspace_init.argtypes = [_P, _P]
        L.ar_kv4_status.argtypes = [_P]
        _lib = L
    return _lib


def _call(name, args, stream):
    rc = getattr(_lib or _ops(), name)(ctypes.addressof(args), stream)
    if rc:
        raise ArError(rc, name)


# ------------------------------------------------------------ what is checked

_codes = None
_torch = None


def _T():
    global _codes, _torch
    if _torch is None:
        import torch
        _codes = {torch.float16: AR_F16, torch.bfloat16: AR_BF16}
        _torch = torch
    return _torch


def _dtype16(what, t):
    code = _codes.get(t.dtype)
    if code is None:
        raise ValueError(f"{what}: dtype {t.dtype} is neither float16 nor bfloat16")
    return code


def _check(what, t, dtype=None, ndim=None, device=None, dense=False, shape=None):
    """One tensor on the current device, of this type, rank and shape."""
    if not t.is_cuda:
        raise ValueError(f"{what}: not a CUDA tensor")
    if device is not None and t.device != device:
        raise ValueError(f"{what}: on {t.device}, not {device}")
    if dtype is not None and t.dtype is not dtype:
        raise ValueError(f"{what}: dtype {t.dtype}, not {dtype}")
    if ndim is not None and t.dim() != ndim:
        raise ValueError(f"{what}: {t.dim()} dimensions, not {ndim}")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{what}: shape {tuple(t.shape)}, not {tuple(shape)}")
    if dense and not t.is_contiguous():
        raise ValueError(f"{what}: not contiguous")


def _last_dense(what, t):
    if t.shape[-1] > 1 and t.stride(-1) != 1:
        raise ValueError(f"{what}: its last dimension is not contiguous")


def _device(what, t):
    torch = _torch or _T()
    if not t.is_cuda:
        raise ValueError(f"{what}: not a CUDA tensor")
    dev = t.device
    if dev.index != torch.cuda.current_device():
        raise ValueError(f"{what}: on {dev}, which is not the current device")
    return dev


class _Ambient:
    """Stands in for `with torch.cuda.stream(...)` where the current stream is meant."""

    def __enter__(self):
        return self

    def __exit__(self, *exc):
        return False


_ambient = _Ambient()


def _stream(stream, device):
    """(raw handle, context in which what the call returns is allocated)."""
    torch = _torch
    if stream is None:
        return torch.cuda.current_stream(device).cuda_stream, _ambient
    if isinstance(stream, int):
        stream = torch.cuda.ExternalStream(stream, device=device) if stream else torch.cuda.default_stream(device)
    return stream.cuda_stream, torch.cuda.stream(stream)


# --------------------------------------------------------------------- plan

class KvPlan(NamedTuple):
    """What kv_plan writes (see ar_kv_plan in ar_ops.h)."""
    lens: object        # int32 [requests]: tokens with the new ones
    cu: object          # int32 [requests + 1]: where each request's new tokens begin
    slots: object       # int64 [max_tokens]
    request: object     # int32 [max_tokens]
    position: object    # int32 [max_tokens]
    free_used: object   # int32 [1]
    status: object      # int32 [1]: an AR_* code

    def check(self):
        """Raise ArError if nothing was handed out (waits for the plan)."""
        code = int(self.status.item())
        if code:
            raise ArError(code, "kv_plan")


def kv_plan(lens, new, table, free_pages, free_used, *, page, max_tokens, out=None, stream=None) -> KvPlan:
    """Block tables and slot maps of a step from int32 `lens` and `new` [requests].

    New pages come from `free_pages` (int32 ids) from entry `free_used[0]` on and
    are written into `table` (int32 [requests, width], updated in place).
    `max_tokens` bounds the step's new tokens.  `out`: a KvPlan of an earlier
    step to write into (its `lens` and `free_used` may be this call's inputs, so
    that a captured step can be replayed).  Whether the pages sufficed is in
    `.status`, on the device; `.check()` raises.
    """
    torch = _torch or _T()
    dev = _device("lens", lens)
    i32, B, cap = torch.int32, lens.shape[0] if lens.dim() == 1 else -1, int(max_tokens)
    _check("lens", lens, i32, 1, dev, True)
    _check("new", new, i32, 1, dev, True, (B,))
    _check("table", table, i32, 2, dev)
    if table.shape[0] != B:
        raise ValueError(f"table: {table.shape[0]} rows for {B} requests")
    _last_dense("table", table)
    _check("free_pages", free_pages, i32, 1, dev, True)
    _check("free_used", free_used, i32, 1, dev, True, (1,))
    if cap < 0:
        raise ValueError("max_tokens is negative")
    raw, where = _stream(stream, dev)
    if out is None:
        with where:
            # one allocation: slots (8 bytes each) first
            room = torch.empty(4 * cap + 2 * B + 3, dtype=i32, device=dev)
            slots, rest = room[:2 * cap].view(torch.int64), room[2 * cap:]
            out = KvPlan(rest[2 * cap:2 * cap + B], rest[2 * cap + B:2 * cap + 2 * B + 1], slots, rest[:cap],
                         rest[cap:2 * cap], rest[-2:-1], rest[-1:])
    else:
        for what, t, dt, n in (("out.lens", out.lens, i32, B), ("out.cu", out.cu, i32, B + 1),
                               ("out.slots", out.slots, torch.int64, cap), ("out.request", out.request, i32, cap),
                               ("out.position", out.position, i32, cap), ("out.free_used", out.free_used, i32, 1),
                               ("out.status", out.status, i32, 1)):
            _check(what, t, dt, 1, dev, True, (n,))
    _call("ar_kv_plan", KvPlanArgs(
        lens.data_ptr(), new.data_ptr(), table.data_ptr(), free_pages.data_ptr(), free_used.data_ptr(),
        out.lens.data_ptr(), out.cu.data_ptr(), out.slots.data_ptr(), out.request.data_ptr(), out.position.data_ptr(),
        out.free_used.data_ptr(), out.status.data_ptr(), table.stride(0) if B > 1 else table.shape[1],
        free_pages.shape[0], B, table.shape[1], int(page), cap), raw)
    return out


# -------------------------------------------------------------------- cache

def kv4_pool(pages, kv_heads, head_dim, page, device="cuda"):
    """A zeroed 4-bit paged cache: uint8 [pages, kv_heads, page // 16, 18 * head_dim] (the layout is in ar_ops.h)."""
    torch = _torch or _T()
    if head_dim not in (64, 128, 256) or page < 16 or page % 16:
        raise ValueError("kv4_pool: head_dim is 64, 128 or 256, page a multiple of 16")
    return torch.zeros(pages, kv_heads, page // 16, 18 * head_dim, dtype=torch.uint8, device=device)


def _pool(pool, dev):
    """(pages, kv heads, head_dim, page) of a pool."""
    _check("pool", pool, _torch.uint8, 4, dev, True)
    pages, heads, tiles, bytes_ = pool.shape
    if bytes_ not in (1152, 2304, 4608) or tiles < 1 or heads < 1:
        raise ValueError(f"pool: shape {tuple(pool.shape)} is not [pages, kv heads, page / 16, 18 * head_dim]")
    return pages, heads, bytes_ // 18, tiles * 16


def _rows(name, k, v, pool, slots, dims, raw):
    pages, heads, D, page = dims
    for what, t in (("k", k), ("v", v)):
        _check(what, t, k.dtype, 3, pool.device, False, (slots.shape[0], heads, D))
        _last_dense(what, t)
    _call(name, Kv4RowsArgs(
        k.data_ptr(), v.data_ptr(), pool.data_ptr(), slots.data_ptr(), k.stride(0), k.stride(1), v.stride(0),
        v.stride(1), pages, slots.shape[0], _dtype16("k", k), heads, D, page), raw)


def kv4_append(k, v, pool, slots, *, stream=None) -> None:
    """Round K and V rows [tokens, kv_heads, head_dim] (float16 or bfloat16, any strides with dense
    channels) to 4 bits and write them to int64 `slots` [tokens] of `pool`; a negative slot is skipped."""
    torch = _torch or _T()
    dev = _device("pool", pool)
    dims = _pool(pool, dev)
    _check("slots", slots, torch.int64, 1, dev, True)
    _rows("ar_kv4_append", k, v, pool, slots, dims, _stream(stream, dev)[0])


def kv4_load(pool, slots, dtype=None, *, out=None, stream=None):
    """(k, v): the values held at int64 `slots` [tokens], rounded to `dtype` (bfloat16 by default), or
    into `out`, a pair of tensors [tokens, kv_heads, head_dim].  Slots outside the pool give zeros."""
    torch = _torch or _T()
    dev = _device("pool", pool)
    dims = _pool(pool, dev)
    _check("slots", slots, torch.int64, 1, dev, True)
    raw, where = _stream(stream, dev)
    if out is None:
        with where:
            room = torch.empty(2, slots.shape[0], dims[1], dims[2], dtype=dtype or torch.bfloat16, device=dev)
        out = (room[0], room[1])
    elif dtype is not None and out[0].dtype is not dtype:
        raise ValueError(f"out: dtype {out[0].dtype}, not {dtype}")
    _rows("ar_kv4_load", out[0], out[1], pool, slots, dims, raw)
    return out


# ---------------------------------------------------------------- attention

def _capturing(stream, dev):
    with _stream(stream, dev)[1]:
        return _torch.cuda.is_current_stream_capturing()


_workspaces = {}
_workspace_lock = threading.Lock()


class Kv4Workspace:
    """Working memory of kv4_attend on one device: one for calls that may overlap on the GPU.  Calls
    without one share a workspace of their stream's (see kv4_workspace), which lives as long as the process."""

    def __init__(self, device=None, stream=None):
        torch = _torch or _T()
        dev = torch.device("cuda", torch.cuda.current_device()) if device is None else torch.device(device)
        if _capturing(stream, dev):
            raise RuntimeError("a kv4_attend workspace cannot be made while a CUDA graph is captured: "
                               "make it (or call kv4_attend once on this stream) before")
        raw, where = _stream(stream, dev)
        L = _lib or _ops()
        with where:
            self.buffer = torch.empty(L.ar_kv4_workspace_bytes(), dtype=torch.uint8, device=dev)
        self.device, self.ptr = self.buffer.device, self.buffer.data_ptr()
        rc = L.ar_kv4_workspace_init(self.ptr, raw)
        if rc:
            raise ArError(rc, "ar_kv4_workspace_init")

    def status(self) -> int:
        """The first error recorded since it was made (AR_OK if none); synchronise with the calls first."""
        return (_lib or _ops()).ar_kv4_status(self.ptr)

    def check(self) -> None:
        code = self.status()
        if code:
            raise ArError(code, "kv4_attend (recorded on the device)")


def kv4_workspace(device=None, stream=None) -> Kv4Workspace:
    """The workspace that kv4_attend uses on this stream when it is given none.

    Calls that are being captured share one of their device's, made with the first workspace on it:
    graphs that may run at the same time need one each (``workspace=``)."""
    torch = _torch or _T()
    dev = torch.device("cuda", torch.cuda.current_device()) if device is None else torch.device(device)
    raw = _stream(stream, dev)[0]
    ws = _workspaces.get((dev.index, raw))
    if ws is None:
        with _workspace_lock:
            ws = _workspaces.get((dev.index, raw))
            if ws is None:
                if _capturing(stream, dev):
                    ws = _workspaces.get((dev.index, "capture"))
                    return ws if ws is not None else Kv4Workspace(dev, stream)    # which says why it cannot
                if (dev.index, "capture") not in _workspaces:
                    _workspaces[dev.index, "capture"] = Kv4Workspace(dev, stream)
                    (torch.cuda.ExternalStream(raw, device=dev) if raw else torch.cuda.default_stream(dev)).synchronize()
                ws = _workspaces[dev.index, raw] = Kv4Workspace(dev, stream)
    return ws


def kv4_attend(q, pool, table, lens, cu=None, *, max_new=None, window=0, sinks=0, scale=None, out=None, lse=None,
               return_lse=False, workspace=None, stream=None):
    """Attention of the requests' newest tokens over their 4-bit cache (see ar_kv4_attend in ar_ops.h).

    q [tokens, q_heads, head_dim], float16 or bfloat16; `table` int32 [requests, width] of page ids;
    `lens` int32 [requests], the new tokens included.  Without `cu`, one token a request; with `cu` (int32
    [requests + 1]) request b's tokens are rows cu[b] .. cu[b + 1] - 1, and `max_new`, the most of
    any request (default: all of them), picks the kernel's shape.  `window` > 0 limits a token to
    the last `window` ones, itself included, and the first `sinks`.  `scale` defaults to head_dim ** -0.5.
    Returns `out`, or (out, lse) with `return_lse` or an `lse` (float32 [tokens, q_heads]) of the caller's.
    """
    torch = _torch or _T()
    dev = _device("pool", pool)
    pages, kv_heads, D, page = _pool(pool, dev)
    i32 = torch.int32
    _check("q", q, None, 3, dev)
    T, heads, d = q.shape
    if d != D:
        raise ValueError(f"q: head_dim {d}, the pool's is {D}")
    if heads < 1 or heads % kv_heads:
        raise ValueError(f"q: {heads} heads for {kv_heads} kv heads")
    _last_dense("q", q)
    code = _dtype16("q", q)
    _check("lens", lens, i32, 1, dev, True)
    B = lens.shape[0]
    _check("table", table, i32, 2, dev)
    if table.shape[0] != B:
        raise ValueError(f"table: {table.shape[0]} rows for {B} requests")
    _last_dense("table", table)
    if cu is not None:
        _check("cu", cu, i32, 1, dev, True, (B + 1,))
    elif T != B:
        raise ValueError(f"q: {T} tokens for {B} requests, and no cu")
    raw, where = _stream(stream, dev)
    if workspace is None:
        workspace = _workspaces.get((dev.index, raw)) or kv4_workspace(dev, stream)
    elif workspace.device != dev:
        raise ValueError(f"workspace: on {workspace.device}, not {dev}")
    if out is None or (lse is None and return_lse):
        with where:
            if out is None:
                out = torch.empty((T, heads, D), dtype=q.dtype, device=dev)
            if lse is None and return_lse:
                lse = torch.empty((T, heads), dtype=torch.float32, device=dev)
    _check("out", out, q.dtype, 3, dev, False, (T, heads, D))
    _last_dense("out", out)
    if lse is not None:
        _check("lse", lse, torch.float32, 2, dev, True, (T, heads))
    _call("ar_kv4_attend", Kv4AttendArgs(
        q.data_ptr(), out.data_ptr(), None if lse is None else lse.data_ptr(), pool.data_ptr(), table.data_ptr(),
        lens.data_ptr(), None if cu is None else cu.data_ptr(), workspace.ptr, q.stride(0), q.stride(1), out.stride(0),
        out.stride(1), table.stride(0) if B > 1 else table.shape[1], pages, code, T, B,
        (T if cu is not None else 1) if max_new is None else int(max_new), heads, kv_heads, D, page, table.shape[1],
        int(window), int(sinks), D ** -0.5 if scale is None else float(scale)), raw)
    return out if lse is None else (out, lse)


# --------------------------------------------------------------------- norm

def add_norm_fp8(x, weight, *, residual=None, eps=1e-6, group=0, out=None, scales=None, residual_out=None, stream=None):
    """(out, scales, h): h = x + residual, out = e4m3(norm(h) * weight / scale), one scale to `group`
    channels (0: one a row).  x and residual [rows, dim], rows of any stride; `residual_out` may be
    residual or x themselves.  Without a residual h is x, and is written only if `residual_out` is given (else None)."""
    torch = _torch or _T()
    dev = _device("x", x)
    _check("x", x, None, 2, dev)
    N, d = x.shape
    code = _dtype16("x", x)
    _last_dense("x", x)
    _check("weight", weight, x.dtype, 1, dev, True, (d,))
    group = int(group)
    if group < 0 or group > d:
        raise ValueError(f"group: {group} is not within 0 .. {d}")
    groups = -(-d // group) if group else 1
    raw, where = _stream(stream, dev)
    with where:
        if out is None:
            out = torch.empty((N, d), dtype=torch.float8_e4m3fn, device=dev)
        if scales is None:
            scales = torch.empty((N, groups), dtype=torch.float32, device=dev)
        if residual_out is None and residual is not None:
            residual_out = torch.empty((N, d), dtype=x.dtype, device=dev)
    if residual is not None:
        _check("residual", residual, x.dtype, 2, dev, False, (N, d))
        _last_dense("residual", residual)
    if residual_out is not None:
        _check("residual_out", residual_out, x.dtype, 2, dev, False, (N, d))
        _last_dense("residual_out", residual_out)
    _check("out", out, torch.float8_e4m3fn, 2, dev, True, (N, d))
    _check("scales", scales, torch.float32, 2, dev, True, (N, groups))
    _call("ar_add_norm_fp8", AddNormFp8Args(
        x.data_ptr(), None if residual is None else residual.data_ptr(), weight.data_ptr(), out.data_ptr(),
        scales.data_ptr(), None if residual_out is None else residual_out.data_ptr(), x.stride(0),
        0 if residual is None else residual.stride(0), 0 if residual_out is None else residual_out.stride(0), N,
        code, d, group, float(eps)), raw)
    return out, scales, residual_out
