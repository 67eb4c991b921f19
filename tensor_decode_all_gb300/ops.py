"""Python binding of include/ar_ops.h: the operators around a decode step's all-reduce.

    plan = kv_plan(lens, new, table, free_pages, free_used, page=, max_tokens=)   # once a step
    kv4_append(k, v, pool, plan.slots)                                            # each layer
    out = kv4_attend(q, pool, table, plan.lens, plan.cu, max_new=)
    ... output projection, Handle.allreduce of the partial sums ...
    y, scales, residual = add_norm_fp8(x, weight, residual=residual)

Every step runs in libtda_ar.so, and there is no CPU path; the tensors are checked,
outputs allocated and arguments marshalled in the extension module beside it
(csrc/ops_binding.cpp), so that a call costs little more than its launch.  Wrong tensors raise ``ValueError`` before anything is
enqueued, codes of the library ``ArError``.  ``stream`` (a torch stream, a raw
handle, or None for the current stream) is where the call is enqueued; what it
returns without an ``out`` of the caller's is allocated for that stream.

For serving only: nothing here has a gradient.  Tensors that require one are taken as data, and
no result requires one, as under ``torch.no_grad()``.
"""
from __future__ import annotations

import ctypes
import threading
from typing import NamedTuple

from . import ar
from .ar import ArError

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


_native = None


def _binding():
    """The extension module that checks the tensors, allocates outputs and calls the library."""
    global _native
    if _native is None:
        _ops()                      # says so if the library is not built
        import torch  # noqa: F401  (its libraries come first)
        from . import _ops_binding
        _ops_binding.set_error(ArError)
        _native = _ops_binding
    return _native


def _on(stream, dev):
    """The torch stream of a torch stream or raw handle."""
    import torch
    if isinstance(stream, int):
        return torch.cuda.ExternalStream(stream, device=dev) if stream else torch.cuda.default_stream(dev)
    return stream


def _index(device) -> int:
    """The index of a CUDA device; "cuda" and None are the current one."""
    import torch
    device = torch.device("cuda" if device is None else device)
    if device.type != "cuda":
        raise ValueError(f"device: {device} is not a CUDA device")
    return torch.cuda.current_device() if device.index is None else device.index


def _under(stream, call, *args, **kwargs):
    """The call with `stream` as the current one."""
    import torch
    with torch.cuda.stream(_on(stream, torch.cuda.current_device())):
        return call(*args, **kwargs)


# --------------------------------------------------------------------- plan

class _KvPlanFields(NamedTuple):
    lens: object        # int32 [requests]: tokens with the new ones
    cu: object          # int32 [requests + 1]: where each request's new tokens begin
    request: object     # int32 [max_tokens]
    position: object    # int32 [max_tokens]
    free_used: object   # int32 [1]
    status: object      # int32 [1]: an AR_* code
    slots: object       # int64 [max_tokens]


class KvPlan(_KvPlanFields):
    """What kv_plan writes (see ar_kv_plan in ar_ops.h)."""

    _stream = None      # the handle of the stream that it is made on

    def _replace(self, **fields):
        plan = super()._replace(**fields)
        plan._stream = self._stream
        return plan

    def check(self):
        """Raise ArError if nothing was handed out.  Waits for the plan, on whatever stream it is made (which has
        to exist still); of a plan in a graph, for replays on the current stream."""
        import torch
        if self._stream is not None:
            here = torch.cuda.current_stream(self.status.device)
            if here.cuda_stream != self._stream:
                here.wait_stream(_on(self._stream, self.status.device))
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
    if stream is not None:
        return _under(stream, kv_plan, lens, new, table, free_pages, free_used, page=page, max_tokens=max_tokens, out=out)
    handle, made = (_native or _binding()).plan(lens, new, table, free_pages, free_used, page, max_tokens, out)
    plan = KvPlan._make(made) if out is None else out
    if isinstance(plan, KvPlan):
        plan._stream = handle
    return plan


# -------------------------------------------------------------------- cache

def kv4_pool(pages, kv_heads, head_dim, page, device="cuda"):
    """A zeroed 4-bit paged cache: uint8 [pages, kv_heads, page // 16, 18 * head_dim] (the layout is in ar_ops.h)."""
    import torch
    if head_dim not in (64, 128, 256) or page < 16 or page % 16:
        raise ValueError("kv4_pool: head_dim is 64, 128 or 256, page a multiple of 16")
    return torch.zeros(pages, kv_heads, page // 16, 18 * head_dim, dtype=torch.uint8, device=device)


def kv4_append(k, v, pool, slots, *, stream=None) -> None:
    """Round K and V rows [tokens, kv_heads, head_dim] (float16 or bfloat16, any strides with dense
    channels) to 4 bits and write them to int64 `slots` [tokens] of `pool`; a slot outside the pool is skipped."""
    if stream is not None:
        return _under(stream, kv4_append, k, v, pool, slots)
    (_native or _binding()).append(k, v, pool, slots)


def kv4_load(pool, slots, dtype=None, *, out=None, stream=None):
    """(k, v): the values held at int64 `slots` [tokens], rounded to `dtype` (bfloat16 by default), or
    into `out`, a pair of tensors [tokens, kv_heads, head_dim].  Slots outside the pool give zeros."""
    if stream is not None:
        return _under(stream, kv4_load, pool, slots, dtype, out=out)
    return (_native or _binding()).load(pool, slots, dtype, out if out is None else tuple(out))


# ---------------------------------------------------------------- attention

_workspaces = {}            # by device and stream, for calls that are not captured
_captured = {}              # by device: the ones of captured calls ...
_capture_streams = {}       # ... dealt out to the streams of a capture, by device and capture, in the order they come
_workspace_lock = threading.Lock()


class Kv4Workspace:
    """Working memory of kv4_attend on one device: one for calls that may overlap on the GPU.  Calls
    without one share a workspace of their stream's (see kv4_workspace), which lives as long as the process.

    Ready for any stream once made (which waits for the current one); whoever makes it keeps it until the
    calls that use it, and the graphs they were captured in, are done."""

    def __init__(self, device=None, stream=None):
        import torch
        if stream is not None:
            return _under(stream, self.__init__, device)
        dev = _index(device)
        if torch.cuda.is_current_stream_capturing():
            raise RuntimeError("a kv4_attend workspace cannot be made while a CUDA graph is captured: "
                               "make it (or call kv4_attend once on this stream) before")
        L = _lib or _ops()
        self.buffer = torch.empty(L.ar_kv4_workspace_bytes(), dtype=torch.uint8, device=torch.device("cuda", dev))
        self.device, self.ptr = dev, self.buffer.data_ptr()
        rc = L.ar_kv4_workspace_init(self.ptr, torch.cuda.current_stream(dev).cuda_stream)
        if rc:
            raise ArError(rc, "ar_kv4_workspace_init")
        torch.cuda.current_stream(dev).synchronize()

    def status(self) -> int:
        """The first error recorded since it was made (AR_OK if none); synchronise with the calls first."""
        return (_lib or _ops()).ar_kv4_status(self.ptr)

    def check(self) -> None:
        code = self.status()
        if code:
            raise ArError(code, "kv4_attend (recorded on the device)")


def kv4_workspace(device=None, stream=None) -> Kv4Workspace:
    """The workspace that kv4_attend uses on this stream when it is given none.

    While the stream is captured that is another one, kept for captured calls: the replays of a graph may
    overlap with calls on the stream it was captured on.  The streams of one capture use one each, of those that
    are made beside the first workspaces of the device's streams (as many, and two at least); a capture of
    more streams than there are is refused.  Different captures use the same: graphs that may run at the
    same time need workspaces of their own (``workspace=``)."""
    import torch
    if stream is not None:
        return _under(stream, kv4_workspace, device)
    dev = _index(device)
    key = dev, torch.cuda.current_stream(dev).cuda_stream
    capture = _binding().capture_id(key[1])
    with _workspace_lock:
        captured = _captured.setdefault(dev, [])
        if capture:
            streams = _capture_streams.setdefault((dev, capture), [])
            if key[1] not in streams:
                if len(streams) >= len(captured):
                    raise RuntimeError(f"kv4_attend is captured on more streams than there are workspaces for it ({len(captured)}): "
                                       "call kv4_workspace() on as many streams before, or give each its own (workspace=)")
                streams.append(key[1])
            return captured[streams.index(key[1])]
        ws = _workspaces.get(key)
        if ws is None:
            while len(captured) < max(2, 1 + sum(d == dev for d, _ in _workspaces)):
                captured.append(Kv4Workspace(dev))
            ws = _workspaces[key] = Kv4Workspace(dev)
            _binding().set_workspace(dev, key[1], ws.ptr)
    return ws


def kv4_workspaces(device=None) -> list:
    """All workspaces kept for kv4_attend on a device, its streams' and those of captured calls, for their
    ``check()`` after a step (synchronise with its calls and replays first)."""
    import torch
    dev = _index(device)
    with _workspace_lock:
        return [ws for (d, _), ws in _workspaces.items() if d == dev] + _captured.get(dev, [])


def kv4_attend(q, pool, table, lens, cu=None, *, max_new=None, window=0, sinks=0, scale=None, out=None, lse=None,
               return_lse=False, workspace=None, stream=None):
    """Attention of the requests' newest tokens over their 4-bit cache (see ar_kv4_attend in ar_ops.h).

    q [tokens, q_heads, head_dim], float16 or bfloat16; `table` int32 [requests, width] of page ids;
    `lens` int32 [requests], the new tokens included.  Without `cu`, one token a request; with `cu` (int32
    [requests + 1]) request b's tokens are rows cu[b] .. cu[b + 1] - 1, and `max_new`, the most of
    any request (default: all of them), picks the kernel's shape.  `window` > 0 limits a token to
    the last `window` ones, itself included, and the first `sinks`.  `scale` defaults to head_dim ** -0.5.
    Rows of no request (past cu[requests], as in a padded step) are not written: in an `out` that the call
    makes they hold whatever the memory held.
    Returns `out`, or (out, lse) with `return_lse` or an `lse` (float32 [tokens, q_heads]) of the caller's.
    """
    if stream is not None:
        return _under(stream, kv4_attend, q, pool, table, lens, cu, max_new=max_new, window=window, sinks=sinks, scale=scale,
                      out=out, lse=lse, return_lse=return_lse, workspace=workspace)
    attend = (_native or _binding()).attend
    if workspace is not None:
        if workspace.device != pool.get_device():
            raise ValueError(f"workspace: on cuda:{workspace.device}, not {pool.device}")
        workspace = workspace.ptr
    made = attend(q, pool, table, lens, cu, max_new, window, sinks, scale, out, lse, return_lse, workspace)
    if made is None:        # this stream's first call, or a captured one
        made = attend(q, pool, table, lens, cu, max_new, window, sinks, scale, out, lse, return_lse, kv4_workspace().ptr)
    if out is None and lse is None:
        return made
    out = made[0] if isinstance(made, tuple) and out is None else made if out is None else out
    return out if lse is None and not return_lse else (out, made[1] if lse is None else lse)


# --------------------------------------------------------------------- norm

def add_norm_fp8(x, weight, *, residual=None, eps=1e-6, group=0, out=None, scales=None, residual_out=None, stream=None):
    """(out, scales, h): h = x + residual, out = e4m3(norm(h) * weight / scale), one scale to `group`
    channels (0: one a row).  x and residual [rows, dim], rows of any stride; `residual_out` may be
    residual or x themselves.  Without a residual h is x, and is written only if `residual_out` is given (else None)."""
    if stream is not None:
        return _under(stream, add_norm_fp8, x, weight, residual=residual, eps=eps, group=group, out=out, scales=scales,
                      residual_out=residual_out)
    made = (_native or _binding()).norm(x, weight, residual, eps, group, out, scales, residual_out)
    if out is None and scales is None and residual_out is None:
        return made
    return (out if out is not None else made[0], scales if scales is not None else made[1],
            residual_out if residual_out is not None else made[2])
