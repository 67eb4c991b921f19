"""Python binding of include/ar_ffn.h: the operators of a decode step's feed-forward half.

    x8, xs, residual = add_norm_fp8(total, weight, residual=residual, group=128)     # (ops.py)
    h = matmul_fp8(x8, xs, gate_up, gate_up_scales)                # a dense layer
    y8, ys = silu_mul_fp8(h)
    partial = matmul_fp8(y8, ys, down, down_scales)

    r = route_experts(logits, k)                                   # a layer with experts
    h = experts_matmul_fp8(x8, xs, gate_up, gate_up_scales, r.offsets, rows=r.rows)
    y8, ys = silu_mul_fp8(h)
    y = experts_matmul_fp8(y8, ys, down, down_scales, r.offsets)
    partial = experts_sum(y, r.weights, r.place)
    ... Handle.allreduce of the partial sums ...

In the manner of ops.py: every step runs in libtda_ar.so, there is no CPU path, wrong tensors raise ``ValueError`` before
anything is enqueued, codes of the library ``ArError``; ``stream`` (a torch stream, a raw handle, or None for the current
stream) is where the call is enqueued.  For serving only: nothing here has a gradient.
"""
from __future__ import annotations

import ctypes
from typing import NamedTuple

from . import ar, ops
from .ops import _under

_P, _I64, _I32 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32


class MatmulFp8Args(ctypes.Structure):
    _fields_ = [("x", _P), ("x_scales", _P), ("weight", _P), ("weight_scales", _P), ("out", _P), ("offsets", _P), ("row_of", _P),
                ("workspace", _P),
                ("x_stride", _I64), ("x_scales_stride", _I64), ("weight_stride", _I64), ("expert_stride", _I64), ("out_stride", _I64),
                ("rows", _I64), ("x_rows", _I64),
                ("dtype", _I32), ("out_dim", _I32), ("dim", _I32), ("experts", _I32), ("x_row_scales", _I32)]


class RouteExpertsArgs(ctypes.Structure):
    _fields_ = [("logits", _P), ("weights", _P), ("expert_ids", _P), ("offsets", _P), ("rows", _P), ("place", _P),
                ("workspace", _P), ("logits_stride", _I64), ("tokens", _I64),
                ("dtype", _I32), ("experts", _I32), ("chosen", _I32), ("normalize", _I32)]


class SiluMulFp8Args(ctypes.Structure):
    _fields_ = [("x", _P), ("out", _P), ("scales", _P), ("x_stride", _I64), ("rows", _I64),
                ("dtype", _I32), ("dim", _I32), ("group", _I32)]


class ExpertsSumArgs(ctypes.Structure):
    _fields_ = [("x", _P), ("weights", _P), ("place", _P), ("out", _P),
                ("x_stride", _I64), ("out_stride", _I64), ("rows", _I64), ("tokens", _I64),
                ("dtype", _I32), ("dim", _I32), ("chosen", _I32)]


STRUCTS = {"ar_matmul_fp8_args": MatmulFp8Args, "ar_route_experts_args": RouteExpertsArgs, "ar_silu_mul_fp8_args": SiluMulFp8Args,
           "ar_experts_sum_args": ExpertsSumArgs}

_lib = None


def _ffn():
    """The loaded library, with this header's entry points typed."""
    global _lib
    if _lib is None:
        L = ar.lib()
        for name in ("ar_matmul_fp8", "ar_route_experts", "ar_silu_mul_fp8", "ar_experts_sum"):
            f = getattr(L, name)
            f.argtypes = [_P, _P]
            f.restype = ctypes.c_int
        L.ar_matmul_fp8_status.argtypes = []
        L.ar_matmul_fp8_workspace.argtypes = [_P]
        L.ar_matmul_fp8_workspace.restype = ctypes.c_size_t
        L.ar_route_experts_workspace.argtypes = [_P]
        L.ar_route_experts_workspace.restype = ctypes.c_size_t
        _lib = L
    return _lib


# ----------------------------------------------------------------- products

def matmul_fp8(x, x_scales, weight, weight_scales, *, rows=None, out=None, dtype=None, stream=None):
    """x times weight^T, both e4m3 with scales (see ar_matmul_fp8 in ar_ffn.h).

    x [rows, dim] (rows of any stride) and `x_scales` float32 [rows, ceil(dim / 128)] or [rows, 1], as add_norm_fp8 gives
    them with group 128 or 0; `weight` [out_dim, dim] and `weight_scales` float32 [ceil(out_dim / 128), ceil(dim / 128)], one
    to a block of 128 x 128.  With `rows` (int32 [n]) row i of the result belongs to x[rows[i]], as for the logits of the
    requests' last tokens.  Returns [rows, out_dim] of `dtype` (float16 or bfloat16, the default), or `out`.
    """
    if stream is not None:
        return _under(stream, matmul_fp8, x, x_scales, weight, weight_scales, rows=rows, out=out, dtype=dtype)
    return (ops._native or ops._binding()).matmul(x, x_scales, weight, weight_scales, None, rows, out, dtype)


def experts_matmul_fp8(x, x_scales, weight, weight_scales, offsets, *, rows=None, out=None, dtype=None, stream=None):
    """The same for rows grouped by expert: rows offsets[e] .. offsets[e + 1] - 1 of the result take weight[e].

    `weight` [experts, out_dim, dim], `weight_scales` [experts, ceil(out_dim / 128), ceil(dim / 128)], `offsets` int32
    [experts + 1], on the GPU.  With `rows` (int32 [n]) row i of the result belongs to x[rows[i]], else to x[i].  Rows of no
    expert (from offsets[experts] on) are not written: in an `out` that the call makes they hold whatever the
    memory held.
    """
    if stream is not None:
        return _under(stream, experts_matmul_fp8, x, x_scales, weight, weight_scales, offsets, rows=rows, out=out, dtype=dtype)
    return (ops._native or ops._binding()).matmul(x, x_scales, weight, weight_scales, offsets, rows, out, dtype)


def matmul_fp8_check(device=None) -> None:
    """Raise ArError if a product on the device has recorded an error since the last check (synchronise with the calls
    and replays first)."""
    import torch
    with torch.cuda.device(ops._index(device)):
        code = _ffn().ar_matmul_fp8_status()
    if code:
        raise ar.ArError(code, "matmul_fp8 (recorded on the device)")


# ------------------------------------------------------------------- router

class Routes(NamedTuple):
    """What route_experts writes (see ar_route_experts in ar_ffn.h)."""
    weights: object     # float32 [tokens, k]
    experts: object     # int32 [tokens, k]: -1 where there was none to choose
    offsets: object     # int32 [experts + 1]: where each expert's rows begin
    rows: object        # int32 [tokens * k]: the token of each row, -1 past the last
    place: object       # int32 [tokens, k]: the row of each pair, or -1


def route_experts(logits, k, *, normalize=True, out=None, stream=None) -> Routes:
    """The k experts of each token with the largest `logits` [tokens, experts] (float32, float16 or bfloat16), their
    softmax weights (over the chosen ones, or with ``normalize=False`` over all), and the rows by expert.
    `out`: Routes of an earlier call to write into."""
    if stream is not None:
        return _under(stream, route_experts, logits, k, normalize=normalize, out=out)
    made = (ops._native or ops._binding()).route(logits, k, normalize, out)
    return Routes._make(made) if out is None else out


# --------------------------------------------------- activation and weighted sum

def silu_mul_fp8(x, *, group=128, out=None, scales=None, stream=None):
    """(out, scales): silu(x[:, :dim]) * x[:, dim:] rounded to e4m3, one scale to `group` channels (0: one a row).  x
    [rows, 2 * dim], float16 or bfloat16, rows of any stride."""
    if stream is not None:
        return _under(stream, silu_mul_fp8, x, group=group, out=out, scales=scales)
    return (ops._native or ops._binding()).silu(x, group, out, scales)


def experts_sum(x, weights, place, *, out=None, stream=None):
    """out[t] = sum over j of weights[t, j] * x[place[t, j]]: x [rows, dim] float16 or bfloat16, `weights` float32 and
    `place` int32 [tokens, k]; places outside x count as nothing.  Returns [tokens, dim] of x's dtype, or `out`."""
    if stream is not None:
        return _under(stream, experts_sum, x, weights, place, out=out)
    return (ops._native or ops._binding()).weighted(x, weights, place, out)
