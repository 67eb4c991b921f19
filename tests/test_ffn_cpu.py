"""The operators of include/ar_ffn.h without a GPU: the header, the binding's structs, the refusals that come before any
CUDA call, and the plain implementations that the GPU tests compare with."""
import ctypes
import os
import shutil
import subprocess

import pytest
import torch

import tensor_decode_all_gb300 as tda
from tensor_decode_all_gb300 import ar, ffn
from tests import ffn_helpers as H


@pytest.fixture(scope="module")
def lib():
    tda.build()
    return ffn._ffn()


def test_symbols_are_declared_and_exported(lib):
    names = tda.declared_symbols(os.path.join(ar._build.INCLUDE, "ar_ffn.h"))
    assert set(names) == {"ar_matmul_fp8", "ar_matmul_fp8_workspace", "ar_matmul_fp8_status", "ar_route_experts", "ar_route_experts_workspace", "ar_silu_mul_fp8", "ar_experts_sum"}
    assert set(names) <= set(tda.declared_symbols())
    for n in names:
        assert hasattr(lib, n)


def test_struct_layouts_match_the_header(tmp_path):
    gcc = shutil.which("gcc")
    if gcc is None:
        pytest.skip("no C compiler")
    lines = ["#include <stdio.h>", "#include <stddef.h>", '#include "ar_ffn.h"', "int main(void) {"]
    for cname, py in ffn.STRUCTS.items():
        lines.append(f'    printf("{cname} size %zu\\n", sizeof({cname}));')
        lines += [f'    printf("{cname} {f} %zu\\n", offsetof({cname}, {f}));' for f, _ in py._fields_]
    src = tmp_path / "layout.c"
    src.write_text("\n".join(lines + ["    return 0;", "}"]) + "\n")
    exe = tmp_path / "layout"
    subprocess.run([gcc, "-std=c99", "-pedantic", "-Wall", "-Werror", "-I", ar._build.INCLUDE, str(src), "-o", str(exe)], check=True)
    got = subprocess.run([str(exe)], check=True, capture_output=True, text=True).stdout.split("\n")
    c = {tuple(x.split()[:2]): int(x.split()[2]) for x in got if x.strip()}
    for cname, py in ffn.STRUCTS.items():
        assert ctypes.sizeof(py) == c[(cname, "size")], cname
        for f, _ in py._fields_:
            assert getattr(py, f).offset == c[(cname, f)], (cname, f)


def _rc(lib, name, args):
    return getattr(lib, name)(ctypes.addressof(args), None)


A = 4096   # an address that no refused call touches


def _matmul(**kw):
    base = dict(x=A, x_scales=A, weight=A, weight_scales=A, out=A, offsets=None, row_of=None, workspace=None, x_stride=256, x_scales_stride=2,
                weight_stride=256, expert_stride=0, out_stride=64, rows=3, x_rows=3, dtype=2, out_dim=64, dim=256, experts=1, x_row_scales=0)
    return ffn.MatmulFp8Args(**{**base, **kw})


def _route(**kw):
    base = dict(logits=A, weights=A, expert_ids=A, offsets=A, rows=A, place=A, workspace=A, logits_stride=8, tokens=3, dtype=4, experts=8, chosen=2, normalize=1)
    return ffn.RouteExpertsArgs(**{**base, **kw})


def _silu(**kw):
    return ffn.SiluMulFp8Args(**{**dict(x=A, out=A, scales=A, x_stride=256, rows=3, dtype=1, dim=128, group=128), **kw})


def _sum(**kw):
    base = dict(x=A, weights=A, place=A, out=A, x_stride=64, out_stride=64, rows=6, tokens=3, dtype=2, dim=64, chosen=2)
    return ffn.ExpertsSumArgs(**{**base, **kw})


@pytest.mark.parametrize("kw,code", [
    (dict(x=None), 1), (dict(x_scales=None), 1), (dict(weight=None), 1), (dict(weight_scales=None), 1), (dict(out=None), 1),
    (dict(x_scales=A + 2), 1), (dict(weight_scales=A + 1), 1), (dict(out=A + 1), 1), (dict(offsets=A + 2), 1),
    (dict(row_of=A + 2), 1), (dict(workspace=A + 8), 1), (dict(dtype=3), 1), (dict(dtype=0), 1), (dict(rows=-1, x_rows=-1), 1), (dict(x_rows=4), 1), (dict(dim=-1), 1),
    (dict(out_dim=-1), 1), (dict(experts=0, offsets=A), 1), (dict(experts=2), 1), (dict(x_row_scales=2), 1),
    (dict(rows=(1 << 30) + 1, x_rows=(1 << 30) + 1), 2), (dict(row_of=A, x_rows=(1 << 30) + 1), 2), (dict(dim=(1 << 20) + 1), 2),
    (dict(out_dim=(1 << 20) + 1), 2), (dict(offsets=A, experts=1025), 2)])
def test_matmul_refusals(lib, kw, code):
    assert _rc(lib, "ar_matmul_fp8", _matmul(**kw)) == code


@pytest.mark.parametrize("kw,code", [
    (dict(logits=None), 1), (dict(weights=None), 1), (dict(expert_ids=None), 1), (dict(offsets=None), 1), (dict(rows=None), 1),
    (dict(place=None), 1), (dict(logits=A + 2), 1), (dict(weights=A + 2), 1), (dict(expert_ids=A + 1), 1), (dict(offsets=A + 1), 1),
    (dict(rows=A + 2), 1), (dict(place=A + 2), 1), (dict(dtype=3), 1), (dict(dtype=5), 1), (dict(tokens=-1), 1), (dict(experts=0, chosen=0), 1),
    (dict(chosen=0), 1), (dict(chosen=9), 1), (dict(normalize=2), 1), (dict(experts=1025), 2), (dict(experts=64, chosen=33), 2),
    (dict(tokens=(1 << 29) + 1), 2), (dict(tokens=1000, workspace=None), 1),
    (dict(tokens=1000, workspace=A + 2), 1)])
def test_route_refusals(lib, kw, code):
    assert _rc(lib, "ar_route_experts", _route(**kw)) == code


@pytest.mark.parametrize("kw,code", [
    (dict(x=None), 1), (dict(out=None), 1), (dict(scales=None), 1), (dict(x=A + 1), 1), (dict(scales=A + 2), 1), (dict(dtype=3), 1),
    (dict(dtype=4), 1), (dict(rows=-1), 1), (dict(dim=-1), 1), (dict(group=-1), 1), (dict(group=129), 1), (dict(rows=(1 << 30) + 1), 2),
    (dict(dim=(1 << 20) + 1), 2)])
def test_silu_refusals(lib, kw, code):
    assert _rc(lib, "ar_silu_mul_fp8", _silu(**kw)) == code


@pytest.mark.parametrize("kw,code", [
    (dict(x=None), 1), (dict(weights=None), 1), (dict(place=None), 1), (dict(out=None), 1), (dict(x=A + 1), 1), (dict(out=A + 1), 1),
    (dict(weights=A + 2), 1), (dict(place=A + 2), 1), (dict(dtype=3), 1), (dict(rows=-1), 1), (dict(tokens=-1), 1), (dict(dim=-1), 1),
    (dict(chosen=-1), 1), (dict(rows=(1 << 30) + 1), 2), (dict(tokens=(1 << 30) + 1), 2), (dict(dim=(1 << 20) + 1), 2), (dict(chosen=1025), 2)])
def test_sum_refusals(lib, kw, code):
    assert _rc(lib, "ar_experts_sum", _sum(**kw)) == code


def test_the_products_workspace(lib):
    """Room for picked rows and their scales, where there are many of them."""
    def size(**kw):
        return lib.ar_matmul_fp8_workspace(ctypes.addressof(_matmul(**kw)))
    assert size(rows=5000, x_rows=5000) == 0 and size(row_of=A) == 0 and size(row_of=A, rows=5000, dim=0) == 0
    assert size(row_of=A, rows=5000, dim=2560, out_dim=2048) == 5000 * (2560 + 20 * 4)
    assert size(row_of=A, rows=5000, dim=2550, out_dim=2048, x_row_scales=1) == 5000 * (2560 + 4)
    assert size(row_of=A, offsets=A, experts=64, rows=500) == 0 and size(row_of=A, offsets=A, experts=0, rows=5000) == 0
    assert lib.ar_matmul_fp8_workspace(None) == 0


def test_the_routers_workspace(lib):
    """None for what one block does, nor for what a sort does; else four bytes to an expert and block."""
    def size(**kw):
        return lib.ar_route_experts_workspace(ctypes.addressof(_route(**kw)))
    assert size(tokens=3) == 0 and size(tokens=0) == 0 and size(tokens=64) == 0
    assert size(tokens=8191, experts=256, chosen=8) == 128 * 256 * 4
    assert size(tokens=1 << 27, experts=256, chosen=8) == 0
    assert size(tokens=100, experts=2000) == 0 and size(tokens=100, chosen=0) == 0
    assert lib.ar_route_experts_workspace(None) == 0


def test_null_and_empty_calls(lib):
    for name in ("ar_matmul_fp8", "ar_route_experts", "ar_silu_mul_fp8", "ar_experts_sum"):
        assert getattr(lib, name)(None, None) == ar.AR_EINVAL
    # nothing to do: no pointer is looked at
    assert _rc(lib, "ar_matmul_fp8", _matmul(rows=0, x_rows=0, x=None, out=None)) == ar.AR_OK
    assert _rc(lib, "ar_matmul_fp8", _matmul(out_dim=0, weight=None)) == ar.AR_OK
    assert _rc(lib, "ar_silu_mul_fp8", _silu(rows=0, x=None)) == ar.AR_OK
    assert _rc(lib, "ar_experts_sum", _sum(tokens=0, out=None)) == ar.AR_OK
    assert _rc(lib, "ar_experts_sum", _sum(dim=0, x=None)) == ar.AR_OK


def test_binding_refuses_cpu_tensors():
    x, s = torch.zeros(3, 128).to(H.F8), torch.ones(3, 1)
    h, i = torch.zeros(3, 8, dtype=torch.bfloat16), torch.zeros(3, 2, dtype=torch.int32)
    for call in (lambda: tda.matmul_fp8(x, s, x, s[:1]), lambda: tda.experts_matmul_fp8(x, s, x[None], s[None, :1], i[0]),
                 lambda: tda.route_experts(h, 2), lambda: tda.silu_mul_fp8(h), lambda: tda.experts_sum(h, s, i[:, :1])):
        with pytest.raises(ValueError, match="not a CUDA tensor"):
            call()
    with pytest.raises(ValueError, match="not a tensor"):
        tda.matmul_fp8(None, s, x, s[:1])


def test_the_plain_product_is_that_of_the_widened_values():
    g = H.gen(3)
    x, w = H.eights(g, 5, 300), H.eights(g, 260, 300)
    xs, ws = H.scales(g, 5, 3), H.scales(g, 3, 3)
    wide_x = x.double() * xs.double().repeat_interleave(128, 1)[:, :300]
    wide_w = w.double() * ws.double().repeat_interleave(128, 0)[:260].repeat_interleave(128, 1)[:, :300]
    out, mag = H.product(x, xs, w, ws)
    assert torch.allclose(out, wide_x @ wide_w.T, rtol=1e-12, atol=1e-12 * mag.max().item())
    assert torch.allclose(mag, wide_x.abs() @ wide_w.abs().T, rtol=1e-12)


def test_the_plain_router_takes_the_lower_number_of_equal_ones():
    inf, nan = float("inf"), float("nan")
    x = torch.tensor([[1.0, 2.0, 2.0, 0.0], [-inf, -inf, -inf, -inf], [nan, -inf, 3.0, -1.0], [0.0, -0.0, 0.0, 0.0]])
    w, e, o, r, p = H.route(x, 3, True)
    assert e.tolist() == [[1, 2, 0], [-1, -1, -1], [2, 3, -1], [0, 1, 2]]
    assert o.tolist() == [0, 2, 4, 7, 8] and r.tolist() == [0, 3, 0, 3, 0, 2, 3, 2] + [-1] * 4
    assert p.tolist() == [[2, 4, 0], [-1] * 3, [5, 7, -1], [1, 3, 6]] and w.sum(1).tolist() == [1, 0, 1, 1]
