"""The operators of include/ar_ops.h without a GPU: the header, the binding's
structs, the refusals that come before any CUDA call, and the test packing."""
import ctypes
import os
import shutil
import subprocess

import numpy as np
import pytest
import torch

import tensor_decode_all_gb300 as tda
from tensor_decode_all_gb300 import ar, ops
from tests import ops_helpers as H


@pytest.fixture(scope="module")
def lib():
    tda.build()
    return ops._ops()


def test_symbols_are_declared_and_exported(lib):
    names = tda.declared_symbols(os.path.join(ar._build.INCLUDE, "ar_ops.h"))
    assert set(names) == {"ar_kv_plan", "ar_kv4_append", "ar_kv4_load", "ar_kv4_attend", "ar_kv4_workspace_bytes",
                          "ar_kv4_workspace_init", "ar_kv4_status", "ar_add_norm_fp8"}
    assert set(names) <= set(tda.declared_symbols())
    for n in names:
        assert hasattr(lib, n)


def test_struct_layouts_match_the_header(tmp_path):
    gcc = shutil.which("gcc")
    if gcc is None:
        pytest.skip("no C compiler")
    lines = ["#include <stdio.h>", "#include <stddef.h>", '#include "ar_ops.h"', "int main(void) {"]
    for cname, py in ops.STRUCTS.items():
        lines.append(f'    printf("{cname} size %zu\\n", sizeof({cname}));')
        lines += [f'    printf("{cname} {f} %zu\\n", offsetof({cname}, {f}));' for f, _ in py._fields_]
    src = tmp_path / "layout.c"
    src.write_text("\n".join(lines + ["    return 0;", "}"]) + "\n")
    exe = tmp_path / "layout"
    subprocess.run([gcc, "-std=c99", "-pedantic", "-Wall", "-Werror", "-I", ar._build.INCLUDE, str(src), "-o", str(exe)],
                   check=True)
    got = subprocess.run([str(exe)], check=True, capture_output=True, text=True).stdout.split("\n")
    c = {tuple(x.split()[:2]): int(x.split()[2]) for x in got if x.strip()}
    for cname, py in ops.STRUCTS.items():
        assert ctypes.sizeof(py) == c[(cname, "size")], cname
        for f, _ in py._fields_:
            assert getattr(py, f).offset == c[(cname, f)], (cname, f)


def _rc(lib, name, args):
    return getattr(lib, name)(ctypes.addressof(args), None)


A = 4096   # an address that no refused call touches


def _rows(**kw):
    base = dict(k=A, v=A, pool=A, slots=A, k_token_stride=256, k_head_stride=128, v_token_stride=256, v_head_stride=128,
                pages=4, tokens=3, dtype=2, kv_heads=2, head_dim=128, page=16)
    return ops.Kv4RowsArgs(**{**base, **kw})


def _attend(**kw):
    base = dict(q=A, out=A, lse=A, pool=A, table=A, lens=A, cu=None, workspace=A, q_token_stride=1024, q_head_stride=128,
                out_token_stride=1024, out_head_stride=128, table_stride=4, pages=4, dtype=2, tokens=3, requests=3,
                max_new=1, q_heads=8, kv_heads=2, head_dim=128, page=16, table_width=4, window=0, sinks=0, scale=0.1)
    return ops.Kv4AttendArgs(**{**base, **kw})


def _plan(**kw):
    base = dict(lens=A, new_tokens=A, table=A, free_pages=A, free_used=A, lens_out=A, cu=A, slots=A, request=A, position=A,
                free_used_out=A, status=A, table_stride=4, free_count=9, requests=3, table_width=4, page=16, max_tokens=3)
    return ops.KvPlanArgs(**{**base, **kw})


def _norm(**kw):
    base = dict(x=A, residual=A, weight=A, out=A, scales=A, residual_out=A, x_stride=64, residual_stride=64,
                residual_out_stride=64, rows=2, dtype=1, dim=64, group=0, eps=1e-6)
    return ops.AddNormFp8Args(**{**base, **kw})


@pytest.mark.parametrize("name", ["ar_kv4_append", "ar_kv4_load"])
@pytest.mark.parametrize("kw", [dict(k=None), dict(v=None), dict(pool=None), dict(slots=None), dict(k=A + 1), dict(pool=A + 8),
                                dict(slots=A + 4), dict(dtype=3), dict(dtype=0), dict(head_dim=96), dict(head_dim=32),
                                dict(page=8), dict(page=24), dict(page=0), dict(tokens=-1), dict(kv_heads=0), dict(pages=-1)])
def test_rows_refusals(lib, name, kw):
    assert _rc(lib, name, _rows(**kw)) == ar.AR_EINVAL


@pytest.mark.parametrize("kw,code", [
    (dict(q=None), 1), (dict(out=None), 1), (dict(pool=None), 1), (dict(table=None), 1), (dict(lens=None), 1),
    (dict(workspace=None), 1), (dict(workspace=A + 128), 1), (dict(q=A + 1), 1), (dict(lse=A + 2), 1), (dict(lens=A + 2), 1),
    (dict(dtype=3), 1), (dict(head_dim=80), 1), (dict(q_heads=7), 1), (dict(q_heads=0), 1), (dict(kv_heads=0), 1),
    (dict(page=20), 1), (dict(tokens=4), 1), (dict(tokens=-1, requests=-1), 1), (dict(table_stride=3), 1), (dict(window=-1), 1),
    (dict(sinks=-1), 1), (dict(pages=-1), 1), (dict(scale=float("nan")), 1), (dict(scale=float("inf")), 1), (dict(max_new=-1), 1),
    (dict(requests=0, cu=A), 1), (dict(requests=8193, tokens=8193), 2)])
def test_attend_refusals(lib, kw, code):
    assert _rc(lib, "ar_kv4_attend", _attend(**kw)) == code


@pytest.mark.parametrize("kw,code", [
    (dict(lens=None), 1), (dict(new_tokens=None), 1), (dict(table=None), 1), (dict(free_pages=None), 1), (dict(free_used=None), 1),
    (dict(lens_out=None), 1), (dict(cu=None), 1), (dict(slots=None), 1), (dict(request=None), 1), (dict(position=None), 1),
    (dict(free_used_out=None), 1), (dict(status=None), 1), (dict(slots=A + 4), 1), (dict(lens=A + 1), 1), (dict(page=17), 1),
    (dict(requests=-1), 1), (dict(max_tokens=-1), 1), (dict(table_width=5), 1), (dict(free_count=-1), 1),
    (dict(requests=8193), 2)])
def test_plan_refusals(lib, kw, code):
    assert _rc(lib, "ar_kv_plan", _plan(**kw)) == code


@pytest.mark.parametrize("kw,code", [
    (dict(x=None), 1), (dict(weight=None), 1), (dict(out=None), 1), (dict(scales=None), 1), (dict(x=A + 1), 1),
    (dict(scales=A + 2), 1), (dict(dtype=3), 1), (dict(rows=-1), 1), (dict(dim=-1), 1), (dict(group=-1), 1), (dict(group=65), 1),
    (dict(eps=-1.0), 1), (dict(eps=float("nan")), 1), (dict(dim=32769), 2)])
def test_norm_refusals(lib, kw, code):
    assert _rc(lib, "ar_add_norm_fp8", _norm(**kw)) == code


def test_null_and_empty_calls(lib):
    for name in ("ar_kv_plan", "ar_kv4_append", "ar_kv4_load", "ar_kv4_attend", "ar_add_norm_fp8"):
        assert getattr(lib, name)(None, None) == ar.AR_EINVAL
    # nothing to do: no pointer is looked at
    assert _rc(lib, "ar_kv4_append", _rows(tokens=0, k=None, v=None)) == ar.AR_OK
    assert _rc(lib, "ar_kv4_attend", _attend(tokens=0, requests=0, q=None, out=None)) == ar.AR_OK
    assert _rc(lib, "ar_add_norm_fp8", _norm(rows=0, x=None)) == ar.AR_OK
    assert lib.ar_kv4_workspace_init(None, None) == ar.AR_EINVAL
    assert lib.ar_kv4_workspace_init(A + 16, None) == ar.AR_EINVAL
    assert lib.ar_kv4_status(None) == ar.AR_EINVAL
    assert lib.ar_kv4_workspace_bytes() % 256 == 0


def test_binding_refuses_cpu_tensors():
    pool = torch.zeros(4, 2, 1, 2304, dtype=torch.uint8)
    q = torch.zeros(3, 8, 128, dtype=torch.bfloat16)
    i = torch.zeros(3, dtype=torch.int32)
    with pytest.raises(ValueError, match="not a CUDA tensor"):
        tda.kv4_attend(q, pool, torch.zeros(3, 4, dtype=torch.int32), i)
    with pytest.raises(ValueError, match="not a CUDA tensor"):
        tda.kv4_append(q[:, :2], q[:, :2], pool, i.long())
    with pytest.raises(ValueError, match="not a CUDA tensor"):
        tda.kv4_load(pool, i.long())
    with pytest.raises(ValueError, match="not a CUDA tensor"):
        tda.kv_plan(i, i, i[None], i, i[:1], page=16, max_tokens=3)
    with pytest.raises(ValueError, match="not a CUDA tensor"):
        tda.add_norm_fp8(q[0], q[0, 0])
    with pytest.raises(ValueError, match="head_dim"):
        tda.kv4_pool(4, 2, 96, 16, device="cpu")
    assert tda.kv4_pool(4, 2, 64, 32, device="cpu").shape == (4, 2, 2, 1152)


@pytest.mark.parametrize("D", [64, 128, 256])
def test_packing_is_a_bijection_and_keeps_tokens_apart(D):
    """Every nibble of a tile belongs to one token and channel, and no byte to two tokens."""
    kb, ks, vb, vs, si = H.cells(D)
    for b, s, base in ((kb, ks, 0), (vb, vs, 8 * D)):
        assert sorted(zip(b.ravel().tolist(), s.ravel().tolist())) == [(base + i // 2, i % 2 * 4) for i in range(16 * D)]
        for byte in np.unique(b):
            assert len(set(np.nonzero(b == byte)[0])) == 1
    assert si.max() == 16 * D // 32 - 1
    g = torch.Generator().manual_seed(D)
    n = torch.randint(-7, 8, (2, 3, 16, D), generator=g)
    s = torch.rand(2, 3, 16, D // 32, generator=g).to(torch.bfloat16)
    kn, ksc, vn, vsc = H.unpack(H.pack(n, s, -n, s * 2))
    assert torch.equal(kn, n.double()) and torch.equal(vn, -n.double())
    assert torch.equal(ksc[..., ::32], s.double()) and torch.equal(vsc[..., 5::32], 2 * s.double())
