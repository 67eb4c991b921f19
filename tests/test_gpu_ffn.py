"""The operators of include/ar_ffn.h against plain implementations in 64 bits (tests/ffn_helpers.py)."""
import ctypes
import math
import os
import subprocess
import sys
import threading

import pytest
import torch

from tests import ffn_helpers as H

pytestmark = pytest.mark.gpu

F8 = H.F8


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__
    __graft_entry__.build()


def _tda():
    import tensor_decode_all_gb300 as tda
    return tda


def _i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _operands(seed, M, N, K, E=None, row_scale=False):
    g = H.gen(seed)
    G, B = -(-K // 128), -(-N // 128)
    lead = () if E is None else (E,)
    return H.eights(g, M, K), H.scales(g, M, 1 if row_scale else G), H.eights(g, *lead, N, K), H.scales(g, *lead, B, G)


# ----------------------------------------------------------------- matmul_fp8

@pytest.mark.parametrize("M,N,K", [
    (1, 128, 128), (1, 1, 16), (2, 8, 144), (3, 129, 256), (7, 300, 1040), (8, 1280, 512), (15, 127, 128), (16, 128, 384), (17, 256, 400),
    (31, 64, 2048), (32, 640, 640), (33, 384, 128), (63, 256, 1152), (64, 512, 512), (65, 136, 272), (100, 1000, 1008), (127, 256, 256), (128, 384, 1024),
    (129, 257, 528), (255, 256, 384), (256, 512, 256), (300, 700, 640), (513, 264, 896), (1000, 1288, 512)])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_products(M, N, K, dtype):
    x, xs, w, ws = _operands(M * 7 + N + K, M, N, K, row_scale=(M + N) % 3 == 0)
    out = _tda().matmul_fp8(x.cuda(), xs.cuda(), w.cuda(), ws.cuda(), dtype=H.DT[dtype])
    assert out.dtype == H.DT[dtype]
    H.check_product(out, x, xs, w, ws)


@pytest.mark.parametrize("M,N,K", [(1, 5, 1), (5, 66, 7), (66, 130, 129), (70, 65, 1001), (130, 129, 255)])
def test_products_of_odd_rows(M, N, K):
    """Rows that do not begin on 16 bytes."""
    x, xs, w, ws = _operands(M + N + K, M, N, K)
    H.check_product(_tda().matmul_fp8(x.cuda(), xs.cuda(), w.cuda(), ws.cuda()), x, xs, w, ws)


def _padded(t, left, right):
    """The same values inside wider rows, on the GPU."""
    wide = torch.full((*t.shape[:-1], t.shape[-1] + left + right), 0x7f, dtype=torch.uint8, device="cuda").view(t.dtype) if t.dtype == F8 else \
        torch.full((*t.shape[:-1], t.shape[-1] + left + right), math.nan, dtype=t.dtype, device="cuda")
    view = wide[..., left:left + t.shape[-1]]
    view.view(torch.uint8 if t.dtype == F8 else t.dtype).copy_(t.cuda().view(torch.uint8 if t.dtype == F8 else t.dtype))
    return view


@pytest.mark.parametrize("M", [5, 200])
@pytest.mark.parametrize("left,right", [(16, 32), (1, 0), (16, 3), (0, 16)])
@pytest.mark.parametrize("which", ["x", "w", "both"])
def test_products_of_strided_rows(M, left, right, which):
    """Rows inside wider ones, on 16 bytes and not; what lies around them is NaN.  The output is strided too."""
    N, K = 200, 336
    x, xs, w, ws = _operands(left * 31 + right + M, M, N, K)
    xd = _padded(x, left, right) if which != "w" else x.cuda()
    wd = _padded(w, left, right) if which != "x" else w.cuda()
    room = torch.full((M, N + 24), 7.0, dtype=torch.bfloat16, device="cuda")
    for at in (0, 8, 3):
        room.fill_(7.0)
        out = room[:, at:at + N]
        assert _tda().matmul_fp8(xd, _padded(xs, 1, 2), wd, ws.cuda(), out=out) is out
        H.check_product(out, x, xs, w, ws)
        assert (room[:, :at] == 7).all() and (room[:, at + N:] == 7).all()


@pytest.mark.parametrize("M", [4, 300])
def test_a_nan_stays_in_its_row_and_column(M):
    N, K = 260, 272
    x, xs, w, ws = _operands(5, M, N, K)
    want = _tda().matmul_fp8(x.cuda(), xs.cuda(), w.cuda(), ws.cuda())
    x2, w2 = x.clone().view(torch.uint8), w.clone().view(torch.uint8)
    x2[M - 2, 200] = 0x7f
    w2[133, 271] = 0xff
    got = _tda().matmul_fp8(x2.view(F8).cuda(), xs.cuda(), w2.view(F8).cuda(), ws.cuda())
    assert got[M - 2].isnan().all() and got[:, 133].isnan().all()
    keep, cols = torch.arange(M, device="cuda") != M - 2, torch.arange(N, device="cuda") != 133
    assert torch.equal(got[keep][:, cols], want[keep][:, cols])


@pytest.mark.parametrize("M", [4, 300])
def test_scales_multiply_each_groups_sum(M):
    """Groups whose scales are 0, huge and tiny; an infinite scale reaches its own row or block alone."""
    N, K = 256, 512
    x, xs, w, ws = _operands(6, M, N, K)
    xs[:, 1] = 0
    xs[:, 2] *= 1e20
    ws[:, 2] *= 1e-20
    H.check_product(_tda().matmul_fp8(x.cuda(), xs.cuda(), w.cuda(), ws.cuda()), x, xs, w, ws)
    ws[1, 3] = math.inf
    got = _tda().matmul_fp8(x.cuda(), xs.cuda(), w.cuda(), ws.cuda())
    assert not got[:, :128].isinf().any() and not got[:, :128].isnan().any() and not got[:, 128:].isfinite().any()


@pytest.mark.parametrize("M", [3, 150])
def test_sums_of_large_and_small_terms(M):
    """A group holds one pair of opposite large terms and many small ones: nothing is lost beyond the bound."""
    N, K = 128, 256
    x, xs, w, ws = _operands(8, M, N, K)
    x, w = (x.float() * 0.01).to(F8), (w.float() * 0.01).to(F8)
    x[:, 5], x[:, 90] = 448.0, -448.0
    w[:, 5], w[:, 90] = 448.0, 448.0
    H.check_product(_tda().matmul_fp8(x.cuda(), xs.cuda(), w.cuda(), ws.cuda()), x, xs, w, ws)


def test_empty_products():
    tda = _tda()
    x, xs, w, ws = (t.cuda() for t in _operands(1, 4, 64, 128))
    assert tda.matmul_fp8(x[:0], xs[:0], w, ws).shape == (0, 64)
    assert tda.matmul_fp8(x, xs, w[:0], ws[:0]).shape == (4, 0)
    out = tda.matmul_fp8(x[:, :0], xs[:, :0], w[:, :0], ws[:, :0])        # no channels: sums of nothing
    assert out.shape == (4, 64) and (out == 0).all()
    assert (tda.matmul_fp8(x[:, :0], xs, w[:, :0], ws[:, :0]) == 0).all()


def test_products_are_the_same_every_time():
    tda = _tda()
    for M, N, K in ((3, 512, 4096), (40, 384, 2048), (700, 640, 1024)):
        ops = [t.cuda() for t in _operands(M, M, N, K)]
        first = tda.matmul_fp8(*ops)
        for _ in range(5):
            assert torch.equal(tda.matmul_fp8(*ops), first)
    torch.cuda.synchronize()
    tda.matmul_fp8_check()


# --------------------------------------------------------- experts_matmul_fp8

def _check_experts(out, x, xs, w, ws, offsets, rows=None):
    for e in range(w.shape[0]):
        a, b = offsets[e], offsets[e + 1]
        if b > a:
            who = torch.arange(a, b) if rows is None else torch.tensor(rows[a:b])
            H.check_product(out[a:b], x.view(torch.uint8)[who].view(F8), xs[who], w[e], ws[e])


@pytest.mark.parametrize("counts", [[1], [0, 3], [5, 0, 0, 17, 1, 0], [16, 16, 16], [130, 0, 1, 64, 33], [300, 7, 129], [0, 0, 0, 40], [1] * 40, [2, 700, 2]])
@pytest.mark.parametrize("N,K", [(128, 256), (200, 400)])
@pytest.mark.parametrize("gather", [False, True])
def test_experts(counts, N, K, gather):
    E, R = len(counts), sum(counts)
    offsets = [0]
    for n in counts:
        offsets.append(offsets[-1] + n)
    T = max(1, R // 2) if gather else R
    x, xs, w, ws = _operands(R + N, T, N, K, E)
    rows = torch.randint(0, T, (R,), generator=H.gen(R)).tolist() if gather else None
    out = _tda().experts_matmul_fp8(x.cuda(), xs.cuda(), w.cuda(), ws.cuda(), _i32(offsets), rows=_i32(rows) if gather else None)
    _check_experts(out, x, xs, w, ws, offsets, rows)


@pytest.mark.parametrize("n", [20, 400])
def test_rows_of_no_expert_stay_as_they_were(n):
    N, K, E = 136, 272, 3
    offsets = [5, 5 + n // 4, 5 + n // 4, n - 7]
    x, xs, w, ws = _operands(n, n, N, K, E)
    out = torch.full((n, N), 3.0, dtype=torch.float16, device="cuda")
    _tda().experts_matmul_fp8(x.cuda(), xs.cuda(), w.cuda(), ws.cuda(), _i32(offsets), out=out)
    _check_experts(out, x, xs, w, ws, offsets)
    assert (out[:5] == 3).all() and (out[n - 7:] == 3).all()


@pytest.mark.parametrize("n", [20, 400])
def test_row_numbers_outside_x_give_zeros(n):
    N, K, E = 136, 272, 2
    x, xs, w, ws = _operands(n, 9, N, K, E)
    rows = torch.randint(0, 9, (n,), generator=H.gen(1))
    bad = {1: -1, 4: 9, n - 1: 2 ** 31 - 1, n // 2: -2 ** 31, n // 2 + 1: 1000}
    for i, v in bad.items():
        rows[i] = v
    out = _tda().experts_matmul_fp8(x.cuda(), xs.cuda(), w.cuda(), ws.cuda(), _i32([0, n // 2, n]), rows=rows.int().cuda())
    assert (out[list(bad)] == 0).all()
    for e, (a, b) in enumerate(((0, n // 2), (n // 2, n))):
        keep = [i for i in range(a, b) if i not in bad]
        H.check_product(out[keep], x.view(torch.uint8)[rows[keep]].view(F8), xs[rows[keep]], w[e], ws[e])
    none = _tda().experts_matmul_fp8(x[:0].cuda(), xs[:0].cuda(), w.cuda(), ws.cuda(), _i32([0, n // 2, n]), rows=rows.int().cuda())
    assert (none == 0).all()


def test_offsets_that_are_wrong_stay_inside():
    """Negative, past the end, decreasing: the call touches nothing around its buffers, and good experts are right."""
    n, N, K, E = 50, 128, 256, 4
    x, xs, w, ws = _operands(2, n, N, K, E)
    for offsets in ([-9, 10, 20, 30, 2 ** 31 - 1], [0, 2 ** 31 - 1, 20, 30, 50], [0, 40, 10, 30, 50], [50, 40, 30, 20, 10], [-5] * 5, [99] * 5):
        room = torch.full((n + 20, N), 5.0, dtype=torch.bfloat16, device="cuda")
        out = _tda().experts_matmul_fp8(x.cuda(), xs.cuda(), w.cuda(), ws.cuda(), _i32(offsets), out=room[10:n + 10])
        torch.cuda.synchronize()
        assert (room[:10] == 5).all() and (room[n + 10:] == 5).all()
        if offsets[0] == -9:
            _check_experts(out, x, xs, w, ws, [0, 10, 20, 30, 50])
    _tda().matmul_fp8_check()


@pytest.mark.parametrize("n", [50, 600])
@pytest.mark.parametrize("K", [1024, 250])
@pytest.mark.parametrize("gather", [False, True])
def test_wrong_offsets_in_every_kernel(n, K, gather):
    """Few rows, many, and rows off 16 bytes, in place and picked: the call stays inside its buffers, and offsets that are good where they are
    brought inside 0 .. rows give the right rows."""
    N, E = 600, 4
    x, xs, w, ws = _operands(n + K, 40 if gather else n, N, K, E)
    rows = torch.randint(0, 40, (n,), generator=H.gen(n)).tolist() if gather else None
    dev = [t.cuda() for t in (x, xs, w, ws)]
    big = 2 ** 31 - 1
    room = torch.empty(n + 20, N, dtype=torch.bfloat16, device="cuda")
    for offsets in ([-9, n // 5, n // 2, n - 7, big], [-big, -1, 0, n + 1, big], [0, big, 20, 30, n], [0, n, 0, n, 0], [0, n - 10, 10, 30, n], [n, 40, 30, 20, 10],
                    [n // 2, n, 0, 5, n // 3], [-5] * 5, [n + 99] * 5):
        room.fill_(5.0)
        out = _tda().experts_matmul_fp8(*dev, _i32(offsets), rows=_i32(rows) if gather else None, out=room[10:n + 10])
        torch.cuda.synchronize()
        assert (room[:10] == 5).all() and (room[n + 10:] == 5).all()
        inside = [min(max(o, 0), n) for o in offsets]
        if inside == sorted(inside):
            _check_experts(out, x, xs, w, ws, inside, rows)
            assert (out[:inside[0]] == 5).all() and (out[inside[-1]:] == 5).all()
    _tda().matmul_fp8_check()


@pytest.mark.parametrize("K,row_scale", [(2560, False), (2672, False), (2560, True)])
@pytest.mark.parametrize("gather", [False, True])
def test_experts_with_an_odd_output_and_many_rows(K, row_scale, gather):
    """Results that leave by twos of bytes from whole and short tiles, experts' ends among them."""
    N, counts = 2301, [300, 100, 512, 0, 1, 700, 129, 306]
    offsets = [0]
    for c in counts:
        offsets.append(offsets[-1] + c)
    R = offsets[-1]
    T = R // 3 if gather else R
    x, xs, w, ws = _operands(K, T, N, K, len(counts), row_scale)
    rows = torch.randint(0, T, (R,), generator=H.gen(K)).tolist() if gather else None
    out = _tda().experts_matmul_fp8(x.cuda(), xs.cuda(), w.cuda(), ws.cuda(), _i32(offsets), rows=_i32(rows) if gather else None, dtype=torch.float16)
    _check_experts(out, x, xs, w, ws, offsets, rows)


@pytest.mark.parametrize("counts", [[3], [0, 5, 70, 0, 1], [200, 64, 65, 0, 300]])
@pytest.mark.parametrize("N,K", [(130, 129), (65, 1001), (64, 7)])
@pytest.mark.parametrize("gather", [False, True])
def test_experts_of_odd_rows(counts, N, K, gather):
    """Rows that do not begin on 16 bytes."""
    offsets = [0]
    for c in counts:
        offsets.append(offsets[-1] + c)
    R = offsets[-1]
    T = max(1, R // 2) if gather else R
    x, xs, w, ws = _operands(R + K, T, N, K, len(counts))
    rows = torch.randint(0, T, (R,), generator=H.gen(R)).tolist() if gather else None
    out = _tda().experts_matmul_fp8(x.cuda(), xs.cuda(), w.cuda(), ws.cuda(), _i32(offsets), rows=_i32(rows) if gather else None)
    _check_experts(out, x, xs, w, ws, offsets, rows)


@pytest.mark.parametrize("layout", ["wider", "no whole rows between", "odd", "side by side", "one for all"])
@pytest.mark.parametrize("R", [20, 1500])
@pytest.mark.parametrize("gather", [False, True])
def test_experts_of_strided_weights(layout, R, gather):
    """Weights inside wider ones; whose experts lie 16 bytes times any number apart, or an odd number; with the experts' rows taking turns; all
    experts the same one.  What lies between them is NaN."""
    E, N, K = 5, 600, 1024
    T = 40 if gather else R
    x, xs, w, ws = _operands(R, T, N, K, E)
    if layout == "one for all":
        w = w.view(torch.uint8)[:1].expand(E, -1, -1).view(F8)
    room = torch.full((E * (N + 16) * (K + 32) + 64,), 0x7f, dtype=torch.uint8, device="cuda").view(F8)
    strides = {"wider": ((N + 16) * (K + 32), K + 32), "no whole rows between": (N * (K + 32) + 48, K + 32), "odd": (N * (K + 32) + 49, K + 32),
               "side by side": (K, E * K), "one for all": (0, K)}[layout]
    wd = room[16:].as_strided((E, N, K), (*strides, 1))
    for e in range(1 if layout == "one for all" else E):
        wd[e].view(torch.uint8).copy_(w[e].view(torch.uint8))
    offsets = [0, R // 7, R // 2, R // 2, R - 3, R]
    rows = torch.randint(0, T, (R,), generator=H.gen(R)).tolist() if gather else None
    out = _tda().experts_matmul_fp8(x.cuda(), xs.cuda(), wd, ws.cuda(), _i32(offsets), rows=_i32(rows) if gather else None)
    _check_experts(out, x, xs, w, ws, offsets, rows)


def test_host_threads_at_once():
    """Threads that call the library at the same time (ctypes lets go of the interpreter's lock), each on its own stream, the first calls of their
    sizes among them."""
    from tensor_decode_all_gb300 import ffn
    lib, jobs = ffn._ffn(), []
    for seed, (M, N, K) in enumerate(((9, 384, 4096), (50, 640, 2048), (128, 768, 1024), (1600, 768, 1024), (3, 130, 129), (20, 1152, 2048))):
        ops = _operands(seed, M, N, K)
        dev = [t.cuda() for t in ops]
        jobs.append((ops, dev, [torch.empty(M, N, dtype=torch.bfloat16, device="cuda") for _ in range(12)], torch.cuda.Stream()))
    torch.cuda.synchronize()
    gate, codes = threading.Barrier(len(jobs)), []

    def work(dev, outs, stream):
        gate.wait()
        for out in outs:
            x, xs, w, ws = dev
            args = ffn.MatmulFp8Args(x=x.data_ptr(), x_scales=xs.data_ptr(), weight=w.data_ptr(), weight_scales=ws.data_ptr(), out=out.data_ptr(), x_stride=x.stride(0),
                                     x_scales_stride=xs.stride(0), weight_stride=w.stride(0), out_stride=out.stride(0), rows=len(x), x_rows=len(x), dtype=2,
                                     out_dim=w.shape[0], dim=x.shape[1], experts=1)
            codes.append(lib.ar_matmul_fp8(ctypes.addressof(args), stream.cuda_stream))

    threads = [threading.Thread(target=work, args=j[1:]) for j in jobs]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert codes == [0] * (12 * len(jobs))
    for ops, _, outs, _ in jobs:
        H.check_product(outs[0], *ops)
        assert all(torch.equal(o, outs[0]) for o in outs[1:])
    _tda().matmul_fp8_check()


def test_the_first_call_of_a_host_thread():
    """A thread that has made no CUDA call before, as a server's worker: each operator, also under a capture."""
    tda = _tda()
    small, large = ([t.cuda() for t in _operands(seed, M, 600, 1024)] for seed, M in ((1, 9), (2, 2000)))
    x, logits, place = torch.randn(9, 256, device="cuda").half(), torch.randn(9, 8, device="cuda"), torch.zeros(9, 2, dtype=torch.int32, device="cuda")
    weights = torch.ones(9, 2, device="cuda")
    calls = [lambda: tda.matmul_fp8(*small), lambda: tda.matmul_fp8(*large), lambda: tda.route_experts(logits, 2)[1], lambda: tda.silu_mul_fp8(x)[1],
             lambda: tda.experts_sum(x, weights, place)]
    want = [f() for f in calls]
    torch.cuda.synchronize()

    def captured(f):
        graph, s = torch.cuda.CUDAGraph(), torch.cuda.Stream()
        with torch.cuda.graph(graph, stream=s, capture_error_mode="thread_local"):
            out = f()
        graph.replay()
        return out

    for f, w in zip(calls, want):
        for run in (f, lambda: captured(f)):
            got = []

            def work():
                try:
                    got.append(run())
                except Exception as e:          # (an exception does not leave the thread)
                    got.append(e)
            t = threading.Thread(target=work)
            t.start()
            t.join()
            torch.cuda.synchronize()
            assert torch.is_tensor(got[0]), got[0]
            assert torch.equal(got[0], w)


def test_weights_past_32_bits():
    """Over 4 GiB of weights: the last expert's product, whose parts may be added otherwise than a single weight's."""
    tda = _tda()
    N, K = 8192, 8192
    E = (1 << 32) // (N * K) + 2
    x, xs, _, ws = _operands(4, 6, N, K, 1)
    w = torch.empty(E, N, K, dtype=torch.uint8, device="cuda").view(F8)
    w[-1].view(torch.uint8).random_(0, 127, generator=H.gen(1, "cuda"))
    got = tda.experts_matmul_fp8(x.cuda(), xs.cuda(), w, ws.expand(E, -1, -1).contiguous().cuda(), _i32([0] * E + [6]))
    H.check_product(got, x, xs, w[-1].cpu(), ws[0])


def test_many_experts_most_without_rows():
    N, K, E = 128, 128, 1024
    x, xs, w, ws = _operands(9, 12, N, K, E)
    counts = [0] * E
    for i, e in enumerate((0, 1, 31, 32, 500, 1023)):
        counts[e] = 2
    offsets = [0]
    for c in counts:
        offsets.append(offsets[-1] + c)
    out = _tda().experts_matmul_fp8(x.cuda(), xs.cuda(), w.cuda(), ws.cuda(), _i32(offsets))
    _check_experts(out, x, xs, w, ws, offsets)


@pytest.mark.parametrize("M,N,K,row_scale", [(5000, 2304, 256, False), (3, 1280, 20000, False), (40, 130, 9000, True), (2500, 333, 384, True), (1100, 4104, 272, False), (2500, 333, 512, False),
                                           (700, 512, 1536, False)])
def test_products_of_many_tiles_and_long_rows(M, N, K, row_scale):
    """Several tiles to a block, rings of stages gone round many times, an odd output, channels shared by clusters."""
    x, xs, w, ws = _operands(M + N, M, N, K, row_scale=row_scale)
    H.check_product(_tda().matmul_fp8(x.cuda(), xs.cuda(), w.cuda(), ws.cuda()), x, xs, w, ws)


def test_large_products_into_strided_rows():
    """Many rows: outputs on 32 bytes, on 16, and on neither, inside wider rows."""
    M, N, K = 3000, 2312, 2048
    x, xs, w, ws = _operands(17, M, N, K)
    dev = [t.cuda() for t in (x, xs, w, ws)]
    want, mag = H.product(x, xs, w, ws)
    limit = H.product_bound(want, mag, ws.shape[1], torch.float16).cuda()
    want = want.cuda()
    for at, more in ((0, 24), (8, 16), (3, 0), (16, 1)):
        room = torch.full((M + 2, at + N + more), 7.0, dtype=torch.float16, device="cuda")
        out = room[1:M + 1, at:at + N]
        _tda().matmul_fp8(*dev, out=out)
        assert ((out.double() - want).abs() <= limit).all()
        assert (room[0] == 7).all() and (room[M + 1] == 7).all() and (room[:, :at] == 7).all() and (room[:, at + N:] == 7).all()


def test_picked_rows_without_a_workspace():
    """The C call with NULL for it: another kernel, the same product."""
    tda = _tda()
    from tensor_decode_all_gb300 import ffn
    n, N, K = 900, 200, 512
    x, xs, w, ws = _operands(3, 33, N, K)
    rows = torch.randint(0, 33, (n,), generator=H.gen(3)).int()
    dev = [t.cuda() for t in (x, xs, w, ws, rows)]
    out = torch.empty(n, N, dtype=torch.bfloat16, device="cuda")
    args = ffn.MatmulFp8Args(x=dev[0].data_ptr(), x_scales=dev[1].data_ptr(), weight=dev[2].data_ptr(), weight_scales=dev[3].data_ptr(), out=out.data_ptr(),
                             offsets=None, row_of=dev[4].data_ptr(), workspace=None, x_stride=K, x_scales_stride=4, weight_stride=K, expert_stride=0,
                             out_stride=N, rows=n, x_rows=33, dtype=2, out_dim=N, dim=K, experts=1, x_row_scales=0)
    lib = ffn._ffn()
    assert lib.ar_matmul_fp8_workspace(ctypes.addressof(args)) == n * (K + 16)
    assert lib.ar_matmul_fp8(ctypes.addressof(args), torch.cuda.current_stream().cuda_stream) == 0
    H.check_product(out, x.view(torch.uint8)[rows.long()].view(F8), xs[rows.long()], w, ws)
    H.check_product(tda.matmul_fp8(*dev[:4], rows=dev[4]), x.view(torch.uint8)[rows.long()].view(F8), xs[rows.long()], w, ws)


def test_no_rows_picked():
    """An empty `rows`: an empty result, as of a step in which no request needs its logits."""
    tda = _tda()
    x, xs, w, ws = (t.cuda() for t in _operands(1, 7, 64, 256, 3))
    none = _i32([])
    assert tda.matmul_fp8(x, xs, w[0], ws[0], rows=none).shape == (0, 64)
    out = torch.empty(0, 64, dtype=torch.float16, device="cuda")
    assert tda.matmul_fp8(x, xs, w[0], ws[0], rows=none, out=out) is out
    assert tda.experts_matmul_fp8(x, xs, w, ws, _i32([0] * 4), rows=none).shape == (0, 64)
    assert tda.matmul_fp8(x[:0], xs[:0], w[0], ws[0], rows=none).shape == (0, 64)


@pytest.mark.parametrize("n", [1, 20, 100, 900])
@pytest.mark.parametrize("K", [512, 130 * 16, 250])
def test_products_of_picked_rows(n, K):
    """`rows`: any number of times, in any order, numbers outside x among them."""
    x, xs, w, ws = _operands(n + K, 33, 200, K)
    rows = torch.randint(0, 33, (n,), generator=H.gen(n))
    bad = [i for i in (0, 7, n - 1) if 1 < i < n]
    for i in bad:
        rows[i] = 33 + i
    out = _tda().matmul_fp8(x.cuda(), xs.cuda(), w.cuda(), ws.cuda(), rows=rows.int().cuda())
    keep = [i for i in range(n) if i not in bad]
    H.check_product(out[keep], x.view(torch.uint8)[rows[keep]].view(F8), xs[rows[keep]], w, ws)
    assert (out[bad] == 0).all()


@pytest.mark.parametrize("E,each,N,K,row_scale", [(100, 3, 512, 256, True), (300, 1, 256, 144, False), (12, 40, 1024, 640, False), (7, 500, 520, 384, True)])
@pytest.mark.parametrize("gather", [False, True])
def test_experts_of_many_tiles(E, each, N, K, row_scale, gather):
    counts = [each + (i * 7) % 3 for i in range(E)]
    offsets = [0]
    for n in counts:
        offsets.append(offsets[-1] + n)
    R = offsets[-1]
    T = max(1, R // 3) if gather else R
    x, xs, w, ws = _operands(E + each, T, N, K, E, row_scale)
    rows = torch.randint(0, T, (R,), generator=H.gen(E)).tolist() if gather else None
    out = _tda().experts_matmul_fp8(x.cuda(), xs.cuda(), w.cuda(), ws.cuda(), _i32(offsets), rows=_i32(rows) if gather else None, dtype=torch.float16)
    _check_experts(out, x, xs, w, ws, offsets, rows)


def test_products_on_several_streams_at_once():
    """Calls of all kinds that overlap on the GPU, each many times: the same results as alone."""
    tda = _tda()
    jobs = []
    for seed, (M, N, K) in enumerate(((3, 1280, 4096), (60, 2048, 2048), (100, 2048, 1024), (1500, 1024, 512))):
        ops = [t.cuda() for t in _operands(seed, M, N, K)]
        jobs.append((lambda ops=ops: tda.matmul_fp8(*ops)))
    x, xs, w, ws = _operands(9, 200, 512, 512, 8)
    o, rows = _i32([0, 100, 300, 300, 500, 900, 1000, 1400, 1600]), torch.randint(0, 200, (1600,), generator=H.gen(3)).int().cuda()
    ex = [t.cuda() for t in (x, xs, w, ws)]
    jobs.append(lambda: tda.experts_matmul_fp8(*ex, o, rows=rows))
    small = _i32([0, 1, 5, 9, 9, 20, 22, 29, 30])
    jobs.append(lambda: tda.experts_matmul_fp8(*ex, small, rows=rows[:30]))
    alone = [j() for j in jobs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in jobs]
    got = [[] for _ in jobs]
    for _ in range(20):
        for j, s, g in zip(jobs, streams, got):
            with torch.cuda.stream(s):
                g.append(j())
    torch.cuda.synchronize()
    for a, g in zip(alone, got):
        assert all(torch.equal(a, b) for b in g)
    tda.matmul_fp8_check()


def test_a_first_call_under_capture():
    """A process whose first calls are captured: nothing that they set up needs another call before."""
    code = """
import sys, torch
sys.path.insert(0, %r)
import tensor_decode_all_gb300 as tda
from tests import ffn_helpers as H
g = H.gen(1)
def operands(M, N, K):
    return [t.cuda() for t in (H.eights(g, M, K), H.scales(g, M, -(-K // 128)), H.eights(g, N, K), H.scales(g, -(-N // 128), -(-K // 128)))]
small, large = operands(5, 640, 2048), operands(700, 512, 512)
logits, x = torch.randn(900, 64, device="cuda"), torch.randn(8, 256, device="cuda").half()
torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    a, b, r, s = tda.matmul_fp8(*small), tda.matmul_fp8(*large), tda.route_experts(logits, 4), tda.silu_mul_fp8(x)
    t = tda.experts_sum(x.repeat(4, 1), torch.ones(8, 2, device="cuda"), torch.arange(16, dtype=torch.int32, device="cuda").view(8, 2))
graph.replay()
torch.cuda.synchronize()
for out, ops in ((a, small), (b, large)):
    H.check_product(out, *(v.cpu() for v in ops))
H.check_silu(*s, x.cpu(), 128)
assert torch.equal(r.experts, tda.route_experts(logits, 4).experts)
tda.matmul_fp8_check()
""" % os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    done = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, timeout=300)
    assert done.returncode == 0, done.stderr[-2000:]


# -------------------------------------------------------------- route_experts

def _check_route(r, logits, k, normalize):
    w, e, o, rows, place = H.route(logits.cpu(), k, normalize)
    assert torch.equal(r.experts.long().cpu(), e) and torch.equal(r.offsets.long().cpu(), o)
    assert torch.equal(r.rows.long().cpu(), rows) and torch.equal(r.place.long().cpu(), place)
    # the difference of two logits is rounded once (2^-24 of it), exp by 2 units, a sum of E terms in a tree or in order, the division
    spread = (logits.double().cpu().nan_to_num(0, 0, 0).abs().amax(1, keepdim=True) * 2) if len(logits) else torch.zeros(0, 1)
    limit = w * (spread * 2.0 ** -23 + (logits.shape[1] + 8) * 2.0 ** -23) + 2.0 ** -140
    assert ((r.weights.double().cpu() - w).abs() <= limit).all()


@pytest.mark.parametrize("T,E,k", [(1, 1, 1), (1, 8, 8), (2, 32, 4), (5, 33, 5), (7, 60, 6), (64, 64, 8), (33, 128, 8), (300, 256, 8), (3, 1024, 32), (1000, 16, 2),
                                   (40, 512, 1), (1025, 100, 7)])
@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("normalize", [True, False])
def test_routes(T, E, k, dtype, normalize):
    """bfloat16 and float16 logits have many equal ones among them."""
    x = (torch.randn(T, E, generator=H.gen(T + E)) * 2).to(H.DT[dtype])
    _check_route(_tda().route_experts(x.cuda(), k, normalize=normalize), x, k, normalize)


@pytest.mark.parametrize("T,E,k", [(65, 16, 16), (64, 1000, 16), (200, 700, 32), (2049, 513, 3), (33000, 12, 8), (5000, 7, 7)])
def test_routes_of_many_tokens(T, E, k):
    """In one block, in many, and past what those take; a column of equal logits, and tokens without an expert."""
    x = torch.randn(T, E, generator=H.gen(T)).half()
    x[:, E // 2] = 1.0
    x[T // 3:T // 3 + 5] = -math.inf
    _check_route(_tda().route_experts(x.cuda(), k), x, k, True)


@pytest.mark.parametrize("normalize", [True, False])
def test_routes_of_special_logits(normalize):
    inf, nan = math.inf, math.nan
    x = torch.randn(12, 40, generator=H.gen(2))
    x[0] = -inf
    x[1] = nan
    x[2] = 0.0
    x[2, ::2] = -0.0
    x[3] = -inf
    x[3, 39] = -5.0
    x[4, 7], x[4, 30] = inf, inf
    x[5, :20] = nan
    x[6] = torch.finfo(torch.float32).min
    x[7] = -torch.finfo(torch.float32).max
    x[7, 3] = torch.finfo(torch.float32).max
    x[8, :36] = -inf
    x[9] = 1e-45
    x[9, 5] = 0.0
    for k in (1, 4, 6):
        r = _tda().route_experts(x.cuda(), k, normalize=normalize)
        _check_route(r, x, k, normalize)
    assert r.experts[0].tolist() == [-1] * 6 and r.weights[0].tolist() == [0.0] * 6
    assert (r.rows[r.offsets[-1]:] == -1).all() and len(r.rows) > r.offsets[-1]


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_routes_of_special_short_logits(dtype):
    """16-bit types' ends: infinities beside their largest number, subnormals, zeros of both signs, NaN of both signs."""
    dt = H.DT[dtype]
    big, tiny = torch.finfo(dt).max, torch.finfo(dt).smallest_normal / 4
    row = [0.0, -0.0, math.nan, -math.nan, math.inf, -math.inf, big, -big, tiny, -tiny, 1.0, -1.0] + [0.5] * 21
    x = torch.tensor([row, row[::-1], [-v for v in row], [v if v == v and abs(v) < 1 else -math.inf for v in row]]).to(dt)
    for k in (1, 5, 12, 32):
        _check_route(_tda().route_experts(x.cuda(), k), x, k, True)
        _check_route(_tda().route_experts(x.cuda(), k, normalize=False), x, k, False)


def test_routes_of_no_tokens_and_strided_logits():
    tda = _tda()
    x = torch.randn(50, 70, generator=H.gen(3))
    r = tda.route_experts(x[:0].cuda(), 2)
    assert r.offsets.tolist() == [0] * 71 and r.rows.numel() == 0 and r.place.shape == (0, 2)
    wide = x.cuda()
    _check_route(tda.route_experts(wide[:, 3:67], 4), x[:, 3:67], 4, True)
    again = tda.route_experts(wide[:, 3:67], 4)
    out = tda.route_experts(wide[:, :64], 4, out=again)
    assert out is again
    _check_route(out, x[:, :64], 4, True)


# ---------------------------------------------------------------- silu_mul_fp8

@pytest.mark.parametrize("N,d,group", [(1, 128, 128), (3, 64, 128), (5, 1, 0), (7, 100, 0), (2, 129, 128), (9, 1000, 128), (61, 3584, 0), (300, 1024, 128),
                                       (17, 640, 64), (33, 512, 32), (4, 2048, 256), (6, 48, 8), (5, 8192, 0), (3, 20000, 0), (8, 777, 100), (1025, 256, 128)])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_silu(N, d, group, dtype):
    x = (torch.randn(N, 2 * d, generator=H.gen(N + d)) * 2).to(H.DT[dtype])
    out, s = _tda().silu_mul_fp8(x.cuda(), group=group)
    assert out.dtype == F8 and s.shape == (N, -(-d // group) if group else 1)
    H.check_silu(out, s, x, group)


@pytest.mark.parametrize("group", [0, 128])
@pytest.mark.parametrize("at,more", [(0, 8), (8, 0), (1, 4), (0, 3)])
def test_silu_of_strided_rows(group, at, more):
    N, d = 37, 384
    x = torch.randn(N, 2 * d + at + more, generator=H.gen(4)).to(torch.float16)
    out = torch.empty(N, d, dtype=F8, device="cuda")
    got = _tda().silu_mul_fp8(x.cuda()[:, at:at + 2 * d], group=group, out=out)
    assert got[0].data_ptr() == out.data_ptr()
    H.check_silu(out, got[1], x[:, at:at + 2 * d], group)


@pytest.mark.parametrize("group", [0, 128])
def test_silu_of_special_rows(group):
    """Zeros (scale 1), a NaN, infinities, gates far from 0, tiny numbers."""
    d = 256
    x = torch.randn(9, 2 * d, generator=H.gen(6)).to(torch.bfloat16)
    x[0] = 0
    x[1, 5] = math.nan
    x[2, d + 7] = math.nan
    x[3, 9] = math.inf
    x[4, :d] = -200.0
    x[5, :d] = 200.0
    x[6] = x[6] * 1e-18
    x[7, :d] *= 40
    out, s = _tda().silu_mul_fp8(x.cuda(), group=group)
    f = out.float().cpu()
    assert (f[0] == 0).all() and (s[0] == 1).all()
    for r, c in ((1, 5), (2, 7)):
        cut = slice(0, d) if group == 0 else slice(c // group * group, c // group * group + group)
        assert f[r, cut].isnan().all()
        if group:
            assert not f[r, group:].isnan().any() and s[r, 0].isnan() and not s[r, 1].isnan()
    assert f[3, 9].isnan() and s[3, 0].isinf()
    keep = [5, 6, 7, 8]
    H.check_silu(out[keep], s[keep], x[keep], group)
    # gates of -200: y is below 2^-140, or 0
    assert (f[4] * s[4].cpu().repeat_interleave(d // s.shape[1])).abs().max() < 1e-40


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("d,group,at", [(256, 128, 0), (256, 0, 0), (8200, 0, 0), (256, 128, 1), (256, 0, 1), (100, 0, 0)])
def test_silu_of_groups_near_zero(dtype, d, group, at):
    """Groups whose largest value is a few steps of the subnormal numbers, zeros among them, in each kernel.

    A scale that rounds to 0 is 1.  Another is off by half a step, 2^-150, so that 448 of it are short of the largest value by up to 224 steps,
    at which out is cut off; out is rounded by 2^-4 of itself, or by 2^-10 where it is small, and y by two steps.
    """
    steps = [1, 2, 5, 40, 100, 223, 224, 225, 230, 300, 448, 640, 672, 1000, 2000]
    wide = torch.zeros(len(steps), 2 * d + at + 7, dtype=H.DT[dtype])
    x = wide[:, at:at + 2 * d]
    for i, n in enumerate(steps):
        for c, part in ((3, 1.0), (90, -0.5)):
            # y: bfloat16 n 2^-149 exactly, float16 22 2^-149 times whole numbers
            x[i, c], x[i, d + c] = (2.0 ** -100, part * n * 2.0 ** -48) if dtype == "bf16" else (-88.0, -part * max(1, round(n / 22)) * 2.0 ** -24)
    if group:
        x[:, group + 5], x[:, d + group + 5] = 2.0, 3.0
    view = wide.cuda()[:, at:at + 2 * d]
    out, s = _tda().silu_mul_fp8(view, group=group)
    f, s = out.double().cpu(), s.double().cpu()
    y = H.silu_mul(x)
    first = slice(0, group or d)
    top = y[:, first].abs().amax(1)
    assert f.isfinite().all() and (f[y == 0] == 0).all() and s.isfinite().all() and (s > 0).all()
    step = 2.0 ** -149
    sure = top < 223 * step                    # (y itself may be off by a step)
    assert (s[sure, 0] == 1).all() and sure.sum() > 3
    big = top > 226 * step
    assert ((s[big, 0] - top[big] / 448).abs() <= step * (0.5 + 1 / 448)).all() and big.sum() > 3
    off = (f * s[:, :1] - y)[:, first].abs()
    back = torch.where(s[:, :1] < 1, s[:, :1], 0.0)
    assert (off <= y[:, first].abs() * 2.0 ** -4 + back * 2.0 ** -10 + (224 + 2) * step).all()
    if group:
        assert (f[:, group + 5] == 448).all()


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("d,group", [(512, 128), (512, 0), (264, 32), (1024, 256), (9000, 0)])
def test_silu_is_the_same_wherever_a_row_lies(dtype, d, group):
    """Rows on 16 bytes and off them take other kernels: the same bits, gates below -8 and special values among them."""
    x = torch.randn(40, 2 * d, generator=H.gen(d)).to(H.DT[dtype])
    x[1, :d] *= 6
    x[2, :d:9] = -20.0
    x[3, 5], x[4, d + 5], x[5, 7], x[6, 7] = math.nan, math.nan, math.inf, -math.inf
    x[7, :d], x[8, d:], x[9] = -80.0, x[8, d:] * 1e-3, 0
    got = []
    for at in (0, 1, 3):
        wide = torch.zeros(40, 2 * d + 8, dtype=H.DT[dtype], device="cuda")
        wide[:, at:at + 2 * d] = x.cuda()
        got.append(_tda().silu_mul_fp8(wide[:, at:at + 2 * d], group=group))
    for out, s in got[1:]:
        assert torch.equal(s.view(torch.int32), got[0][1].view(torch.int32)) and torch.equal(out.view(torch.uint8), got[0][0].view(torch.uint8))
    H.check_silu(got[0][0][10:], got[0][1][10:], x[10:], group)


def test_empty_silu():
    x = torch.randn(4, 256, device="cuda").half()
    out, s = _tda().silu_mul_fp8(x[:0])
    assert out.shape == (0, 128) and s.shape == (0, 1)
    out, s = _tda().silu_mul_fp8(x[:, :0])
    assert out.shape == (4, 0) and (s == 1).all()


# ----------------------------------------------------------------- experts_sum

@pytest.mark.parametrize("T,k,d,R", [(1, 1, 8, 1), (1, 8, 4096, 8), (5, 4, 1000, 20), (3, 2, 7, 6), (64, 8, 1024, 512), (300, 6, 136, 1800), (9, 3, 33, 27), (7, 32, 256, 100),
                                     (1000, 2, 64, 50)])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_sums(T, k, d, R, dtype):
    g = H.gen(T + k + d)
    x = torch.randn(R, d, generator=g).to(H.DT[dtype])
    w = torch.rand(T, k, generator=g)
    place = torch.randint(0, R, (T, k), generator=g).int()
    H.check_weighted(_tda().experts_sum(x.cuda(), w.cuda(), place.cuda()), x, w, place)


@pytest.mark.parametrize("d", [64, 65])
def test_sums_without_some_rows(d):
    """Places outside x count as nothing, whatever their weight and whatever lies there."""
    g = H.gen(7)
    x = torch.randn(30, d, generator=g).to(torch.float16)
    w = torch.rand(20, 5, generator=g)
    place = torch.randint(0, 30, (20, 5), generator=g).int()
    place[3], place[4, 2], place[5, 0], place[6, 4] = -1, 30, 2 ** 31 - 1, -2 ** 31
    w[3], w[4, 2] = math.nan, math.inf
    wide = torch.full((32, d + 16), math.nan, dtype=torch.float16, device="cuda")
    wide[1:31, 8:8 + d] = x.cuda()
    room = torch.full((20, d + 8), 9.0, dtype=torch.float16, device="cuda")
    out = _tda().experts_sum(wide[1:31, 8:8 + d], w.cuda(), place.cuda(), out=room[:, 8:])
    H.check_weighted(out, x, w, place)
    assert (out[3] == 0).all() and (room[:, :8] == 9).all()


def test_empty_sums():
    tda = _tda()
    x = torch.randn(4, 16, device="cuda").half()
    w, p = torch.ones(3, 2, device="cuda"), torch.zeros(3, 2, dtype=torch.int32, device="cuda")
    assert tda.experts_sum(x, w[:0], p[:0]).shape == (0, 16)
    assert (tda.experts_sum(x[:0], w, p) == 0).all()
    assert (tda.experts_sum(x, w[:, :0], p[:, :0]) == 0).all()
    assert tda.experts_sum(x[:, :0], w, p).shape == (3, 0)


# -------------------------------------------------------------- as they are used

def _layer(tda, x8, xs, router, gu, gus, dn, dns, k):
    r = tda.route_experts(router, k)
    h = tda.experts_matmul_fp8(x8, xs, gu, gus, r.offsets, rows=r.rows)
    y8, ys = tda.silu_mul_fp8(h)
    y = tda.experts_matmul_fp8(y8, ys, dn, dns, r.offsets)
    return r, h, y8, ys, y, tda.experts_sum(y, r.weights, r.place)


def _layer_inputs(T, E, d, f, seed):
    g = H.gen(seed)
    x = torch.randn(T, d, generator=g).to(torch.bfloat16)
    gu, gus = H.eights(g, E, 2 * f, d), H.scales(g, E, -(-2 * f // 128), -(-d // 128), size=d ** -0.5 / 150)
    dn, dns = H.eights(g, E, d, f), H.scales(g, E, -(-d // 128), -(-f // 128), size=f ** -0.5 / 150)
    return x, torch.randn(T, E, generator=g), gu, gus, dn, dns


def _check_layer(got, x8, xs, router, gu, gus, dn, dns, k):
    """Each step against the definition on what the step before gave."""
    r, h, y8, ys, y, out = (t.cpu() if torch.is_tensor(t) else t for t in got)
    _check_route(r, router, k, True)
    o, rows = r.offsets.tolist(), r.rows.tolist()
    n = o[-1]
    _check_experts(h, x8.cpu(), xs.cpu(), gu, gus, o, rows)
    H.check_silu(y8[:n], ys[:n], h[:n], 128)
    _check_experts(y, y8, ys, dn, dns, o)
    H.check_weighted(out, y[:n], r.weights.cpu(), r.place.cpu())


@pytest.mark.parametrize("T,E,d,f,k", [(1, 8, 256, 128, 2), (5, 8, 512, 192, 4), (33, 16, 256, 256, 3), (150, 4, 384, 128, 2)])
@pytest.mark.parametrize("masked", [False, True])
def test_a_layer_with_experts(T, E, d, f, k, masked):
    tda = _tda()
    x, router, gu, gus, dn, dns = _layer_inputs(T, E, d, f, T + E)
    if masked:
        router[:, :E - 1] = -math.inf           # one expert for all, and less than k of them
        router[T // 2] = -math.inf              # and a token with none
    x8, xs, _ = tda.add_norm_fp8(x.cuda(), torch.ones(d, dtype=torch.bfloat16, device="cuda"), group=128)
    got = _layer(tda, x8, xs, router.cuda(), gu.cuda(), gus.cuda(), dn.cuda(), dns.cuda(), k)
    _check_layer(got, x8, xs, router, gu, gus, dn, dns, k)
    if masked:
        assert (got[-1][T // 2] == 0).all()
    torch.cuda.synchronize()
    tda.matmul_fp8_check()


def test_a_captured_layer_replays_with_new_inputs():
    """The chain in a graph: replayed with other inputs, on another stream, beside an eager run on a third."""
    tda = _tda()
    T, E, d, f, k = 9, 8, 256, 128, 2
    x, router, gu, gus, dn, dns = _layer_inputs(T, E, d, f, 1)
    weights = [t.cuda() for t in (gu, gus, dn, dns)]
    one = torch.ones(d, dtype=torch.bfloat16, device="cuda")
    xd, rd = x.cuda(), router.cuda()
    def step():
        x8, xs, _ = tda.add_norm_fp8(xd, one, group=128)
        return x8, xs, _layer(tda, x8, xs, rd, *weights, k)
    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        x8, xs, got = step()
    for seed in (2, 3, 4):
        x2, router2, *_ = _layer_inputs(T, E, d, f, seed)
        xd.copy_(x2)
        rd.copy_(router2)
        side, third = torch.cuda.Stream(), torch.cuda.Stream()
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            graph.replay()
        with torch.cuda.stream(third):
            e8, es, eager = step()
        torch.cuda.synchronize()
        _check_layer(got, x8, xs, router2, gu, gus, dn, dns, k)
        n = int(eager[0].offsets[-1])
        for a, b in zip(got[1:], eager[1:]):
            assert torch.equal(a[:n].float(), b[:n].float())


def test_a_stream_of_the_callers():
    """`stream=`: a torch stream and a raw handle; the call is enqueued there."""
    tda = _tda()
    x, xs, w, ws = _operands(1, 20, 256, 256)
    side = torch.cuda.Stream()
    dev = [t.cuda() for t in (x, xs, w, ws)]
    torch.cuda.synchronize()
    for s in (side, side.cuda_stream):
        out = tda.matmul_fp8(*dev, stream=s)
        side.synchronize()
        H.check_product(out, x, xs, w, ws)


def test_outputs_beside_their_inputs():
    """Columns of one buffer's rows are no overlap; columns that they share are one."""
    tda = _tda()
    x = torch.randn(30, 64, generator=H.gen(1)).to(torch.bfloat16)
    w, place = torch.rand(20, 3, generator=H.gen(2)), torch.randint(0, 30, (20, 3), generator=H.gen(3)).int()
    for at, first in ((0, 64), (64, 0), (72, 0), (0, 72), (72, 8)):
        room = torch.zeros(30, 136, dtype=torch.bfloat16, device="cuda")
        view = room[:, first:first + 64]
        view.copy_(x)
        out = room[4:24, at:at + 64]
        assert tda.experts_sum(view, w.cuda(), place.cuda(), out=out) is out
        H.check_weighted(out, x, w, place)
        assert torch.equal(view.cpu(), x)
        for a in (1, 63):
            near = room[4:24, abs(first - a):abs(first - a) + 64]
            with pytest.raises(ValueError, match="overlaps"):
                tda.experts_sum(view, w.cuda(), place.cuda(), out=near)
    wide = torch.zeros(40, 512, dtype=torch.uint8, device="cuda")
    x, xs, wt, ws = _operands(4, 40, 64, 256)
    x8 = wide[:, :256].view(F8)
    wide[:, :256].copy_(x.view(torch.uint8))
    out = wide[:, 256:384].view(torch.bfloat16)
    tda.matmul_fp8(x8, xs.cuda(), wt.cuda(), ws.cuda(), out=out)
    H.check_product(out, x, xs, wt, ws)


def test_refusals_on_the_gpu():
    tda = _tda()
    x, xs, w, ws = (t.cuda() for t in _operands(1, 4, 128, 256))
    o, h, f = _i32([0, 4]), torch.zeros(4, 8, device="cuda").half(), torch.zeros(4, 8, device="cuda")
    bad = [
        (lambda: tda.matmul_fp8(x.float(), xs, w, ws), "x: dtype"),
        (lambda: tda.matmul_fp8(x, xs.half(), w, ws), "x_scales: dtype"),
        (lambda: tda.matmul_fp8(x, xs[:3], w, ws), "x_scales: shape"),
        (lambda: tda.matmul_fp8(x, xs.repeat(1, 2), w, ws), "x_scales: shape"),
        (lambda: tda.matmul_fp8(x, xs, w[:, :128], ws), "weight: 128 channels"),
        (lambda: tda.matmul_fp8(x, xs, w, ws[:, :1]), "weight_scales"),
        (lambda: tda.matmul_fp8(x, xs, w[None], ws), "weight: 3 dimensions"),
        (lambda: tda.matmul_fp8(x.T, xs, w, ws), "last dimension"),
        (lambda: tda.matmul_fp8(x, xs, w, ws, dtype=torch.float32), "neither"),
        (lambda: tda.matmul_fp8(x, xs, w, ws, dtype=1), "not a torch.dtype"),
        (lambda: tda.matmul_fp8(x, xs, w, ws, out=h), "out: shape"),
        (lambda: tda.matmul_fp8(x, xs, w, ws, out=torch.zeros(4, 128, device="cuda")), "neither"),
        (lambda: tda.matmul_fp8(x, xs, w, ws, dtype=torch.bfloat16, out=torch.zeros(4, 128, device="cuda").half()), "out: dtype"),
        (lambda: tda.matmul_fp8(x, xs, w, ws, out=x.view(torch.bfloat16)), "overlaps an input"),
        (lambda: tda.matmul_fp8(x, xs, w, ws, out=torch.zeros(1, 128, device="cuda").half().expand(4, -1)), "overlap"),
        (lambda: tda.experts_matmul_fp8(x, xs, w, ws, o), "weight: 2 dimensions"),
        (lambda: tda.experts_matmul_fp8(x, xs, w[None], ws[None], _i32([0, 2, 4])), "offsets: shape"),
        (lambda: tda.experts_matmul_fp8(x, xs, w[None], ws[None], o.long()), "offsets: dtype"),
        (lambda: tda.experts_matmul_fp8(x, xs, w[None], ws[None], o, rows=o.long()), "rows: dtype"),
        (lambda: tda.experts_matmul_fp8(x, xs, w[:0, None], ws[:0, None], o[:1]), "channels|experts|shape"),
        (lambda: tda.experts_matmul_fp8(x, xs, w[None], ws[None], o.cpu()), "not a CUDA tensor"),
        (lambda: tda.route_experts(f, 0), "k: 0"),
        (lambda: tda.route_experts(f, 9), "k: 9"),
        (lambda: tda.route_experts(f.double(), 2), "none of"),
        (lambda: tda.route_experts(f[:, :0], 1), "no experts"),
        (lambda: tda.route_experts(f, 2, out=tda.route_experts(f[:3], 2)), "out.weights: shape"),
        (lambda: tda.silu_mul_fp8(h[:, :7]), "7 channels"),
        (lambda: tda.silu_mul_fp8(f), "neither"),
        (lambda: tda.silu_mul_fp8(h, group=-1), "group"),
        (lambda: tda.silu_mul_fp8(h, out=torch.zeros(4, 5, device="cuda").to(F8)), "out: shape"),
        (lambda: tda.silu_mul_fp8(h, scales=f), "scales: shape"),
        (lambda: tda.experts_sum(h, f, o), "place"),
        (lambda: tda.experts_sum(h, f, torch.zeros(4, 7, device="cuda").int()), "place: shape"),
        (lambda: tda.experts_sum(h, f, torch.zeros(4, 8, device="cuda").int(), out=h), "overlaps"),
    ]
    for call, msg in bad:
        with pytest.raises(ValueError, match=msg):
            call()
    with pytest.raises(tda.ArError):
        tda.route_experts(torch.zeros(2, 1025, device="cuda"), 2)
    with pytest.raises(tda.ArError):
        tda.route_experts(torch.zeros(2, 64, device="cuda"), 33)
