"""Corners of the operators of include/ar_ops.h on the GPU: values, streams, captures and rows at the edge of what
each is specified for, against the same 64-bit implementations as test_gpu_ops.py."""
import math

import numpy as np
import pytest
import torch

from tests import ops_helpers as H
from tests.test_gpu_ops import _attend_case, _check_attend, _check_norm, _gen, _i32, _tda

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__
    __graft_entry__.build()


# ---------------------------------------------------------------- attention

@pytest.mark.parametrize("window,sinks", [(0, 0), (20, 2)])
def test_attend_many_segments_to_a_warp(window, sinks):
    """8192 short requests: every warp walks through several segments, whole ones and parts.  The requests repeat 64
    different ones (page ids may), so that the plain implementation need not run 8192 times."""
    tda = _tda()
    kinds, B, D = 64, 8192, 64
    g = np.random.RandomState(3)
    lens = [int(x) for x in g.randint(1, 150, kinds)]
    q, pool, K, V, table, cu = _attend_case(47, kinds, lens, [1] * kinds, 2, 4, D, 16, "bf16")
    want, wl, mag, big, top = H.attend(q, K, V, table, lens, cu, window, sinks, D ** -0.5)
    bo, bl = H.attend_bounds(want, wl, mag, big, top, D ** -0.5, q.dtype, max(lens))
    pick = torch.from_numpy(g.randint(0, kinds, B))
    out, lse = tda.kv4_attend(q[pick].cuda(), pool.cuda(), _i32(table)[pick.cuda()], _i32(lens)[pick.cuda()], window=window,
                              sinks=sinks, return_lse=True)
    assert ((out.cpu().double() - want[pick]).abs() <= bo[pick]).all()
    assert ((lse.cpu().double() - wl[pick]).abs() <= bl[pick]).all()


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("D,G,max_new", [(128, 8, 1), (64, 4, 1), (256, 8, 1), (128, 8, 2), (64, 8, 2)])
@pytest.mark.parametrize("inf", [math.inf, -math.inf])
def test_attend_infinity_in_k_is_nan(dtype, D, G, max_new, inf):
    """An infinity that kv4_append met in K reads back as NaN (0 x inf), so every row that sees its token is NaN,
    whatever shape the call takes, and no other row changes."""
    tda = _tda()
    B, n, page = 48, 40, 16
    q, pool, K, V, table, cu = _attend_case(53, B, [n] * B, [1] * B, 1, G, D, page, dtype)
    pd, args = pool.cuda(), (_i32(table), _i32([n] * B), _i32(cu))
    clean = tda.kv4_attend(q.cuda(), pd, *args, max_new=max_new, return_lse=True)
    k = torch.randn(B // 2, 1, D, generator=_gen(54)).to(H.DT[dtype])
    for b in range(B // 2):
        k[b, 0, (7 * b) % D] = inf
    slots = torch.tensor([table[b][(b + 3) % n // page] * page + (b + 3) % n % page for b in range(B // 2)])
    tda.kv4_append(k.cuda(), k.nan_to_num(0, 0, 0).cuda(), pd, slots.cuda())
    out, lse = tda.kv4_attend(q.cuda(), pd, *args, max_new=max_new, return_lse=True)
    assert out[:B // 2].isnan().all() and lse[:B // 2].isnan().all()
    assert torch.equal(out[B // 2:], clean[0][B // 2:]) and torch.equal(lse[B // 2:], clean[1][B // 2:])


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("D,G,max_new", [(128, 8, 1), (64, 4, 1), (256, 8, 1), (128, 8, 2)])
def test_attend_large_channels_in_k(dtype, D, G, max_new):
    """One large channel to each group of K, as trained caches have: most nibbles are 0 and sum |q k| small beside
    sum |q|, and the queries have an offset; the bounds on the scores' sums (of |q k|) hold all the same."""
    tda = _tda()
    lens, page = [300, 77, 1, 64], 16
    q, pool, K, V, table, cu = _attend_case(59, 4, lens, [1] * 4, 2, G, D, page, dtype)
    kn, ks, vn, vs = H.unpack(pool)
    small = kn.sign() * (kn.abs() == 7)
    large = torch.zeros(D)
    large[5::32] = 7
    kn = torch.where(large > 0, large * kn.sign(), small)
    pool = H.pack(kn, ks[..., ::32].to(torch.bfloat16), vn, vs[..., ::32].to(torch.bfloat16))
    K = (kn * ks).reshape(K.shape)
    q = q.float() + 3
    q[..., 5::32] *= 2.0 ** -12
    q = q.to(H.DT[dtype])
    out, lse = tda.kv4_attend(q.cuda(), pool.cuda(), _i32(table), _i32(lens), max_new=max_new, return_lse=True)
    _check_attend(q, K, V, table, lens, cu, 0, 0, D ** -0.5, out, lse)


@pytest.mark.parametrize("D,G,max_new", [(128, 8, 1), (64, 8, 2), (256, 4, 1)])
@pytest.mark.parametrize("small", [10, 18, 26])
def test_attend_small_channels_beside_large_ones(D, G, max_new, small):
    """Groups of V at 2^-small of the others: a weight is off by 2^-11 of itself, or by 2^-33 of the largest scale where
    it is small, so a channel by n x 7 of those at most, beside what the other bounds allow."""
    tda = _tda()
    lens, page = [400, 33, 3000], 16
    q, pool, K, V, table, cu = _attend_case(89, 3, lens, [1] * 3, 1, G, D, page, "f16")
    kn, ks, vn, vs = H.unpack(pool)
    vs[..., 32:64] *= 2.0 ** -small
    pool = H.pack(kn, ks[..., ::32].to(torch.bfloat16), vn, vs[..., ::32].to(torch.bfloat16))
    V = (vn * vs).reshape(V.shape)
    out, lse = tda.kv4_attend(q.cuda(), pool.cuda(), _i32(table), _i32(lens), max_new=max_new, return_lse=True)
    want, wl, mag, big, _ = H.attend(q, K, V, table, lens, cu, 0, 0, D ** -0.5)
    none = torch.zeros(want.shape[:2], dtype=torch.float64)
    bound = H.attend_bounds(want, wl, mag, big, none, D ** -0.5, q.dtype, max(lens))[0]
    bound += torch.tensor(lens).view(-1, 1, 1) * 7 * 2.0 ** -33 * vs.max()
    assert ((out.cpu().double() - want).abs() <= bound).all()


@pytest.mark.parametrize("n,new,max_new", [(64, 1, 1), (50, 1, 1), (64, 1, 2), (50, 3, 3)])
def test_attend_nan_in_v_under_a_vanishing_weight(n, new, max_new):
    """A token whose weight is below binary32's smallest number still has its NaN seen, in a tile that some rows see
    in part as in a whole one."""
    tda = _tda()
    D, page = 128, 16
    q, pool, K, V, table, cu = _attend_case(67, 1, [n], [new], 1, 8, D, page, "f16")
    kn, ks, vn, vs = H.unpack(pool)
    q[:] = 1
    pid = table[0][0]
    kn[pid, 0, 0, 3], ks[pid, 0, 0, 3] = -7, 8.0      # a score of -7 x 8 x sqrt(128), -634
    vs[pid, 0, 0, 3, 64:96] = math.nan
    pool = H.pack(kn, ks[..., ::32].to(torch.bfloat16), vn, vs[..., ::32].to(torch.bfloat16))
    out = tda.kv4_attend(q.cuda(), pool.cuda(), _i32(table), _i32([n]), _i32(cu), max_new=max_new)
    assert out[:, :, 64:96].isnan().all()
    assert not out[:, :, :64].isnan().any() and not out[:, :, 96:].isnan().any()


@pytest.mark.parametrize("D,G,max_new", [(128, 8, 1), (64, 8, 3)])
def test_attend_leaves_rows_of_no_request_alone(D, G, max_new):
    """Two calls that share q, out and lse, each over its part of the requests, with rows of padding behind both;
    and a call after a refused plan, whose cu is all 0."""
    tda = _tda()
    lens, new, page = [70, 1, 333, 40], [3, 1, 2, 1], 16
    q, pool, K, V, table, cu = _attend_case(83, 4, lens, new, 2, G, D, page, "bf16")
    pad = 5
    qd = torch.cat((q, torch.full((pad, *q.shape[1:]), math.nan, dtype=q.dtype))).cuda()
    out, lse = torch.full_like(qd, 5.0), torch.full(qd.shape[:2], 5.0, device="cuda")
    pd, td, ld, cd = pool.cuda(), _i32(table), _i32(lens), _i32(cu)
    tda.kv4_attend(qd, pd, td, ld, torch.zeros_like(cd), max_new=max_new, out=out, lse=lse)
    assert (out == 5).all() and (lse == 5).all()
    tda.kv4_attend(qd, pd, td[2:], ld[2:], cd[2:], max_new=max_new, out=out, lse=lse)
    assert (out[:4] == 5).all() and (lse[:4] == 5).all()
    tda.kv4_attend(qd, pd, td[:2], ld[:2], cd[:3], max_new=max_new, out=out, lse=lse)
    assert (out[-pad:] == 5).all() and (lse[-pad:] == 5).all()
    _check_attend(q, K, V, table, lens, cu, 0, 0, D ** -0.5, out[:-pad], lse[:-pad])
    tda.kv4_workspace().check()


@pytest.mark.parametrize("D,G,max_new", [(128, 8, 1), (64, 8, 2), (256, 4, 1)])
@pytest.mark.parametrize("n", [200, 20011])
@pytest.mark.parametrize("small,large", [(0.0, 2.0 ** 13), (2.0 ** -60, 2.0 ** 20), (0.0, 2.0 ** 60), (2.0 ** -90, 2.0 ** 90)])
def test_attend_v_of_zeros_before_large_v(D, G, max_new, n, small, large):
    """Early tokens with V far below the later ones' keep their weights in the sum, also where the parts are joined."""
    tda = _tda()
    page = 64
    q, pool, K, V, table, cu = _attend_case(97, 1, [n], [1], 1, G, D, page, "bf16")
    kn, ks, vn, vs = H.unpack(pool)
    tok = torch.zeros(pool.shape[0], page, dtype=torch.float64)
    for i, pid in enumerate(table[0][:-(-n // page)]):
        tok[pid] = torch.arange(page) + i * page
    size = torch.where(tok < n // 2 + 5, small, large).view(pool.shape[0], 1, page // 16, 16, 1)
    vs = vs * size
    pool = H.pack(kn, ks[..., ::32].to(torch.bfloat16), vn, vs[..., ::32].to(torch.bfloat16))
    kn, ks, vn, vs = H.unpack(pool)
    V = (vn * vs).reshape(V.shape)
    out, lse = tda.kv4_attend(q.cuda(), pool.cuda(), _i32(table), _i32([n]), max_new=max_new, return_lse=True)
    _check_attend(q, K, V, table, [n], cu, 0, 0, D ** -0.5, out, lse)


# --------------------------------------------------------------- workspaces

def test_a_workspace_is_ready_on_every_stream():
    """Its zeros are written on the current stream, and a call on another one need not wait for that."""
    torch.cuda._sleep(200_000_000)
    _tda().Kv4Workspace()
    assert torch.cuda.current_stream().query()


def _small_call(B=2):
    q, pool, K, V, table, cu = _attend_case(61, B, [20] * B, [1] * B, 1, 8, 64, 16, "bf16")
    return q.cuda(), pool.cuda(), _i32(table), _i32([20] * B)


@pytest.mark.parametrize("warm", [True, False])
def test_captured_calls_keep_to_their_own_workspace(warm):
    """Whether or not the stream ran calls before its capture: what a replay records is in the workspace that
    kv4_workspace gave inside the capture, which kv4_workspaces lists, and in no stream's own."""
    tda = _tda()
    s = torch.cuda.Stream()
    q, pool, table, lens = _small_call()
    tda.kv4_attend(q, pool, table, lens)
    if warm:
        tda.kv4_attend(q, pool, table, lens, stream=s)
    table = table.clone()
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.stream(s), torch.cuda.graph(graph, stream=s):
        tda.kv4_attend(q, pool, table, lens)
        used = tda.kv4_workspace()
    own = [tda.kv4_workspace(), tda.kv4_workspace(stream=s)]
    every = tda.kv4_workspaces()
    assert used not in own and used in every and all(w in every for w in own)
    table[0, 0] = pool.shape[0]
    try:
        graph.replay()
        torch.cuda.synchronize()
        assert used.status() == tda.ar.AR_EINVAL
        assert [w.status() for w in own] == [0, 0]
    finally:
        tda.ops._ops().ar_kv4_workspace_init(used.ptr, None)
        torch.cuda.synchronize()


@pytest.mark.parametrize("warm", [True, False])
def test_a_graph_with_parallel_branches(warm):
    """Two streams of one capture attend at the same time, over long requests whose parts are joined."""
    tda = _tda()
    main, side = torch.cuda.Stream(), torch.cuda.Stream()
    cases = []
    for seed, n, G in ((71, 9001, 8), (73, 7003, 4)):
        q, pool, K, V, table, cu = _attend_case(seed, 2, [n, 333], [1, 1], 2, G, 128, 64, "bf16")
        cases.append((q.cuda(), pool.cuda(), _i32(table), _i32([n, 333])))
    want = [tda.kv4_attend(*c) for c in cases]
    if warm:
        for s, c in zip((main, side), cases):
            tda.kv4_attend(*c, stream=s)
    torch.cuda.synchronize()
    graph, got = torch.cuda.CUDAGraph(), [[], []]
    with torch.cuda.stream(main), torch.cuda.graph(graph, stream=main):
        side.wait_stream(main)
        for _ in range(10):
            with torch.cuda.stream(side):
                got[1].append(tda.kv4_attend(*cases[1]))
            got[0].append(tda.kv4_attend(*cases[0]))
        with torch.cuda.stream(side):
            second = tda.kv4_workspace()
        assert tda.kv4_workspace() is not second
        main.wait_stream(side)
    for _ in range(5):
        graph.replay()
        torch.cuda.synchronize()
        for g, w in zip(got, want):
            assert all(torch.equal(x, w) for x in g)
            for x in g:
                x.zero_()


def test_replays_beside_calls_on_the_captured_stream():
    """The usual warm-up, then a capture on the same stream: replays on another stream overlap with its calls."""
    tda = _tda()
    s, other = torch.cuda.Stream(), torch.cuda.Stream()
    q, pool, K, V, table, cu = _attend_case(79, 2, [9001, 333], [1, 1], 2, 8, 128, 64, "bf16")
    args = q.cuda(), pool.cuda(), _i32(table), _i32([9001, 333])
    want = tda.kv4_attend(*args, stream=s)
    graph, got = torch.cuda.CUDAGraph(), []
    torch.cuda.synchronize()
    with torch.cuda.stream(s), torch.cuda.graph(graph, stream=s):
        for _ in range(20):
            got.append(tda.kv4_attend(*args))
    torch.cuda.synchronize()
    with torch.cuda.stream(other):
        graph.replay()
    got += [tda.kv4_attend(*args, stream=s) for _ in range(20)]
    torch.cuda.synchronize()
    assert all(torch.equal(x, want) for x in got)


def test_a_capture_of_more_streams_than_workspaces_is_refused(monkeypatch):
    tda = _tda()
    args = _small_call()
    tda.kv4_attend(*args)
    dev = torch.cuda.current_device()
    monkeypatch.setitem(tda.ops._captured, dev, tda.ops._captured[dev][:2])
    main, *sides = [torch.cuda.Stream() for _ in range(4)]
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.stream(main), torch.cuda.graph(graph, stream=main):
        for s in sides:
            s.wait_stream(main)
        with pytest.raises(RuntimeError, match="captured on more streams"):
            for s in sides:
                tda.kv4_attend(*args, stream=s)
        for s in sides:
            main.wait_stream(s)


@pytest.mark.parametrize("device", ["cuda", torch.device("cuda"), "cuda:0", 0])
def test_workspaces_by_the_name_of_their_device(device):
    tda = _tda()
    ws = tda.Kv4Workspace(device)
    assert ws.buffer.device == torch.device("cuda", 0) and ws.device == 0 and ws.status() == 0
    args = _small_call()
    assert torch.equal(tda.kv4_attend(*args, workspace=ws), tda.kv4_attend(*args))
    assert tda.kv4_workspace(device) is tda.kv4_workspace() and tda.kv4_workspaces(device) == tda.kv4_workspaces()


# --------------------------------------------------------------------- plan

@pytest.mark.parametrize("how", ["stream=", "current", "handle", "out"])
def test_plan_check_waits_for_the_stream_of_the_plan(how):
    """A refused plan on a busy stream that is not the current one when its check is called."""
    tda = _tda()
    s = torch.cuda.Stream()
    lens, new, table, free, used = _i32([3]), _i32([40]), _i32([[5, -1]]), _i32([7, 8]), _i32([0])
    args, kw = (lens, new, table, free, used), dict(page=16, max_tokens=64)
    out = None
    if how == "out":
        out = tda.kv_plan(lens, _i32([1]), table, free, used, **kw)
        out.check()
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        torch.cuda._sleep(200_000_000)
    if how == "current":
        with torch.cuda.stream(s):
            plan = tda.kv_plan(*args, **kw)
    else:
        plan = tda.kv_plan(*args, **kw, out=out, stream=s.cuda_stream if how == "handle" else s)
    plan = plan._replace(lens=plan.lens)
    with pytest.raises(tda.ArError) as e:
        plan.check()
    assert e.value.code == tda.ar.AR_ETOOBIG
    assert isinstance(plan, tuple) and len(plan) == 7 and plan._fields[0] == "lens"


# --------------------------------------------------------------------- norm

def _shifted(x, shift):
    """x on the GPU, its rows `shift` elements off 16 bytes (each shift takes another kernel)."""
    room = torch.zeros(x.shape[0], x.shape[1] + 8, dtype=x.dtype, device="cuda")
    view = room[:, shift:shift + x.shape[1]]
    view.copy_(x)
    return view


@pytest.mark.parametrize("shift", [0, 1])
@pytest.mark.parametrize("group", [0, 128])
def test_norm_of_rows_whose_squares_overflow(group, shift):
    """An infinity in the row, or finite values whose squares pass binary32: y is 0 (scale 1) wherever h is finite, and
    NaN in the infinity's group."""
    d = 1024
    x = torch.randn(4, d, generator=_gen(1)).to(torch.bfloat16)
    x[0, 9], x[1, 9], x[2, 9] = math.inf, -math.inf, 1e20
    out, scales, _ = _tda().add_norm_fp8(_shifted(x, shift), torch.ones(d, dtype=torch.bfloat16, device="cuda"), group=group)
    f = out.float().cpu()
    assert (f[2] == 0).all() and (scales[2] == 1).all()
    assert f[:2, :group or d].isnan().all() and scales[:2, 0].isnan().all()
    assert (f[:2, group or d:] == 0).all() and (scales[:2, 1:] == 1).all()
    _check_norm(x[3:], None, torch.ones(d, dtype=torch.bfloat16), 1e-6, group, out[3:], scales[3:], None)


@pytest.mark.parametrize("shift", [0, 1])
@pytest.mark.parametrize("group", [0, 128])
@pytest.mark.parametrize("d", [1024, 6144])
def test_norm_with_a_nan_in_the_weight(d, group, shift):
    """It spoils the scale and output of its own group, in every row, whichever kernel the rows take."""
    x = torch.randn(3, d, generator=_gen(1)).to(torch.bfloat16)
    w = torch.ones(d, dtype=torch.bfloat16)
    w[d // 2 + 3] = math.nan
    out, scales, _ = _tda().add_norm_fp8(_shifted(x, shift), w.cuda(), group=group)
    n = group or d
    bad = torch.arange(d) // n == (d // 2 + 3) // n
    f = out.float().cpu()
    assert f[:, bad].isnan().all() and not f[:, ~bad].isnan().any()
    assert torch.equal(scales.cpu().isnan(), bad.view(1, -1, n)[..., 0].expand(3, -1))


@pytest.mark.parametrize("shift", [0, 1])
@pytest.mark.parametrize("group", [0, 128])
def test_norm_of_groups_near_zero(group, shift):
    """Groups whose largest |y| is a few steps of the subnormal numbers, or whose scale has no finite reciprocal, zeros among them.

    A scale that rounds to 0 is 1.  Another is off by half a step, 2^-150 (and 2^-20 for the root and products), so that 448 of it are short of the
    largest |y| by up to 224 steps, at which out is cut off; out is rounded by 2^-4 of itself, or by 2^-10 where it is small, and y by two steps.
    """
    d, step = 256, 2.0 ** -149
    steps = [1, 2, 5, 40, 100, 222, 224, 228, 230, 300, 448, 640, 672, 1000, 2000, 2.0 ** 17, 2.0 ** 22, 2.0 ** 26, 2.0 ** 31, 2.0 ** 47]
    x = torch.zeros(len(steps), d, dtype=torch.bfloat16)
    w = torch.ones(d, dtype=torch.bfloat16)
    x[:, 200] = 2.0 ** 57                      # the root of the mean is 2^53
    for i, n in enumerate(steps):
        x[i, 3], x[i, 90], x[i, 91] = n * 2.0 ** -96, -n * 2.0 ** -97, n * 2.0 ** -107
    if not group:
        w[200] = 0
    out, scales, _ = _tda().add_norm_fp8(_shifted(x, shift), w.cuda(), eps=0.0, group=group)
    f, s = out.double().cpu(), scales.double().cpu()[:, :1]
    xd = x.double()
    y = xd / (xd * xd).mean(1, keepdim=True).sqrt() * w.double()
    first = slice(0, group or d)
    top = y[:, first].abs().amax(1)
    assert f.isfinite().all() and (f[y == 0] == 0).all() and scales.isfinite().all() and (scales > 0).all()
    sure, big = top < 223 * step, top > 227 * step
    assert sure.sum() > 3 and (s[sure] == 1).all()
    assert ((s[big, 0] - top[big] / 448).abs() <= step * (0.5 + 1 / 448) + top[big] / 448 * 2.0 ** -20).all()
    off, mag = (f * s - y)[:, first].abs(), y[:, first].abs()
    back = torch.where(s < 1, s, 0.0)
    assert (off <= mag * (2.0 ** -4 + 2.0 ** -19) + back * 2.0 ** -10 + (224 + 2) * step).all()
    if group:
        assert (f[:, 200] == 448).all()


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_norm_of_rows_without_channels(dtype):
    """Their scale is 1, as of any row whose largest |y| is 0; it is written."""
    x = torch.empty(5, 0, dtype=H.DT[dtype], device="cuda")
    scales = torch.full((5, 1), 7.0, device="cuda")
    out, same, _ = _tda().add_norm_fp8(x, x[0], scales=scales)
    assert same is scales and (scales == 1).all() and out.shape == (5, 0)


@pytest.mark.parametrize("shape", [(0, 64), (5, 0), (0, 0)])
def test_norm_of_nothing_with_a_residual(shape):
    """An empty step gives empty tensors, the sum with the residual among them."""
    x = torch.empty(shape, dtype=torch.bfloat16, device="cuda")
    w = torch.ones(shape[1], dtype=torch.bfloat16, device="cuda")
    out, scales, h = _tda().add_norm_fp8(x, w, residual=x)
    assert out.shape == h.shape == shape and h.dtype == x.dtype and scales.shape == (shape[0], 1)


def test_norm_with_a_weight_from_the_call_before():
    """A weight that the call before writes, again and again at the same place, in one row after another's reads."""
    tda = _tda()
    d = 2048
    g = _gen(5)
    x = torch.randn(300, d, generator=g).to(torch.bfloat16).cuda()
    ws = [(1 + 0.2 * torch.randn(1, d, generator=g)).to(torch.bfloat16).cuda() for _ in range(40)]
    want = [tda.add_norm_fp8(x, w[0])[0].view(torch.uint8) for w in ws]
    zero, weight = torch.zeros(1, d, dtype=torch.bfloat16, device="cuda"), torch.zeros(1, d, dtype=torch.bfloat16, device="cuda")
    torch.cuda.synchronize()
    got = []
    for w in ws:
        tda.add_norm_fp8(w, w[0], residual=zero, residual_out=weight)
        got.append(tda.add_norm_fp8(x, weight[0])[0])
    assert all(torch.equal(a.view(torch.uint8), b) for a, b in zip(got, want))


# -------------------------------------------------------------------- cache

@pytest.mark.parametrize("D", [64, 128, 256])
def test_append_of_groups_whose_scale_rounds_to_zero(D):
    """max|x| / 7 of bfloat16 values below 4 x 2^-133 is no bfloat16 number but 0: n = 0, not a quotient by 0."""
    tda = _tda()
    rows = torch.zeros(5, 1, D, dtype=torch.bfloat16)
    for i in range(5):
        rows[i, 0, ::3], rows[i, 0, 1::3] = 2.0 ** -133 * i, -(2.0 ** -133) * i
    pool = torch.full((1, 1, 1, 18 * D), 0xa5, dtype=torch.uint8, device="cuda")
    slots = torch.arange(5, device="cuda")
    tda.kv4_append(rows.cuda(), rows.flip(0).cuda(), pool, slots)
    kn, ks, vn, vs = (x[0, 0, 0, :5] for x in H.unpack(pool.cpu()))
    assert (kn[:4] == 0).all() and (ks[:4] == 0).all() and (vn[1:] == 0).all() and (vs[1:] == 0).all()
    # 4 x 2^-133 / 7 rounds to 2^-133, and x / scale is 4
    want = rows[4, 0].double() * 2.0 ** 133
    assert (ks[4] == 2.0 ** -133).all() and torch.equal(kn[4], want) and torch.equal(vn[0], want)
    k, v = tda.kv4_load(pool, slots)
    assert (k[:4] == 0).all() and torch.equal(k[4], rows[4].cuda()) and torch.equal(v[0], rows[4].cuda())


# ----------------------------------------------------------------- refusals

def test_written_tensors_whose_elements_overlap_are_refused():
    """As everywhere in torch; read ones may be expanded."""
    tda = _tda()
    q, pool, table, lens = _small_call()
    x = torch.ones(4, 64, dtype=torch.bfloat16, device="cuda")
    slots = torch.arange(2, device="cuda")
    k, v = tda.kv4_load(pool, slots)
    bad = [lambda: tda.add_norm_fp8(x, x[0], residual_out=x[:1].expand(4, 64)),
           lambda: tda.kv4_attend(q, pool, table, lens, out=torch.zeros_like(q[:1]).expand_as(q)),
           lambda: tda.kv4_load(pool, slots, out=(k[:1].expand_as(k), v)),
           lambda: tda.kv4_load(pool, slots, out=(k, v[:1].expand_as(v)))]
    for f in bad:
        with pytest.raises(ValueError, match="out: its elements overlap"):
            f()
    same = tda.add_norm_fp8(x, x[0], residual=x[:1].expand(4, 64))
    assert (same[2] == 2).all()
    tda.kv4_append(k[:1].expand_as(k), v[:1].expand_as(v), pool, slots)
    again = tda.kv4_load(pool, slots)
    assert torch.equal(again[0][1], again[0][0]) and torch.equal(again[1][1], again[1][0])


def test_nothing_has_a_gradient():
    """Tensors that require one (a module's parameters) are data, in grad mode too; the same bits come out."""
    tda = _tda()
    q, pool, table, lens = _small_call()
    x, w = torch.randn(4, 64, device="cuda").to(torch.bfloat16), torch.nn.Parameter(torch.ones(64, dtype=torch.bfloat16, device="cuda"))
    with torch.enable_grad():
        got = tda.add_norm_fp8(x, w, residual=x.clone().requires_grad_())
        out = tda.kv4_attend(q.clone().requires_grad_(), pool, table, lens)
    want = tda.add_norm_fp8(x, w.detach(), residual=x)
    assert all(not t.requires_grad for t in (*got, out))
    assert torch.equal(got[0].view(torch.uint8), want[0].view(torch.uint8)) and torch.equal(out, tda.kv4_attend(q, pool, table, lens))
