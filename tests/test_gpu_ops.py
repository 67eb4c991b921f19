"""The operators of include/ar_ops.h on the GPU against plain implementations in
64 bits (tests/ops_helpers.py), whose bounds come from what each kernel rounds."""
import math

import numpy as np
import pytest
import torch

from tests import ops_helpers as H

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__
    __graft_entry__.build()


def _tda():
    import tensor_decode_all_gb300 as tda
    return tda


def _gen(seed):
    return torch.Generator().manual_seed(seed)


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


# --------------------------------------------------------------------- plan

def _plan_case(lens, new, page, width, free, used, cap, seed=0):
    g = np.random.RandomState(seed)
    table = [[int(g.randint(0, 1000)) if i * page < n else -1 for i in range(width)] for n in lens]
    dev = dict(lens=_i32(lens), new=_i32(new), table=_i32(table).view(len(lens), width), free=_i32(free), used=_i32([used]))
    code, want = H.plan(lens, new, table, free, used, page, cap)
    return dev, code, want, table


def _plan_same(p, want, table, dev, what=""):
    for name in ("lens", "cu", "slots", "request", "position", "free_used", "status"):
        assert getattr(p, name).tolist() == want[name], (what, name)
    assert dev["table"].tolist() == table, what


@pytest.mark.parametrize("B,page,new,cap_over", [
    (1, 16, [1], 0), (1, 16, [0], 3), (5, 16, [1, 0, 17, 16, 33], 5), (64, 32, [1], 0), (1000, 16, [1, 1, 40], 7),
    (1025, 64, [1, 0, 2], 100), (3, 16, [5000, 1, 2], 1), (8192, 16, [1], 0)])
def test_plan(B, page, new, cap_over):
    g = np.random.RandomState(B)
    lens = [int(x) for x in g.randint(0, 200, B)]
    lens[0] = 0 if B > 2 else 32
    new = [new[i % len(new)] for i in range(B)]
    width = -(-(200 + max(new)) // page)
    free = [int(x) for x in g.permutation(B * width + 9) + 5000]
    dev, code, want, table = _plan_case(lens, new, page, width, free, 3, sum(new) + cap_over)
    p = _tda().kv_plan(dev["lens"], dev["new"], dev["table"], dev["free"], dev["used"], page=page, max_tokens=sum(new) + cap_over)
    assert code == 0
    p.check()
    _plan_same(p, want, table, dev)


@pytest.mark.parametrize("what,code", [
    ("len", 1), ("new", 1), ("used", 1), ("entry", 1), ("sum", 1), ("width", 2), ("cap", 2), ("free", 4), ("both", 1)])
def test_plan_hands_out_nothing_when_it_cannot(what, code):
    tda = _tda()
    lens, new, used, cap, nfree = [20, 5, 31, 0], [1, 12, 2, 40], 1, 60, 20
    if what in ("len", "both"):
        lens[1] = -1
    if what == "new":
        new[2] = -3
    if what == "sum":
        new[2] = 2 ** 31 - 10
    if what == "used":
        used = -1
    if what in ("width", "both"):
        new[3] = 65
    if what == "cap":
        cap = 54
    if what == "free":
        nfree = 5
    free = list(range(100, 100 + nfree))
    dev, _, _, _ = _plan_case([max(n, 0) for n in lens], new, 16, 4, free, used, cap)
    table = dev["table"].tolist()
    if what == "entry":
        table[0][1] = -1
        dev["table"] = _i32(table)
    dev["lens"] = _i32(lens)
    got, want = H.plan(lens, new, [list(r) for r in table], free, used, 16, cap)
    assert got == code
    p = tda.kv_plan(dev["lens"], dev["new"], dev["table"], dev["free"], dev["used"], page=16, max_tokens=cap)
    _plan_same(p, want, table, dev, what)
    with pytest.raises(tda.ArError) as e:
        p.check()
    assert e.value.code == code


def test_plan_in_place_in_a_graph():
    """A captured step whose lengths and free count are updated in place, replayed step after step."""
    tda = _tda()
    B, page, steps = 300, 16, 40
    lens = [i % 37 for i in range(B)]
    free = list(range(B * 6))
    table = [[-1] * 6 for _ in range(B)]
    dev = dict(lens=_i32([0] * B), table=_i32(table), free=_i32(free), used=_i32([0]))
    first = tda.kv_plan(dev["lens"], _i32(lens), dev["table"], dev["free"], dev["used"], page=page, max_tokens=sum(lens))
    assert H.plan([0] * B, lens, table, free, 0, page, sum(lens))[0] == 0
    one, lens_dev, used_dev = _i32([1] * B), first.lens.clone(), first.free_used.clone()
    out = tda.kv_plan(lens_dev, one, dev["table"].clone(), dev["free"], used_dev, page=page, max_tokens=B)
    out = out._replace(lens=lens_dev, free_used=used_dev)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        tda.kv_plan(lens_dev, one, dev["table"], dev["free"], used_dev, page=page, max_tokens=B, out=out)
    used = int(first.free_used)
    for step in range(steps):
        graph.replay()
        code, want = H.plan(lens, [1] * B, table, free, used, page, B)
        assert code == 0
        _plan_same(out, want, table, dev, step)
        lens, used = want["lens"], want["free_used"][0]


def test_plan_of_no_requests():
    tda = _tda()
    e = _i32([])
    p = tda.kv_plan(e, e, torch.empty(0, 4, dtype=torch.int32, device="cuda"), e, _i32([0]), page=16, max_tokens=2)
    assert p.cu.tolist() == [0] and p.slots.tolist() == [-1, -1] and p.status.tolist() == [0] and p.free_used.tolist() == [0]


# -------------------------------------------------------------------- cache

def _write(pool, slots, k, v, page):
    """The pool (CPU) after ar_kv4_append by its definition."""
    D = k.shape[-1]
    kb, ksh, vb, vsh, si = H.cells(D)
    pool = pool.clone()
    kn, ks = H.quantise(k)
    vn, vs = H.quantise(v)
    for i, slot in enumerate(slots):
        if slot < 0 or slot >= pool.shape[0] * page:
            continue
        r = slot % 16
        for h in range(k.shape[1]):
            tile = pool[slot // page, h, slot % page // 16].numpy()
            for n, b, sh in ((kn, kb, ksh), (vn, vb, vsh)):
                u = n[i, h].numpy().astype(np.uint8) + np.uint8(8)
                for x in (0, 4):
                    m = sh[r] == x
                    tile[b[r, m]] = tile[b[r, m]] & (0xf0 >> x) | u[m] << x
            for at, s in ((16 * D, ks), (17 * D, vs)):
                tile[at + 2 * r * (D // 32):at + 2 * (r + 1) * (D // 32)] = s[i, h].contiguous().view(torch.uint8).numpy()
    return pool


def _same_pool(got, want):
    """Bytes equal, except that any NaN scale is as good as another."""
    D = got.shape[-1] // 18
    assert torch.equal(got[..., :16 * D], want[..., :16 * D])
    a, b = (x[..., 16 * D:].contiguous().view(torch.bfloat16).float() for x in (got, want))
    assert torch.equal(a.isnan(), b.isnan()) and torch.equal(a.nan_to_num(7), b.nan_to_num(7))


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("D,Hk,page,T", [(128, 1, 16, 1), (64, 3, 32, 37), (128, 8, 64, 130), (256, 2, 16, 19)])
@pytest.mark.parametrize("order", ["runs", "scattered"])
def test_append_and_load(dtype, D, Hk, page, T, order):
    tda = _tda()
    g = _gen(T + D)
    pages = -(-T // page) + 3
    pool = H.random_pool(g, pages, Hk, D, page)[0]
    dev = pool.cuda()
    qkv = (torch.randn(T, 2 * Hk + 3, D, generator=g) * torch.rand(T, 2 * Hk + 3, 1, generator=g) * 3).to(H.DT[dtype])
    slots = torch.randperm(pages * page, generator=g)[:T] if order == "scattered" else torch.arange(5, 5 + T)
    if T > 10:
        slots[3], slots[7] = -1, pages * page
    k, v = qkv[:, 3:3 + Hk], qkv[:, 3 + Hk:]
    kd = qkv.cuda()
    tda.kv4_append(kd[:, 3:3 + Hk], kd[:, 3 + Hk:], dev, slots.cuda())
    want = _write(pool, slots.tolist(), k, v, page)
    _same_pool(dev.cpu(), want)
    gk, gv = tda.kv4_load(dev, slots.cuda(), H.DT[dtype])
    kn, ks, vn, vs = H.unpack(want)
    for got, n, s in ((gk, kn, ks), (gv, vn, vs)):
        val = (n * s).reshape(pages, Hk, page, D)
        for i, slot in enumerate(slots.tolist()):
            exact = val[slot // page, :, slot % page] if 0 <= slot < pages * page else torch.zeros(Hk, D)
            assert torch.equal(got[i].cpu(), exact.to(H.DT[dtype])), i


@pytest.mark.parametrize("shift", [1, 3])
def test_append_and_load_with_odd_strides(shift):
    """Rows that start off 16 bytes, heads that are outermost, loads into such rows."""
    tda = _tda()
    g = _gen(shift)
    T, Hk, D, page = 21, 2, 128, 16
    flat = torch.randn(Hk * T * (D + 5) + 8, generator=g).to(torch.bfloat16)
    k = flat[shift:shift + Hk * T * (D + 5)].view(Hk, T, D + 5)[..., :D].transpose(0, 1)
    fd = flat.cuda()
    kd = fd[shift:shift + Hk * T * (D + 5)].view(Hk, T, D + 5)[..., :D].transpose(0, 1)
    pool = torch.zeros(3, Hk, 1, 18 * D, dtype=torch.uint8)
    dev = pool.cuda()
    slots = torch.arange(T) + 9
    tda.kv4_append(kd, kd, dev, slots.cuda())
    _same_pool(dev.cpu(), _write(pool, slots.tolist(), k, k, page))
    room = torch.full_like(fd, 77.0)
    od = room[shift:shift + Hk * T * (D + 5)].view(Hk, T, D + 5)[..., :D].transpose(0, 1)
    dense = tda.kv4_load(dev, slots.cuda())
    tda.kv4_load(dev, slots.cuda(), out=(od, torch.empty_like(dense[1])))
    assert torch.equal(od, dense[0])
    assert (room == 77.0).sum() >= room.numel() - T * Hk * D


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_append_of_special_values(dtype):
    """Groups of zeros, of the smallest and largest numbers, with infinities and NaN; ties of the rounding."""
    tda = _tda()
    dt = H.DT[dtype]
    tiny, top = torch.finfo(dt).smallest_normal, torch.finfo(dt).max
    rows = torch.randn(12, 1, 128, generator=_gen(3))
    rows[0] = 0
    rows[1, 0, :32] = tiny * torch.rand(32, generator=_gen(4))
    rows[2, 0, 32:64] = -top
    rows[3, 0, 64] = math.inf
    rows[4, 0, 64] = -math.inf
    rows[5, 0, 127] = math.nan
    rows[6, 0, :32] = math.inf
    rows[7, 0, :32] = torch.arange(32) * 0.5 - 7        # x / scale at .5 exactly: scale 1
    rows[7, 0, 0], rows[7, 0, 31] = -7, 7
    rows[8, 0] = -0.0
    rows[9, 0, 5] = top
    rows = rows.to(dt)
    pool = torch.full((1, 1, 1, 2304), 0xa5, dtype=torch.uint8)
    dev = pool.cuda()
    slots = torch.arange(12)
    tda.kv4_append(rows.cuda(), rows.flip(0).cuda(), dev, slots.cuda())
    want = _write(pool, slots.tolist(), rows, rows.flip(0), 16)
    _same_pool(dev.cpu(), want)
    k, _ = tda.kv4_load(dev, slots.cuda(), dt)
    assert k[3, 0, 64:96].isnan().all() and not k[3, 0, :64].isnan().any()
    assert k[5, 0, 96:].isnan().all() and (k[0] == 0).all()


# ---------------------------------------------------------------- attention

def _attend_case(seed, B, lens, new, Hk, G, D, page, dtype, q_scale=1.0):
    g = _gen(seed)
    T = sum(new)
    width = max(1, -(-max(lens + [1]) // page) + 1)
    pages = sum(-(-n // page) for n in lens) + 2
    pool, K, V = H.random_pool(g, pages, Hk, D, page)
    perm = torch.randperm(pages, generator=g).tolist()
    table, at = [], 0
    for n in lens:
        m = -(-n // page)
        table.append(perm[at:at + m] + [-7] * (width - m))
        at += m
    q = (torch.randn(T, Hk * G, D, generator=g) * q_scale).to(H.DT[dtype])
    cu = [0]
    for m in new:
        cu.append(cu[-1] + m)
    return q, pool, K, V, table, cu


def _check_attend(q, K, V, table, lens, cu, window, sinks, scale, out, lse):
    want, wl, mag, big, top = H.attend(q, K, V, table, lens, cu, window, sinks, scale)
    bo, bl = H.attend_bounds(want, wl, mag, big, top, scale, q.dtype, max(lens + [1]))
    got, gl = out.cpu().double(), lse.cpu().double()
    none = wl == -math.inf
    assert (got[none] == 0).all() and (gl[none] == -math.inf).all()
    assert torch.isfinite(got).all()
    over = ((got - want).abs() / bo).amax().item() if got.numel() else 0
    assert over <= 1, f"out off by {over:.3g} times its bound"
    over = ((gl - wl)[~none].abs() / bl[~none]).amax().item() if (~none).any() else 0
    assert over <= 1, f"lse off by {over:.3g} times its bound"


ATTEND = [
    # lens, new (None: one each), Hk, G, D, page, window, sinks
    ([1], None, 1, 1, 128, 16, 0, 0),
    ([1, 15, 16, 17, 31, 32, 33], None, 2, 8, 128, 16, 0, 0),
    ([63, 64, 65, 127, 128, 129], None, 1, 4, 128, 64, 0, 0),
    ([1000, 3, 517], None, 2, 8, 64, 32, 0, 0),
    ([777, 40], None, 1, 8, 256, 16, 0, 0),
    ([700], None, 3, 5, 128, 16, 0, 0),
    ([333, 90], None, 1, 16, 128, 16, 0, 0),
    ([400, 61], None, 2, 24, 64, 16, 0, 0),
    ([5000], None, 1, 8, 128, 16, 0, 0),
    ([0, 9, 0, 100], None, 1, 8, 128, 16, 0, 0),
    # several new tokens, requests without any among them
    ([20, 9, 300, 64], [3, 0, 8, 1], 2, 6, 128, 16, 0, 0),
    ([40, 17], [40, 17], 1, 2, 128, 16, 0, 0),
    ([260, 130], [130, 2], 1, 8, 64, 32, 0, 0),
    ([90, 33], [7, 5], 2, 3, 256, 16, 0, 0),
    ([5, 70], [9, 70], 1, 4, 128, 16, 0, 0),          # more new tokens than the cache holds: rows that see nothing
    # windows and sinks
    ([1000, 3, 517], None, 2, 8, 128, 16, 1, 0),
    ([1000, 3, 517], None, 2, 8, 128, 16, 100, 4),
    ([1000, 30, 517], None, 1, 8, 64, 32, 128, 17),
    ([1000, 30, 517], [9, 30, 1], 1, 4, 128, 64, 33, 1),
    ([600, 40], [50, 7], 2, 8, 128, 16, 16, 0),
    ([300], None, 1, 8, 128, 16, 1000, 4),
    ([300], None, 1, 8, 128, 16, 100, 400),
    ([300], None, 1, 8, 128, 16, 0, 50),
]


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("case", range(len(ATTEND)))
def test_attend(case, dtype):
    lens, new, Hk, G, D, page, window, sinks = ATTEND[case]
    tda = _tda()
    one = new is None
    q, pool, K, V, table, cu = _attend_case(case, len(lens), lens, new or [1] * len(lens), Hk, G, D, page, dtype)
    ws = tda.Kv4Workspace()
    out, lse = tda.kv4_attend(q.cuda(), pool.cuda(), _i32(table), _i32(lens), None if one else _i32(cu),
                              max_new=None if case % 2 else max(new or [1]), window=window, sinks=sinks, return_lse=True,
                              workspace=ws)
    torch.cuda.synchronize()
    ws.check()
    _check_attend(q, K, V, table, lens, cu, window, sinks, D ** -0.5, out, lse)


@pytest.mark.parametrize("D,G,new", [(128, 8, 1), (64, 4, 3), (256, 8, 1)])
def test_attend_split_over_many_blocks(D, G, new):
    """One long request: the tokens are split over blocks and joined; the same bits every time."""
    tda = _tda()
    lens = [20011]
    q, pool, K, V, table, cu = _attend_case(5, 1, lens, [new], 2, G, D, 64, "f16")
    args = (q.cuda(), pool.cuda(), _i32(table), _i32(lens), _i32(cu))
    out, lse = tda.kv4_attend(*args, return_lse=True)
    _check_attend(q, K, V, table, lens, cu, 0, 0, D ** -0.5, out, lse)
    for _ in range(20):
        again = tda.kv4_attend(*args, return_lse=True)
        assert torch.equal(again[0], out) and torch.equal(again[1], lse)


@pytest.mark.parametrize("mult,scale", [(1e-3, None), (12.0, None), (1.0, 0.0), (1.0, -0.2), (3e30, 1e-31), (1e-30, 1e29)])
def test_attend_range_of_q(mult, scale):
    """Queries and scales far from one: sharp and flat softmaxes, bf16's whole range."""
    tda = _tda()
    lens = [300, 77, 1]
    q, pool, K, V, table, cu = _attend_case(9, 3, lens, [1] * 3, 2, 8, 128, 16, "bf16", mult)
    out, lse = tda.kv4_attend(q.cuda(), pool.cuda(), _i32(table), _i32(lens), scale=scale, return_lse=True)
    _check_attend(q, K, V, table, lens, cu, 0, 0, 128 ** -0.5 if scale is None else scale, out, lse)


@pytest.mark.parametrize("size", [1e-4, 1.0, 3e4, 1e-30, 1e30])
def test_attend_range_of_v(size):
    """V scales from bf16's smallest to its largest, rising along the tokens and differing by group."""
    tda = _tda()
    D, page, n = 128, 16, 400
    q, pool, K, V, table, cu = _attend_case(11, 1, [n], [1], 1, 8, D, page, "bf16")
    factor = torch.logspace(-3, 3, n).view(-1, 1) * torch.tensor([1.0, 1e-2, 30.0, 1e-3]).view(1, 4) * size
    kn, ks, vn, vs = H.unpack(pool)
    new = torch.zeros(pool.shape[0] * page, 4)
    for i, pid in enumerate(table[0][:n // page]):
        new[pid * page:(pid + 1) * page] = factor[i * page:(i + 1) * page]
    vs16 = (new * 0.3).to(torch.bfloat16).view(pool.shape[0], 1, 1, 16, 4)
    pool = H.pack(kn, ks[..., ::32].to(torch.bfloat16), vn, vs16)
    kn, ks, vn, vs = H.unpack(pool)
    V = (vn * vs).reshape(V.shape)
    out, lse = tda.kv4_attend(q.cuda(), pool.cuda(), _i32(table), _i32([n]), return_lse=True)
    _check_attend(q, K, V, table, [n], cu, 0, 0, D ** -0.5, out, lse)


def test_attend_sharp_scores_late_and_early():
    """The largest scores first, last and in the middle of long requests, 60 above the rest."""
    tda = _tda()
    n, D, page = 3000, 128, 16
    lens = [n] * 3
    q, pool, K, V, table, cu = _attend_case(13, 3, lens, [1] * 3, 1, 8, D, page, "f16")
    kn, ks, vn, vs = H.unpack(pool)
    for b, at in enumerate((0, n // 2, n - 1)):
        row = (q[b, 0].double() / q[b, 0].double().abs().max() * 7).round()
        pid, r = table[b][at // page], at % page
        kn[pid, 0, 0, r] = row
        ks[pid, 0, 0, r] = 2.0
    pool = H.pack(kn, ks[..., ::32].to(torch.bfloat16), vn, vs[..., ::32].to(torch.bfloat16))
    K = (kn * ks).reshape(K.shape)
    out, lse = tda.kv4_attend(q.cuda(), pool.cuda(), _i32(table), _i32(lens), return_lse=True)
    _check_attend(q, K, V, table, lens, cu, 0, 0, D ** -0.5, out, lse)


@pytest.mark.parametrize("new", [1, 5])
@pytest.mark.parametrize("window,sinks", [(0, 0), (40, 3)])
def test_attend_never_touches_what_is_masked(new, window, sinks):
    """Tokens past the length, in pages of no request, behind the window: NaN and infinite scales there
    change nothing."""
    tda = _tda()
    lens, D, page = [37, 201, 16], 128, 16
    q, pool, K, V, table, cu = _attend_case(17, 3, lens, [new] * 3, 2, 4, D, page, "bf16")
    args = (_i32(table), _i32(lens), _i32(cu))
    clean = tda.kv4_attend(q.cuda(), pool.cuda(), *args, window=window, sinks=sinks, return_lse=True)
    seen = torch.zeros(pool.shape[0], page, dtype=torch.bool)
    for b, n in enumerate(lens):
        for j in range(n):
            low = n - new - window + 1 if window else 0
            if j >= low or j < sinks:
                seen[table[b][j // page], j % page] = True
    scales = pool[..., 16 * D:].contiguous().view(torch.bfloat16).view(pool.shape[0], 2, 1, 2, 16, 4)
    poison = torch.tensor([math.nan, math.inf, -math.inf, 3e38]).to(torch.bfloat16)
    scales = torch.where(seen.view(-1, 1, 1, 1, 16, 1), scales, poison)
    bad = pool.clone()
    bad[..., 16 * D:] = scales.contiguous().view(torch.uint8).view(*pool.shape[:3], 2 * D)
    got = tda.kv4_attend(q.cuda(), bad.cuda(), *args, window=window, sinks=sinks, return_lse=True)
    assert torch.equal(got[0], clean[0]) and torch.equal(got[1], clean[1])
    _check_attend(q, K, V, table, lens, cu, window, sinks, D ** -0.5, *got)


def test_attend_nan_in_sight_stays_where_it_belongs():
    """A visible NaN group of V reaches its own 32 channels, a NaN of K its request's rows, and nothing else."""
    tda = _tda()
    lens, D, page = [50, 50, 50], 128, 16
    q, pool, K, V, table, cu = _attend_case(19, 3, lens, [1] * 3, 1, 8, D, page, "bf16")
    clean = tda.kv4_attend(q.cuda(), pool.cuda(), _i32(table), _i32(lens))
    scales = pool[..., 16 * D:].contiguous().view(torch.bfloat16).view(pool.shape[0], 2, 16, 4)
    scales[table[1][1], 1, 3, 2] = math.nan
    scales[table[2][0], 0, 5, 0] = math.nan
    pool[..., 16 * D:] = scales.view(torch.uint8).view(pool.shape[0], 1, 1, 2 * D)
    got = tda.kv4_attend(q.cuda(), pool.cuda(), _i32(table), _i32(lens))
    assert torch.equal(got[0], clean[0])
    assert got[1, :, 64:96].isnan().all() and torch.equal(got[1, :, :64], clean[1, :, :64])
    assert torch.equal(got[1, :, 96:], clean[1, :, 96:])
    assert got[2].isnan().all()


def test_attend_strides_and_given_outputs():
    """q inside a fused projection, out in a wider buffer, rows off 16 bytes, a wider table."""
    tda = _tda()
    lens, Hk, G, D, page = [130, 47], 2, 4, 64, 16
    q, pool, K, V, table, cu = _attend_case(23, 2, lens, [1] * 2, Hk, G, D, page, "f16")
    fused = torch.zeros(2, Hk * G + 4, D + 3, dtype=torch.float16, device="cuda")
    fused[:, 2:2 + Hk * G, 1:1 + D] = q.cuda()
    wide = torch.full((2, Hk * G + 2, D + 1), 5.0, dtype=torch.float16, device="cuda")
    tab = torch.full((2, len(table[0]) + 9), -1, dtype=torch.int32, device="cuda")
    tab[:, :len(table[0])] = _i32(table)
    lse = torch.empty(2, Hk * G, device="cuda")
    out, same = tda.kv4_attend(fused[:, 2:2 + Hk * G, 1:1 + D], pool.cuda(), tab[:, :len(table[0])], _i32(lens),
                               out=wide[:, 1:1 + Hk * G, :D], lse=lse)
    assert same is lse
    _check_attend(q, K, V, table, lens, cu, 0, 0, D ** -0.5, out, lse)
    assert (wide[:, 0] == 5).all() and (wide[:, -1] == 5).all() and (wide[:, :, D:] == 5).all()


def test_attend_reports_what_the_device_finds():
    """Page ids outside the pool, lengths past the table, rows outside q: AR_EINVAL in the workspace, and
    the other requests are right."""
    tda = _tda()
    lens, D, page = [40, 60, 33], 128, 16
    q, pool, K, V, table, cu = _attend_case(29, 3, lens, [1] * 3, 1, 8, D, page, "bf16")
    qd, pd = q.cuda(), pool.cuda()
    want, lse, mag, big, top = H.attend(q, K, V, table, lens, cu, 0, 0, D ** -0.5)
    bound = H.attend_bounds(want, lse, mag, big, top, D ** -0.5, q.dtype, max(lens))[0]
    for what in ("high", "low", "long", "negative", "rows"):
        ws = tda.Kv4Workspace()
        t, n, c = [list(r) for r in table], list(lens), list(cu)
        if what == "high":
            t[1][2] = pool.shape[0]
        if what == "low":
            t[1][0] = -1
        if what == "long":
            n[1] = len(t[1]) * page + 1
        if what == "negative":
            n[1] = -1
        if what == "rows":
            c = [0, 1, 1, 5]
        got = tda.kv4_attend(qd, pd, _i32(t), _i32(n), _i32(c), workspace=ws)
        torch.cuda.synchronize()
        assert ws.status() == tda.ar.AR_EINVAL, what
        with pytest.raises(tda.ArError):
            ws.check()
        for b in (0,) if what == "rows" else (0, 2):
            assert ((got[b].cpu().double() - want[b]).abs() <= bound[b]).all(), what


def test_attend_on_streams_and_in_a_graph():
    tda = _tda()
    lens, D, page = [900, 130, 64], 128, 16
    q, pool, K, V, table, cu = _attend_case(31, 3, lens, [1] * 3, 2, 8, D, page, "bf16")
    qd, pd, td, ld = q.cuda(), pool.cuda(), _i32(table), _i32(lens)
    want = tda.kv4_attend(qd, pd, td, ld)
    streams = [torch.cuda.Stream() for _ in range(3)]
    torch.cuda.synchronize()
    outs = [[tda.kv4_attend(qd, pd, td, ld, stream=s) for s in streams] for _ in range(10)]
    torch.cuda.synchronize()
    assert all(torch.equal(o, want) for row in outs for o in row)
    s = streams[0]
    out = torch.zeros_like(want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(s):
        with torch.cuda.graph(graph, stream=s):
            tda.kv4_attend(qd, pd, td, ld, out=out)
    for i in range(3):
        qd.copy_(torch.roll(q.cuda(), i, 0))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, tda.kv4_attend(qd, pd, td, ld))


def test_workspace_is_not_made_inside_a_capture():
    tda = _tda()
    s = torch.cuda.Stream()
    x = torch.zeros(8, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(s), torch.cuda.graph(graph, stream=s):
        x.add_(1)
        with pytest.raises(RuntimeError, match="captured"):
            tda.Kv4Workspace()


# --------------------------------------------------------------------- norm

def _e4m3_near(got, want):
    """got (e4m3 values) against the unrounded quotients: within half a step, plus 2^-20 of the value for binary32."""
    got, mag = got.double(), want.abs()
    step = torch.exp2(torch.floor(torch.log2(mag.clamp(min=2.0 ** -6))) - 3)
    # 448 is the largest: at the top of a group the quotient is 448 but for rounding
    return ((got - want).abs() <= step / 2 + mag * 2.0 ** -20).all()


def _check_norm(x, r, w, eps, group, out, scales, ro):
    q, s, h = H.norm_fp8(x, r, w, eps, group)
    # binary32: squares summed in order of at most dim / 256 + 16 terms a lane, the root and products a few 2^-24
    rel = (x.shape[1] / 256 + 40) * 2.0 ** -24
    assert ((scales.cpu().double() - s).abs() <= s * rel).all()
    assert _e4m3_near(out.cpu().float(), q)
    if ro is not None:
        f32 = (x.float() + r.float()) if r is not None else x.float()
        assert torch.equal(ro.cpu(), f32.to(x.dtype))


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("N,d,group", [
    (1, 1, 0), (1, 1, 1), (3, 7, 0), (2, 8, 8), (5, 64, 32), (4, 127, 0), (4, 128, 128), (3, 200, 128), (2, 1000, 128),
    (7, 1024, 0), (3, 4096, 128), (2, 5120, 0), (33, 2048, 64), (2, 8192, 0), (2, 8192, 128), (2, 12288, 256), (1, 16384, 128),
    (2, 20000, 0), (1, 32768, 128), (1, 32760, 0), (2, 4097, 128), (2, 6144, 100), (300, 512, 0), (4, 2048, 1024), (600, 1536, 128)])
def test_norm(dtype, N, d, group):
    tda = _tda()
    g = _gen(N * d)
    x, r = ((torch.randn(N, d, generator=g) * s).to(H.DT[dtype]) for s in (0.3, 2.0))
    w = (1 + 0.3 * torch.randn(d, generator=g)).to(H.DT[dtype])
    out, scales, ro = tda.add_norm_fp8(x.cuda(), w.cuda(), residual=r.cuda(), eps=1e-5, group=group)
    _check_norm(x, r, w, 1e-5, group, out, scales, ro)
    out, scales, ro = tda.add_norm_fp8(x.cuda(), w.cuda(), eps=1e-5, group=group)
    assert ro is None
    _check_norm(x, None, w, 1e-5, group, out, scales, None)


@pytest.mark.parametrize("d,group", [(512, 0), (512, 128), (4100, 0), (9000, 128)])
def test_norm_strides_and_in_place(d, group):
    tda = _tda()
    g = _gen(d)
    N = 6
    xw = torch.randn(N, d + 11, generator=g).to(torch.bfloat16)
    rw = torch.randn(N, d + 5, generator=g).to(torch.bfloat16)
    w = torch.rand(d, generator=g).to(torch.bfloat16)
    for off in (0, 3):
        x, r = xw[:, off:off + d], rw[:, :d]
        xd, rd = xw.cuda()[:, off:off + d], rw.cuda()[:, :d]
        out, scales, ro = tda.add_norm_fp8(xd, w.cuda(), residual=rd, residual_out=rd, group=group)
        assert ro is rd
        _check_norm(x, r, w, 1e-6, group, out, scales, ro)
        again = tda.add_norm_fp8(xd, w.cuda(), residual=rw.cuda()[:, :d], residual_out=xd, group=group)
        assert torch.equal(again[0].view(torch.uint8), out.view(torch.uint8)) and torch.equal(xd, rd)


@pytest.mark.parametrize("group", [0, 128])
def test_norm_of_special_rows(group):
    """Zeros (scale 1), one huge value, a NaN, an infinity, tiny numbers."""
    tda = _tda()
    d = 1024
    x = torch.randn(6, d, generator=_gen(1)).to(torch.bfloat16)
    x[0] = 0
    x[1, 5] = 1e6
    x[2, 7] = math.nan
    x[3, 9] = math.inf
    x[4] = x[4] * 1e-20
    w = torch.ones(d, dtype=torch.bfloat16)
    out, scales, _ = tda.add_norm_fp8(x.cuda(), w.cuda(), group=group)
    f = out.float().cpu()
    assert (f[0] == 0).all() and (scales[0] == 1).all()
    assert f[2].isnan().all()
    assert f[3, 9].isnan()
    keep = [1, 4, 5]
    _check_norm(x[keep], None, w, 1e-6, group, out[keep], scales[keep], None)


def test_binding_refusals_on_the_gpu():
    tda = _tda()
    dev = "cuda"
    pool = tda.kv4_pool(4, 2, 128, 16)
    q = torch.zeros(3, 8, 128, dtype=torch.bfloat16, device=dev)
    k = torch.zeros(3, 2, 128, dtype=torch.bfloat16, device=dev)
    t, n, s = torch.zeros(3, 4, dtype=torch.int32, device=dev), _i32([1, 1, 1]), torch.zeros(3, dtype=torch.int64, device=dev)
    f8 = torch.float8_e4m3fn
    bad = [
        (lambda: tda.kv4_attend(q.float(), pool, t, n), "dtype"),
        (lambda: tda.kv4_attend(q[:, :7], pool, t, n), "7 heads for 2"),
        (lambda: tda.kv4_attend(q[..., :64], pool, t, n), "head_dim 64"),
        (lambda: tda.kv4_attend(q[:2], pool, t, n), "2 tokens for 3"),
        (lambda: tda.kv4_attend(q, pool, t[:2], n), "2 rows for 3"),
        (lambda: tda.kv4_attend(q, pool, t.long(), n), "table: dtype"),
        (lambda: tda.kv4_attend(q, pool, t, n.long()), "lens: dtype"),
        (lambda: tda.kv4_attend(q, pool, t, n, n), "cu: shape"),
        (lambda: tda.kv4_attend(q, pool[..., :2000], t, n), "pool: not contiguous"),
        (lambda: tda.kv4_attend(q, pool.view(4, 2, 2, 1152)[:, :, :, :1000].contiguous(), t, n), "pool: shape"),
        (lambda: tda.kv4_attend(q, pool, t, n, out=q[:, :4]), "out: shape"),
        (lambda: tda.kv4_attend(q, pool, t, n, lse=torch.zeros(3, 7, device=dev)), "lse: shape"),
        (lambda: tda.kv4_attend(q.transpose(1, 2).contiguous().transpose(1, 2), pool, t, n), "last dimension"),
        (lambda: tda.kv4_append(k, k[:2], pool, s), "v: shape"),
        (lambda: tda.kv4_append(k, k.half(), pool, s), "v: dtype"),
        (lambda: tda.kv4_append(k.float(), k.float(), pool, s), "neither"),
        (lambda: tda.kv4_append(k, k, pool, s.int()), "slots: dtype"),
        (lambda: tda.kv4_load(pool, s, torch.float32), "neither"),
        (lambda: tda.kv4_load(pool, s, torch.float16, out=(k, k)), "out: dtype"),
        (lambda: tda.kv_plan(n, n, t[:2], n, n[:1], page=16, max_tokens=3), "table: 2 rows"),
        (lambda: tda.kv_plan(n, n[:2], t, n, n[:1], page=16, max_tokens=3), "new: shape"),
        (lambda: tda.kv_plan(n, n, t, n, n, page=16, max_tokens=3), "free_used: shape"),
        (lambda: tda.kv_plan(n, n, t, n, n[:1], page=16, max_tokens=-1), "negative"),
        (lambda: tda.add_norm_fp8(q[0], q[0, 0, :64]), "weight: shape"),
        (lambda: tda.add_norm_fp8(q[0], q[0, 0], residual=q[0, :4]), "residual: shape"),
        (lambda: tda.add_norm_fp8(q[0], q[0, 0], group=129), "group"),
        (lambda: tda.add_norm_fp8(q[0], q[0, 0], out=torch.zeros(8, 127, device=dev).to(f8)), "out: shape"),
    ]
    for f, msg in bad:
        with pytest.raises(ValueError, match=msg):
            f()
    with pytest.raises(tda.ArError):
        tda.kv_plan(n, n, t, n, n[:1], page=17, max_tokens=3)
    with pytest.raises(tda.ArError):
        tda.kv4_attend(q, pool, t, n, window=-1)


# ------------------------------------------------------- sizes and places

@pytest.mark.parametrize("page", [48, 112])
def test_pages_that_are_no_power_of_two(page):
    tda = _tda()
    lens, Hk, D = [page * 3 + 5, 7, page], 2, 128
    q, pool, K, V, table, cu = _attend_case(37, 3, lens, [1] * 3, Hk, 8, D, page, "bf16")
    out, lse = tda.kv4_attend(q.cuda(), pool.cuda(), _i32(table), _i32(lens), return_lse=True)
    _check_attend(q, K, V, table, lens, cu, 0, 0, D ** -0.5, out, lse)
    k = torch.randn(page + 3, Hk, D, generator=_gen(2)).to(torch.bfloat16)
    slots = torch.arange(page + 3) + 11
    dev = pool.cuda()
    tda.kv4_append(k.cuda(), k.flip(0).cuda(), dev, slots.cuda())
    _same_pool(dev.cpu(), _write(pool, slots.tolist(), k, k.flip(0), page))


@pytest.mark.parametrize("new", [[1], [0, 1, 3, 0, 0, 2]])
def test_attend_many_requests(new):
    """More requests than a block has threads, most of them short, some without new tokens."""
    tda = _tda()
    B = 1500
    g = np.random.RandomState(1)
    lens = [int(x) for x in g.randint(1, 40, B)]
    lens[700] = 3000
    new = [min(new[i % len(new)], lens[i]) for i in range(B)]
    q, pool, K, V, table, cu = _attend_case(41, B, lens, new, 1, 4, 64, 16, "f16")
    out, lse = tda.kv4_attend(q.cuda(), pool.cuda(), _i32(table), _i32(lens), _i32(cu), max_new=max(new), return_lse=True)
    _check_attend(q, K, V, table, lens, cu, 0, 0, 64 ** -0.5, out, lse)


def test_offsets_past_32_bits():
    """A cache of over 4 GiB: pages at its end are written, read back and attended over like those at its start."""
    tda = _tda()
    D, page, n = 128, 16, 75
    pages = (4 << 30) // 2304 + 50
    pool = torch.empty(pages, 1, 1, 2304, dtype=torch.uint8, device="cuda")
    g = _gen(43)
    k, v = ((torch.randn(n, 1, D, generator=g)).to(torch.bfloat16).cuda() for _ in range(2))
    q = torch.randn(1, 8, D, generator=g).to(torch.bfloat16).cuda()
    slots = torch.arange(n, device="cuda")
    got = []
    for first in (0, pages - 5):
        at = slots + first * page
        tda.kv4_append(k, v, pool, at)
        table = torch.arange(first, first + 5, dtype=torch.int32, device="cuda")[None]
        got.append((*tda.kv4_load(pool, at), tda.kv4_attend(q, pool, table, _i32([n]))))
    for a, b in zip(*got):
        assert torch.equal(a, b)
    assert (got[0][0].float() - k.float()).abs().max() < 0.5 and got[0][2].abs().sum() > 0


def test_attend_refuses_to_write_over_q():
    tda = _tda()
    q, pool, K, V, table, cu = _attend_case(1, 1, [20], [1], 1, 8, 64, 16, "f16")
    qd = q.cuda()
    with pytest.raises(tda.ArError):
        tda.kv4_attend(qd, pool.cuda(), _i32(table), _i32([20]), out=qd)
