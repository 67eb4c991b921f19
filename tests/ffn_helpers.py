"""Plain implementations, in 64 bits, of the operators of include/ar_ffn.h, and how far a kernel may be off.
Nothing here calls the library."""
import math

import torch

DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
HALF = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}     # half a step, relative to the value
TINY = {torch.bfloat16: 2.0 ** -134, torch.float16: 2.0 ** -25}   # half a step where numbers are subnormal
F8 = torch.float8_e4m3fn


def gen(seed, device="cpu"):
    return torch.Generator(device=device).manual_seed(seed)


def eights(g, *shape, spread=150.0):
    """e4m3 values, normally distributed, some zeros among them."""
    return (torch.randn(*shape, generator=g) * spread).clamp(-448, 448).to(F8)


def scales(g, *shape, size=0.01):
    return torch.randn(*shape, generator=g).mul(0.5).exp().mul(size)


def product(x, xs, w, ws):
    """(out, sum of the terms' magnitudes), float64: x [M, K], xs [M, G or 1], w [N, K], ws [ceil(N / 128), G]."""
    M, K, N = x.shape[0], x.shape[1], w.shape[0]
    out, mag = torch.zeros(M, N, dtype=torch.float64), torch.zeros(M, N, dtype=torch.float64)
    block = torch.arange(N) // 128
    for g in range(ws.shape[1]):
        cut = slice(128 * g, min(K, 128 * g + 128))
        s = xs[:, g if xs.shape[1] > 1 else 0].double()[:, None] * ws[block, g].double()[None]
        a, b = x[:, cut].double(), w[:, cut].double()
        out += s * (a @ b.T)
        mag += s.abs() * (a.abs() @ b.abs().T)
    return out, mag


def product_bound(want, mag, groups, dtype):
    """How far a product may be off.

    Terms are exact (4 bits times 4).  A group's sum is made in at most 8 steps of a matrix instruction, each of which
    may cut what lies below 2^-22 of the largest partial sum, so it is off by less than 2^-19 of the terms' magnitudes.  The product of
    the two scales, and that times the group's sum, are rounded to 2^-24 each; the running sum once a group and up to 16
    times more where parts are added: (groups + 18) 2^-24 of the magnitudes together.  Then the rounding of the output.
    """
    inner = mag * (2.0 ** -19 + (groups + 18) * 2.0 ** -24)
    return inner + (want.abs() + inner) * HALF[dtype] + TINY[dtype]


def check_product(got, x, xs, w, ws):
    want, mag = product(x, xs, w, ws)
    limit = product_bound(want, mag, ws.shape[1], got.dtype)
    off = (got.double().cpu() - want).abs()
    assert got.shape == want.shape
    bad = ~(off <= limit)
    assert not bad.any(), f"{int(bad.sum())} of {bad.numel()} too far off, first {bad.nonzero()[0].tolist()}, by {(off / limit).nan_to_num(math.inf).max():.3g} limits"


def route(logits, k, normalize):
    """(weights float64, experts, offsets, rows, place) by the definition, pair by pair."""
    T, E = logits.shape
    x = logits.double()
    big = torch.finfo(torch.float32).max
    x = torch.where(x > big, big, x)
    weights, experts = torch.zeros(T, k, dtype=torch.float64), torch.full((T, k), -1, dtype=torch.int64)
    per = [[] for _ in range(E)]
    for t in range(T):
        row = x[t].tolist()
        able = [e for e in range(E) if row[e] > -math.inf]           # (not NaN either)
        pick = sorted(able, key=lambda e: (-row[e], e))[:k]
        if not pick:
            continue
        m = row[pick[0]]
        total = sum(math.exp(row[e] - m) for e in (pick if normalize else able))
        for j, e in enumerate(pick):
            experts[t, j] = e
            weights[t, j] = math.exp(row[e] - m) / total
            per[e].append((t, j))
    offsets, rows, place = [0], torch.full((T * k,), -1, dtype=torch.int64), torch.full((T, k), -1, dtype=torch.int64)
    at = 0
    for e in range(E):
        for t, j in per[e]:
            rows[at] = t
            place[t, j] = at
            at += 1
        offsets.append(at)
    return weights, experts, torch.tensor(offsets), rows, place


def silu_mul(x):
    x = x.double()
    d = x.shape[1] // 2
    return x[:, :d] * torch.sigmoid(x[:, :d]) * x[:, d:]


def check_silu(out, scales_, x, group):
    """e4m3 output and scales against y in 64 bits.

    exp(-g) goes through a power of two whose argument is rounded, for gates from -8 on: 11.6 at most, so by 2^-21, and off by
    11.6 2^-26.2 because log2(e) is, which is ln 2 (4.8e-7 + 1.5e-7) = 4.4e-7 of the power; the instruction adds 2^-22 = 2.4e-7, the sum
    2^-24, the reciprocal 2^-23, two products 2^-23: y is off by less than 1.0e-6 < 2^-19.9 of itself (smaller gates, by
    exp of 2 units in the last place: less), and by 2^-148 where a step is subnormal.  The scale is the largest |y| over 448, 2^-23 more: below
    2^-19.7; out is y / scale (2^-19.9 + 2^-19.7 + 2^-22 < 2^-18.6) rounded to e4m3, by at most 2^-4 of it or half the subnormal step, 2^-10.
    """
    y = silu_mul(x)
    N, d = y.shape
    group = min(group, d) or max(d, 1)
    for i, a in enumerate(range(0, max(d, 1), group)):
        part = y[:, a:a + group]
        top = part.abs().amax(1) if part.shape[1] else torch.zeros(N, dtype=torch.float64)
        want = torch.where(top > 0, top / 448, 1.0)
        s = scales_[:, i].double().cpu()
        small = top < 2.0 ** -140                                     # (zero or not: either is within the rounding)
        assert ((s - want).abs() <= want * 2.0 ** -19.7 + 2.0 ** -149)[~small].all(), "scale"
        v = part / want[:, None]
        off = (out[:, a:a + group].double().cpu() - v).abs()
        limit = v.abs() * (2.0 ** -4 + 2.0 ** -18.6) + 2.0 ** -10 * (1 + 2.0 ** -18.6)
        assert (off <= limit)[~small].all(), f"values, off by {(off / limit)[~small].max()} limits"


def weighted(x, w, place):
    T, k = w.shape
    out, mag = torch.zeros(T, x.shape[1], dtype=torch.float64), torch.zeros(T, x.shape[1], dtype=torch.float64)
    for j in range(k):
        p = place[:, j].long()
        there = ((p >= 0) & (p < x.shape[0]))[:, None]
        if x.shape[0] == 0:
            break
        v = torch.where(there, x[p.clamp(0, x.shape[0] - 1)].double(), 0.0)
        v = torch.where(there, v * w[:, j, None].double(), 0.0)
        out += v
        mag += v.abs()
    return out, mag


def check_weighted(got, x, w, place):
    """Each step is one rounding of at most 2^-24 of what has been added up, then that of the output."""
    want, mag = weighted(x, w, place)
    inner = mag * w.shape[1] * 2.0 ** -24
    limit = inner + (want.abs() + inner) * HALF[got.dtype] + TINY[got.dtype]
    assert ((got.double().cpu() - want).abs() <= limit).all()
