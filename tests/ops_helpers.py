"""Plain implementations, in 64 bits, of the operators of include/ar_ops.h, and
the 4-bit cache's packing from its documented layout.  Nothing here calls the library."""
import math

import numpy as np
import torch

DT = {"bf16": torch.bfloat16, "f16": torch.float16}
EPS = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}   # one rounding, relative: 8 and 11 significant bits


def cells(D):
    """(K byte, K shift, V byte, V shift, scale index) of every token and channel of a tile: arrays [16, D]."""
    G = D // 32
    r, c = np.meshgrid(np.arange(16), np.arange(D), indexing="ij")
    j = c // 32
    kw = (r * 4 + c % 32 // 8) * G + j
    ki = c % 8
    vw = (r // 8 * 32 + c % 32 // 4 * 4 + r % 8 // 2) * G + j
    vi = r % 2 * 4 + c % 4
    return kw * 4 + ki // 2, ki % 2 * 4, 8 * D + vw * 4 + vi // 2, vi % 2 * 4, r * G + j


def pack(kn, ks, vn, vs):
    """Whole numbers n [..., 16, D] and bfloat16 scales [..., 16, D / 32] -> tiles uint8 [..., 18 D] (CPU tensors)."""
    D = kn.shape[-1]
    lead = kn.shape[:-2]
    kb, ksh, vb, vsh, _ = cells(D)
    tiles = np.zeros((int(np.prod(lead, dtype=np.int64)), 18 * D), np.uint8)
    for n, b, sh in ((kn, kb, ksh), (vn, vb, vsh)):
        u = (n.reshape(-1, 16, D).numpy().astype(np.int64) + 8).astype(np.uint8)
        for half in (0, 4):
            m = sh == half
            tiles[:, b[m]] |= u[:, m] << half
    for at, s in ((16 * D, ks), (17 * D, vs)):
        tiles[:, at:at + D] = s.contiguous().reshape(-1, D // 2).view(torch.uint8).numpy()
    return torch.from_numpy(tiles).view(*lead, 18 * D)


def unpack(tiles):
    """tiles uint8 [..., 18 D] (CPU) -> n and scales as float64: kn [..., 16, D], ks [..., 16, D] (spread), vn, vs."""
    D = tiles.shape[-1] // 18
    lead = tiles.shape[:-1]
    kb, ksh, vb, vsh, si = cells(D)
    t = tiles.reshape(-1, 18 * D).numpy()
    out = []
    for b, sh, at in ((kb, ksh, 16 * D), (vb, vsh, 17 * D)):
        n = (t[:, b] >> sh & 15).astype(np.float64) - 8
        s = torch.from_numpy(np.ascontiguousarray(t[:, at:at + D])).view(torch.bfloat16).double().numpy()[:, si]
        out += [torch.from_numpy(n).view(*lead, 16, D), torch.from_numpy(s).view(*lead, 16, D)]
    return out


def quantise(x):
    """float [..., D] -> (n, scales bfloat16 [..., D / 32]) by ar_kv4_append's definition, binary32 like it."""
    x = x.float().reshape(*x.shape[:-1], -1, 32)
    top = x.abs().amax(-1, keepdim=True)
    top = torch.where(x.isnan().any(-1, keepdim=True), math.nan, top)
    s = torch.from_numpy((top.numpy() / np.float32(7)).astype(np.float32)).to(torch.bfloat16)
    with np.errstate(all="ignore"):
        n = np.rint((x.numpy() / s.float().numpy()).astype(np.float32))
    n = torch.from_numpy(np.where(np.isnan(n), 0, np.clip(n, -7, 7)))
    return n.flatten(-2), s.squeeze(-1)


def random_pool(g, pages, Hk, D, page, spread=0.3):
    """(pool on the CPU, K values, V values as float64 [pages, Hk, page, D])."""
    lead = (pages, Hk, page // 16)
    parts = []
    for _ in range(2):
        n = (torch.randn(*lead, 16, D, generator=g) * 3).round().clamp(-7, 7)
        s = (torch.randn(*lead, 16, D // 32, generator=g) * spread).exp().mul(0.3).to(torch.bfloat16)
        parts += [n, s]
    pool = pack(*parts)
    kn, ks, vn, vs = unpack(pool)
    return pool, (kn * ks).reshape(pages, Hk, page, D), (vn * vs).reshape(pages, Hk, page, D)


def attend(q, K, V, table, lens, cu, window, sinks, scale):
    """out, lse, sum_j p_j |v_j|, and each row's largest sum_c |q_c k_jc| and largest p_j |v_jc|, all float64."""
    T, Hq, D = q.shape
    Hk, page = K.shape[1], K.shape[2]
    G = Hq // Hk
    out, mag = torch.zeros(T, Hq, D, dtype=torch.float64), torch.zeros(T, Hq, D, dtype=torch.float64)
    lse, big = torch.full((T, Hq), -math.inf, dtype=torch.float64), torch.zeros(T, Hq, dtype=torch.float64)
    top = torch.zeros(T, Hq, dtype=torch.float64)
    for b, n in enumerate(lens):
        a, e = cu[b], cu[b + 1]
        j = torch.arange(n)
        ids = torch.tensor([int(table[b][i]) for i in range(-(-n // page))], dtype=torch.long)
        k = K[ids].transpose(0, 1).reshape(Hk, -1, D)[:, :n]
        v = V[ids].transpose(0, 1).reshape(Hk, -1, D)[:, :n]
        for i in range(a, e):
            p = n - (e - a) + (i - a)
            see = j <= p
            if window:
                see &= (j > p - window) | (j < sinks)
            if not see.any():
                continue
            for h in range(Hk):
                qh = q[i, h * G:(h + 1) * G].double()
                kh, vh = k[h][see], v[h][see]
                x = qh @ kh.T * scale
                z = torch.logsumexp(x, -1)
                w = (x - z[:, None]).exp()
                out[i, h * G:(h + 1) * G] = w @ vh
                mag[i, h * G:(h + 1) * G] = w @ vh.abs()
                lse[i, h * G:(h + 1) * G] = z
                big[i, h * G:(h + 1) * G] = (qh.abs() @ kh.abs().T).amax(-1)
                top[i, h * G:(h + 1) * G] = (w * vh.abs().amax(-1)).amax(-1)
    return out, lse, mag, big, top


def attend_bounds(want, lse, mag, big, top, scale, dtype, n):
    """How far a row may be off, from what ar_kv4_attend rounds.

    A score: exact products, binary32 sums.  A chain of at most 16 partial sums (D / 16 steps, then the groups) of
    terms below sum|q k|, each rounded by at most 2^-22 of it (a tensor core may cut bits below the largest
    addend), and the row's fp16 copy of q loses less than 2^-24 of its largest element: together below
    2^-17 sum|q k|.  delta is that times the scale, plus 2^-22 |score| for the exponent's own argument.
    Weights: each is off by delta, the exponential's 2^-21 and one rounding to fp16 (2^-11); they are summed over n
    tokens in binary32 (lane by lane, at most n / 8 + 64 additions of 2^-24).  The output is rounded once.
    Where numbers get small: an fp16 weight is off by up to 2^-25 where the largest p_j s_j of its tokens stands at
    2^6 or more, so n of them with |v| <= 7 s are off by n * 7 * 2^-31 of that; and out by half its type's smallest step.
    """
    delta = big * abs(scale) * 2.0 ** -17 + (lse.abs().nan_to_num(0, 0, 0) + 10) * 2.0 ** -22
    sums = (n / 8 + 64) * 2.0 ** -24
    w = 2 * delta + 2.0 ** -20 + 2 * sums
    floor = top * n * 2.0 ** -28 + torch.finfo(dtype).tiny * torch.finfo(dtype).eps / 2
    return want.abs() * EPS[dtype] + mag * (w[..., None] + 2.0 ** -11) * 1.5 + floor[..., None], delta + sums + 2.0 ** -20


def norm_fp8(x, residual, weight, eps, group):
    """y / scale, scales and h, float64 (before the rounding to e4m3)."""
    h = x.double() + (residual.double() if residual is not None else 0)
    y = h / torch.sqrt((h * h).mean(-1, keepdim=True) + eps) * weight.double()
    q, scales = [], []
    for a in range(0, x.shape[1], group or x.shape[1]):
        part = y[:, a:a + (group or x.shape[1])]
        top = part.abs().amax(-1, keepdim=True)
        scales.append(torch.where(top > 0, top / 448, 1.0))
        q.append(part / scales[-1])
    return torch.cat(q, 1), torch.cat(scales, 1), h


def plan(lens, new, table, free, used, page, cap):
    """(code, dict) by ar_kv_plan's definition; table is a list of lists, changed only if the code is 0."""
    need, tokens, code = [], sum(new), 0
    total_pages = 0
    for b, (n, m) in enumerate(zip(lens, new)):
        if n < 0 or m < 0 or n + m > 2 ** 31 - 1:
            code = 1
            need.append(0)
            continue
        need.append(-(-(n + m) // page) - -(-n // page))
        total_pages += need[-1]
        if -(-(n + m) // page) <= len(table[b]) and m > 0 and n % page and table[b][n // page] < 0:
            code = 1
    if used < 0 or (code == 0 and used + total_pages > 2 ** 31 - 1):
        code = 1
    if code == 0 and (tokens > cap or any(-(-(n + m) // page) > len(t) for n, m, t in zip(lens, new, table))):
        code = 2
    if code == 0 and used + total_pages > len(free):
        code = 4
    if code:
        return code, dict(lens=list(lens), cu=[0] * (len(lens) + 1), slots=[-1] * cap, request=[-1] * cap,
                          position=[-1] * cap, free_used=[used], status=[code])
    out = dict(lens=[], cu=[0], slots=[], request=[], position=[], status=[0])
    at = used
    for b, (n, m) in enumerate(zip(lens, new)):
        for i in range(need[b]):
            table[b][-(-n // page) + i] = free[at]
            at += 1
        for p in range(n, n + m):
            out["slots"].append(table[b][p // page] * page + p % page)
            out["request"].append(b)
            out["position"].append(p)
        out["lens"].append(n + m)
        out["cu"].append(out["cu"][-1] + m)
    for name in ("slots", "request", "position"):
        out[name] += [-1] * (cap - tokens)
    out["free_used"] = [at]
    return 0, out
