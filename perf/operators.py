"""Cases of the operators around the all-reduce of a decode step.

  plan    kv_plan                    where the new tokens go: block tables, slot maps
  append  kv4_append, kv4_load       K and V rows into the 4-bit paged cache, and back as values
  attend  kv4_attend                 attention over that cache, with or without a window and sinks
  norm    add_norm_fp8               residual, RMS norm, e4m3 output with scales

The cache ("pool") is uint8 [pages, kv heads, page / 16, 18 * D].  The last axis is a tile of 16 tokens of one head:
K nibbles (8 D bytes), V nibbles (8 D), K scales (bf16 [16][D / 32]) and V scales (the same).  A nibble holds n + 8 and
stands for n * scale, one scale to 32 channels.  K nibbles are ordered [token][t 4][group][i 8] with channel
32 * group + 8 * t + i; V nibbles [half 2][g 8][t 4][group][odd 2][i 4] with token 8 * half + 2 * t + odd and channel
32 * group + 4 * g + i; of a byte's two nibbles the low one comes first.
"""
import math

import torch

own = False  # set by whoever measures: the framework's kernels instead of the plain forms

GOLDEN = 0.6180339887498949
DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16}


# ------------------------------------------------------------------ the cases

def listed():
    return [
        # One chat on one rank of eight: 1 kv head, one new token.  Latency.
        dict(name="attend_one", op="attend", B=1, lo=1003, hi=1003, q=1, Hk=1, G=8, D=128, page=16, window=0, sinks=0, dtype="bf16"),
        # An ordinary decode step of a server: ragged contexts.
        dict(name="attend_batch", op="attend", B=64, lo=517, hi=8001, q=1, Hk=8, G=8, D=128, page=16, window=0, sinks=0, dtype="bf16"),
        # One very long document.
        dict(name="attend_long", op="attend", B=1, lo=262139, hi=262139, q=1, Hk=8, G=4, D=128, page=64, window=0, sinks=0, dtype="f16"),
        # Layers with a sliding window and sinks, long contexts, heads of 64.
        dict(name="attend_window", op="attend", B=128, lo=301, hi=16001, q=1, Hk=8, G=8, D=64, page=32, window=1024, sinks=4, dtype="bf16"),
        # Drafted tokens checked in one pass: 1 to 6 new tokens a request, 6 heads to a kv head.
        dict(name="attend_verify", op="attend", B=24, lo=777, hi=9000, q=6, Hk=4, G=6, D=128, page=16, window=0, sinks=0, dtype="bf16"),
        # A full card: 64 requests of up to 32 Ki tokens.
        dict(name="attend_large", op="attend", B=64, lo=16385, hi=32768, q=1, Hk=8, G=8, D=128, page=64, window=0, sinks=0, dtype="bf16"),
        # The cache write of a decode step, and of a chunk of prompt.
        dict(name="append_step", op="append", T=64, runs=64, Hk=8, G=8, D=128, page=16, dtype="bf16"),
        dict(name="append_chunk", op="append", T=8191, runs=5, Hk=8, G=4, D=128, page=64, dtype="bf16"),
        # The plan of a decode step, and of one that mixes decode with chunks of prompt.
        dict(name="plan_step", op="plan", B=64, lo=1, hi=8000, new=1, big=0, page=16),
        dict(name="plan_mixed", op="plan", B=1000, lo=0, hi=16000, new=1, big=2049, page=16),
        # After the all-reduce of a decode step: one scale a row.  And of a chunk: one scale to 128 channels.
        dict(name="norm_step", op="norm", N=8, d=8192, group=0, dtype="bf16"),
        dict(name="norm_chunk", op="norm", N=8192, d=5120, group=128, dtype="f16"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["attend", "attend", "attend", "attend", "append", "append", "plan", "norm", "norm"])
    dtype = rng.choice(["bf16", "bf16", "f16"])
    if op == "attend":
        while True:
            c = dict(op=op, B=_log(rng, 1, 128), lo=0, hi=_log(rng, 20, 262144), q=rng.choice([1, 1, 1, 2, 3, 5, 8]),
                     Hk=rng.choice([1, 2, 4, 8]), G=rng.choice([1, 2, 4, 5, 6, 8, 8, 16]), D=rng.choice([64, 128, 128]),
                     page=rng.choice([16, 32, 64]), window=0, sinks=0, dtype=dtype)
            c["lo"] = max(c["q"], int(c["hi"] * rng.uniform(0.05, 1.0)))
            c["hi"] = max(c["hi"], c["lo"])
            if rng.random() < 0.35:
                c["window"], c["sinks"] = _log(rng, 100, 4096), rng.choice([0, 1, 4, 16])
            # no more than the largest listed case, also in what the plain form reads
            if c["B"] * c["hi"] * c["Hk"] * c["D"] <= 64 * 28000 * 8 * 128:
                return c
    if op == "append":
        T = _log(rng, 1, 16384)
        return dict(op=op, T=T, runs=rng.choice([1, max(1, T // 300), max(1, T // 7), T]), Hk=rng.choice([1, 2, 4, 8]),
                    G=rng.choice([1, 4, 8]), D=rng.choice([64, 128, 128]), page=rng.choice([16, 32, 64]), dtype=dtype)
    if op == "plan":
        return dict(op=op, B=_log(rng, 1, 2048), lo=0, hi=_log(rng, 50, 32768), new=rng.choice([1, 1, 4]),
                    big=rng.choice([0, 0, _log(rng, 100, 4096)]), page=rng.choice([16, 32, 64]))
    while True:
        c = dict(op=op, N=_log(rng, 1, 16384), d=rng.choice([1024, 2048, 4096, 5120, 6144, 8192, 12288, _log(rng, 64, 16384)]),
                 group=rng.choice([0, 128]), dtype=dtype)
        if c["N"] * c["d"] <= 2 ** 27:
            return c


def _spread(n, lo, hi):
    """n whole numbers spread over [lo, hi], ragged, the same for every seed."""
    return [lo + int((hi - lo) * ((i + 1) * GOLDEN % 1.0) + 0.5) for i in range(n)]


def _new_tokens(c):
    """New tokens of each request of an attend case: 1 .. q, the largest among them."""
    return [c["q"] - i % c["q"] for i in range(c["B"])]


def _plan_new(c):
    """New tokens of each request of a plan case: `new`, every 97th request a chunk, every 31st idle."""
    return [c["big"] if c["big"] and i % 97 == 3 else 0 if i % 31 == 30 else c["new"] for i in range(c["B"])]


def _visible(c):
    """(tokens that some row of the request sees, sum over its new tokens of those each sees) for each request."""
    out = []
    for n, q in zip(_spread(c["B"], c["lo"], c["hi"]), _new_tokens(c)):
        seen, first = 0, n
        for p in range(n - q, n):
            low = max(0, p - c["window"] + 1) if c["window"] else 0
            seen += p - low + 1 + min(c["sinks"], low)
            first = min(first, low)
        out.append((n - first + min(c["sinks"], first), seen))
    return out


def work(c):
    if c["op"] == "attend":
        rows, heads = sum(_new_tokens(c)), c["Hk"] * c["G"]
        vis = _visible(c)
        cache = sum(u for u, _ in vis) * c["Hk"] * (c["D"] + c["D"] // 8)
        return dict(bytes=cache + rows * heads * (c["D"] * 4 + 4) + 4 * sum(-(-u // c["page"]) for u, _ in vis),
                    flops=4 * c["D"] * heads * sum(s for _, s in vis))
    if c["op"] == "append":
        n = c["T"] * c["Hk"] * c["D"]
        return dict(bytes=2 * (2 * n + n * 9 // 16) * 2 + 16 * c["T"], flops=8 * n)
    if c["op"] == "plan":
        new = _plan_new(c)
        cap, B = max(1, sum(new)), c["B"]
        return dict(bytes=12 * B + 16 * cap + 8 * (cap // c["page"]) + 4 * B, flops=10 * (B + cap))
    n = c["N"] * c["d"]
    return dict(bytes=7 * n + 2 * c["d"] + 4 * c["N"] * (-(-c["d"] // c["group"]) if c["group"] else 1), flops=9 * n)


# ----------------------------------------------------------------- the inputs

def _random_tiles(shape, D, g):
    """Tiles of a cache that holds normally distributed K and V: nibbles and scales of groups of 32."""
    n = math.prod(shape)
    tiles = torch.empty(n, 18 * D, dtype=torch.uint8, device="cuda")
    step = max(1, (1 << 27) // (16 * D))
    for i in range(0, n, step):
        m = min(step, n - i)
        x = torch.randn(m, 16 * D, 2, device="cuda", generator=g, dtype=torch.float16)
        x = (x * 3.2).round_().clamp_(-7, 7).add_(8).to(torch.uint8)
        tiles[i:i + m, :16 * D] = x[..., 0] | (x[..., 1] << 4)
        s = torch.randn(m, D, device="cuda", generator=g).mul_(0.25).exp_().mul_(0.3)
        tiles[i:i + m, 16 * D:] = s.to(torch.bfloat16).view(torch.uint8)
    return tiles.view(*shape, 18 * D)


def prepare(c, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    dev = "cuda"
    if c["op"] == "norm":
        dt, d = DTYPES[c["dtype"]], c["d"]
        big = 1 + 12 * (torch.rand(d, device=dev, generator=g) < 0.004)   # a few channels run large, as in trained models
        x = (torch.randn(c["N"], d, device=dev, generator=g) * 0.3).to(dt)
        r = (torch.randn(c["N"], d, device=dev, generator=g) * big).to(dt)
        w = (1 + 0.2 * torch.randn(d, device=dev, generator=g)).to(dt)
        return dict(c=c, x=x, residual=r, weight=w)
    if c["op"] == "plan":
        B, P = c["B"], c["page"]
        lens = torch.randint(c["lo"], c["hi"] + 1, (B,), device=dev, generator=g).int()
        new = torch.tensor(_plan_new(c), dtype=torch.int32, device=dev)
        width = -(-(c["hi"] + max(c["new"], c["big"])) // P)
        cap = max(1, sum(_plan_new(c)))
        pages = B * width + 64
        perm = torch.randperm(pages, device=dev, generator=g).int()
        table = torch.where(torch.arange(width, device=dev)[None] * P < lens[:, None], perm[:B * width].view(B, width), -1)
        free = torch.randperm(cap // P + B + 8, device=dev, generator=g).int() + pages
        used = torch.randint(0, 4, (1,), device=dev, generator=g).int()
        return dict(c=c, lens=lens, new=new, table=table.int().contiguous(), free=free, used=used, cap=cap)
    Hk, D, P, dt = c["Hk"], c["D"], c["page"], DTYPES[c["dtype"]]
    if c["op"] == "append":
        T, heads = c["T"], c["Hk"] * (c["G"] + 2)
        qkv = torch.randn(T, heads, D, device=dev, generator=g).to(dt)     # what the projection gives: q, k and v side by side
        cuts = [T * i // c["runs"] for i in range(c["runs"] + 1)]
        at = torch.arange(T, device=dev)
        run_of = torch.searchsorted(torch.tensor(cuts[1:], device=dev), at, right=True)
        start = torch.randint(0, P, (c["runs"],), device=dev, generator=g)
        position = at - torch.tensor(cuts, device=dev)[run_of] + start[run_of]
        width = -(-(max(b - a for a, b in zip(cuts, cuts[1:])) + P) // P)
        table = torch.randperm(c["runs"] * width, device=dev, generator=g).view(c["runs"], width)
        slots = table[run_of, position // P] * P + position % P
        pool = _random_tiles((c["runs"] * width, Hk, P // 16), D, g)
        return dict(c=c, k=qkv[:, Hk * c["G"]:Hk * (c["G"] + 1)], v=qkv[:, Hk * (c["G"] + 1):], slots=slots, pool=pool)
    lens, new = _spread(c["B"], c["lo"], c["hi"]), _new_tokens(c)
    width = -(-max(lens) // P)
    need = [-(-n // P) for n in lens]
    perm = torch.randperm(sum(need), device=dev, generator=g).int()
    ends = torch.tensor(need, device=dev).cumsum(0)
    col = torch.arange(width, device=dev)[None]
    first = (ends - torch.tensor(need, device=dev))[:, None]
    table = torch.where(col < (ends[:, None] - first), perm[(first + col).clamp(max=sum(need) - 1)], -1).int().contiguous()
    pool = _random_tiles((sum(need), Hk, P // 16), D, g)
    q = torch.randn(sum(new), Hk * c["G"], D, device=dev, generator=g).to(dt)
    cu = torch.tensor([0] + new, device=dev).cumsum(0).int()
    return dict(c=c, q=q, pool=pool, table=table, lens=torch.tensor(lens, dtype=torch.int32, device=dev), cu=cu, most=max(new))


# ------------------------------------------------------------- the plain forms

def _nibbles(b):
    return torch.stack((b & 15, b >> 4), -1)


def _tiles_to_values(tiles, D):
    """uint8 [..., 18 D] -> K and V, float32 [..., 16, D]."""
    lead, G = tiles.shape[:-1], D // 32
    ks = tiles[..., 16 * D:17 * D].contiguous().view(torch.bfloat16).view(*lead, 16, G, 1).float()
    vs = tiles[..., 17 * D:].contiguous().view(torch.bfloat16).view(*lead, 16, G, 1).float()
    n = len(lead)
    k = _nibbles(tiles[..., :8 * D]).view(*lead, 16, 4, G, 8)
    k = k.transpose(n + 1, n + 2).reshape(*lead, 16, G, 32).float().sub_(8).mul_(ks).view(*lead, 16, D)
    v = _nibbles(tiles[..., 8 * D:16 * D]).view(*lead, 2, 8, 4, G, 2, 4)
    v = v.permute(*range(n), n, n + 2, n + 4, n + 3, n + 1, n + 5).reshape(*lead, 16, G, 32)
    return k, v.float().sub_(8).mul_(vs).view(*lead, 16, D)


def _plain_attend(s):
    c, q, lens, cu = s["c"], s["q"], s["lens"].long(), s["cu"].long()
    B, Hk, G, D, P, most = c["B"], c["Hk"], c["G"], c["D"], c["page"], s["most"]
    k, v = _tiles_to_values(s["pool"][s["table"].clamp(min=0).long()].transpose(1, 2), D)   # [B, Hk, W, P / 16, 16, D]
    L = s["table"].shape[1] * P
    k, v = k.reshape(B, Hk, L, D), v.reshape(B, Hk, L, D)
    count = cu[1:] - cu[:-1]
    i = torch.arange(most, device="cuda")
    at = (cu[:-1, None] + i).clamp(max=q.shape[0] - 1)                                       # [B, most]
    qp = q[at].float().view(B, most, Hk, G, D).permute(0, 2, 1, 3, 4).reshape(B, Hk, most * G, D)
    p = (lens - count)[:, None] + i
    j = torch.arange(L, device="cuda")
    seen = j <= p[..., None]
    if c["window"]:
        seen &= (j > p[..., None] - c["window"]) | (j < c["sinks"])
    seen = seen[:, None, :, None, :].expand(B, 1, most, G, L).reshape(B, 1, most * G, L)
    v = torch.where(j[:, None] < lens[:, None, None, None], v, 0.0)
    x = torch.matmul(qp, k.transpose(2, 3)).mul_(D ** -0.5).masked_fill_(~seen, -math.inf)
    m = x.amax(-1, keepdim=True).clamp(min=-3e38)
    x = x.sub_(m).exp_()
    l = x.sum(-1, keepdim=True)
    o = torch.matmul(x, v) / l.clamp(min=1e-37)
    lse = (m + l.log()).view(B, Hk, most, G)
    o = o.view(B, Hk, most, G, D)
    t = torch.arange(q.shape[0], device="cuda")
    b = torch.searchsorted(cu[1:].contiguous(), t, right=True)
    i = t - cu[b]
    return o[b, :, i].reshape(-1, Hk * G, D).to(q.dtype), lse[b, :, i].reshape(-1, Hk * G)


def _plain_quantise(x):
    """float32 [..., D] -> nibbles (n + 8) and bfloat16 scales."""
    x = x.view(*x.shape[:-1], -1, 32)
    s = (x.abs().amax(-1, keepdim=True) / 7).to(torch.bfloat16)
    n = torch.where(s == 0, 0.0, (x / s.float()).round().clamp(-7, 7)).nan_to_num(0.0)
    return (n + 8).to(torch.uint8).flatten(-2), s.squeeze(-1)


def _plain_append(s):
    c, pool, slots = s["c"], s["pool"], s["slots"]
    D, P, G, dev = c["D"], c["page"], c["D"] // 32, "cuda"
    kn, ks = _plain_quantise(s["k"].float())
    vn, vs = _plain_quantise(s["v"].float())
    page, r = slots // P, slots % 16
    tile = slots % P // 16
    page, tile, head = page[:, None, None], tile[:, None, None], torch.arange(c["Hk"], device=dev)[None, :, None]
    # K: a token's D / 2 bytes lie side by side
    kn = kn.view(-1, c["Hk"], G, 4, 8).transpose(2, 3).reshape(-1, c["Hk"], D)
    pool[page, head, tile, r[:, None, None] * (D // 2) + torch.arange(D // 2, device=dev)] = kn[..., ::2] | (kn[..., 1::2] << 4)
    # V: two bytes for each g and group
    vn = vn.view(-1, c["Hk"], G, 8, 4).transpose(2, 3).reshape(-1, c["Hk"], D)
    g, j, e = torch.meshgrid(torch.arange(8, device=dev), torch.arange(G, device=dev), torch.arange(2, device=dev), indexing="ij")
    half, t, odd = (x[:, None, None] for x in (r // 8, r % 8 // 2, r % 2))
    at = 8 * D + 4 * ((half * 32 + g.reshape(-1) * 4 + t) * G + j.reshape(-1)) + 2 * odd + e.reshape(-1)
    pool[page, head, tile, at] = vn[..., ::2] | (vn[..., 1::2] << 4)
    at = 16 * D + r[:, None, None] * 2 * G + torch.arange(2 * G, device=dev)
    pool[page, head, tile, at] = ks.contiguous().view(torch.uint8)
    pool[page, head, tile, at + D] = vs.contiguous().view(torch.uint8)
    # and back
    k, v = _tiles_to_values(pool[slots // P, :, slots % P // 16], D)
    at = r[:, None, None, None].expand(-1, c["Hk"], 1, D)
    return k.gather(2, at).squeeze(2).to(s["k"].dtype), v.gather(2, at).squeeze(2).to(s["v"].dtype)


def _plain_plan(s):
    c, lens, new, table, P = s["c"], s["lens"].long(), s["new"].long(), s["table"], s["c"]["page"]
    cu = torch.zeros(c["B"] + 1, dtype=torch.int64, device="cuda")
    cu[1:] = new.cumsum(0)
    had = (lens + P - 1) // P
    need = (lens + new + P - 1) // P - had
    first = need.cumsum(0) - need
    col = torch.arange(table.shape[1], device="cuda")[None]
    fresh = (col >= had[:, None]) & (col < (had + need)[:, None])
    at = (s["used"] + first[:, None] + col - had[:, None]).clamp(0, s["free"].numel() - 1)
    table.copy_(torch.where(fresh, s["free"][at.long()], table))
    t = torch.arange(s["cap"], device="cuda")
    b = torch.searchsorted(cu[1:].contiguous(), t, right=True)
    live = b < c["B"]
    b = b.clamp(max=c["B"] - 1)
    p = lens[b] + t - cu[b]
    page = table[b, (p // P).clamp(max=table.shape[1] - 1)].long()
    return dict(lens=(lens + new).int(), cu=cu.int(), slots=torch.where(live, page * P + p % P, -1),
                request=torch.where(live, b, -1).int(), position=torch.where(live, p, -1).int(),
                free_used=(s["used"] + need.sum()).int(), status=torch.zeros(1, dtype=torch.int32, device="cuda"), table=table)


def _plain_norm(s):
    c, d = s["c"], s["c"]["d"]
    h = s["x"].float() + s["residual"].float()
    y = h * torch.rsqrt(h.square().mean(-1, keepdim=True) + 1e-6) * s["weight"].float()
    group = c["group"] or d
    full = -(-d // group)
    yg = torch.nn.functional.pad(y, (0, full * group - d)).view(-1, full, group)
    scale = yg.abs().amax(-1) / 448
    scale = torch.where(scale > 0, scale, 1.0)
    out = (yg / scale[..., None]).clamp(-448, 448).view(-1, full * group)[:, :d].to(torch.float8_e4m3fn)
    return out, scale, h.to(s["x"].dtype)


def run(s):
    c = s["c"]
    if not own:
        return {"attend": _plain_attend, "append": _plain_append, "plan": _plain_plan, "norm": _plain_norm}[c["op"]](s)
    import tensor_decode_all_gb300 as tda
    if c["op"] == "attend":
        return tda.kv4_attend(s["q"], s["pool"], s["table"], s["lens"], s["cu"], max_new=s["most"], window=c["window"],
                              sinks=c["sinks"], return_lse=True)
    if c["op"] == "append":
        tda.kv4_append(s["k"], s["v"], s["pool"], s["slots"])
        return tda.kv4_load(s["pool"], s["slots"], s["k"].dtype)
    if c["op"] == "plan":
        p = tda.kv_plan(s["lens"], s["new"], s["table"], s["free"], s["used"], page=c["page"], max_tokens=s["cap"])
        return dict(lens=p.lens, cu=p.cu, slots=p.slots, request=p.request, position=p.position, free_used=p.free_used,
                    status=p.status, table=s["table"])
    return tda.add_norm_fp8(s["x"], s["weight"], residual=s["residual"], eps=1e-6, group=c["group"])


# ----------------------------------------------------- the definitions, 64 bits

def _cell(pool, page, tile, D, token, channel, values):
    """One value of the cache by its address: tokens and channels broadcast against each other."""
    G, j, r = D // 32, channel // 32, token % 16
    if values == "k":
        word, i, base = (r * 4 + channel % 32 // 8) * G + j, channel % 8, 0
    else:
        word, i, base = (r // 8 * 32 + channel % 32 // 4 * 4 + r % 8 // 2) * G + j, r % 2 * 4 + channel % 4, 8 * D
    byte = pool[page, :, tile, base + 4 * word + i // 2].long()             # [..., Hk]
    n = (byte >> (4 * (i % 2)).unsqueeze(-1)) % 16 - 8
    at = (16 * D if values == "k" else 17 * D) + 2 * (r * G + j)
    bits = pool[page, :, tile, at].int() | (pool[page, :, tile, at + 1].int() << 8)
    return n.double() * (bits << 16).view(torch.float32).double()


def _exact_attend(c, s):
    D, P, G, out, sums = c["D"], c["page"], c["G"], [], []
    channel = torch.arange(D, device="cuda")[None, :]
    for b, n in enumerate(s["lens"].tolist()):
        a, e = s["cu"][b].item(), s["cu"][b + 1].item()
        low = max(0, n - (e - a) - c["window"] + 1) if c["window"] else 0
        token = torch.arange(low, n, device="cuda")
        if low:
            token = torch.cat((torch.arange(min(low, c["sinks"]), device="cuda"), token))
        token = token[:, None]
        page, tile = s["table"][b].long()[token // P], token % P // 16
        k, v = (_cell(s["pool"], page, tile, D, token, channel, w) for w in "kv")            # [L, D, Hk]
        q = s["q"][a:e].double().view(e - a, c["Hk"], G, D)
        x = torch.einsum("qhgd,ldh->qhgl", q, k) / math.sqrt(D)
        p = torch.arange(n - (e - a), n, device="cuda")[:, None]
        hidden = token.T > p
        if c["window"]:
            hidden |= (token.T <= p - c["window"]) & (token.T >= c["sinks"])
        x = x.masked_fill(hidden[:, None, None, :], -math.inf)
        z = torch.logsumexp(x, -1, keepdim=True)
        out.append(torch.einsum("qhgl,ldh->qhgd", (x - z).exp(), v).reshape(e - a, -1, D))
        sums.append(z.reshape(e - a, -1))
    return torch.cat(out), torch.cat(sums)


def _exact_rows(x):
    x = x.double().view(*x.shape[:2], -1, 32)
    top = (x.abs().amax(-1, keepdim=True) / 7).clamp(min=1e-300)
    m, _ = torch.frexp(top)
    s = torch.round(m * 256) / 256 * (top / m)                             # to 8 bits, ties to even; top / m is a power of two
    return (torch.round(x / s).clamp(-7, 7) * s).flatten(-2)


def exact(c, seed):
    if c["op"] == "attend" and sum(_spread(c["B"], c["lo"], c["hi"])) * c["Hk"] * c["D"] > 2 ** 31:
        return None  # the gather by cells takes too long
    s = prepare(c, seed)
    if c["op"] == "attend":
        return _exact_attend(c, s)
    if c["op"] == "append":
        return _exact_rows(s["k"]), _exact_rows(s["v"])
    if c["op"] == "plan":
        return None  # whole numbers
    h = s["x"].double() + s["residual"].double()
    y = h / torch.sqrt((h * h).mean(1, keepdim=True) + 1e-6) * s["weight"].double()
    scales, parts = [], []
    for a in range(0, c["d"], c["group"] or c["d"]):
        part = y[:, a:a + (c["group"] or c["d"])]
        top = part.abs().amax(1, keepdim=True)
        scales.append(torch.where(top > 0, top / 448, 1.0))
        parts.append(part / scales[-1])
    return torch.cat(parts, 1), torch.cat(scales, 1), h
