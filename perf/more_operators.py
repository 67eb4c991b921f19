"""Cases of the operators of a decode step's feed-forward half.

  matmul   matmul_fp8           e4m3 product with a scale to 128 channels of a row and to each 128 x 128 block of the weight
  experts  experts_matmul_fp8   the same for rows grouped by expert, ragged, taken in place or gathered from the tokens
  route    route_experts        the router's choice: k experts a token, their weights, and the rows in the experts' order
  silu     silu_mul_fp8         silu(gate) * up, rounded to e4m3 with scales
  sum      experts_sum          the weighted sum of each token's rows
"""
import math

import torch

own = False  # set by whoever measures: the framework's kernels instead of the plain forms

GOLDEN = 0.6180339887498949
DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
F8 = torch.float8_e4m3fn


# ------------------------------------------------------------------ the cases

def listed():
    return [
        # The q, k and v projection of one rank of eight, 8 requests decoding.  Latency.
        dict(name="matmul_step", op="matmul", M=8, N=1280, K=8192, row_scale=False, dtype="bf16"),
        # The down projection of a larger batch, one scale a row: the weight's bytes count.
        dict(name="matmul_batch", op="matmul", M=61, N=8192, K=3584, row_scale=True, dtype="f16"),
        # A chunk of prompt.
        dict(name="matmul_chunk", op="matmul", M=8191, N=5120, K=8192, row_scale=False, dtype="bf16"),
        # 5 requests decoding with 4 of 32 experts each: gate and up of the experts, tokens gathered.
        dict(name="experts_step", op="experts", T=5, k=4, E=32, N=2048, K=4096, gather=True, dtype="bf16"),
        # A server's batch: 256 requests, 8 of 128 experts, a few rows each, all weights read.
        dict(name="experts_batch", op="experts", T=256, k=8, E=128, N=2048, K=4096, gather=True, dtype="bf16"),
        # The experts' down projection for a chunk of prompt.
        dict(name="experts_chunk", op="experts", T=4099, k=8, E=64, N=4096, K=2048, gather=False, dtype="bf16"),
        # The router of a decode step, and of a chunk with some experts switched off.
        dict(name="route_step", op="route", T=5, E=32, k=4, normalize=True, off=0, dtype="f32"),
        dict(name="route_chunk", op="route", T=8191, E=256, k=8, normalize=False, off=8, dtype="bf16"),
        # The activation of a dense layer's decode step, and of a chunk's rows by expert.
        dict(name="silu_step", op="silu", N=61, d=3584, group=0, dtype="f16"),
        dict(name="silu_chunk", op="silu", N=32767, d=1024, group=128, dtype="bf16"),
        # The experts' results of a decode step, and of a chunk.
        dict(name="sum_step", op="sum", T=5, k=4, d=4096, dtype="bf16"),
        dict(name="sum_chunk", op="sum", T=4099, k=8, d=4096, dtype="bf16"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _features(rng, lo, hi):
    """Out features: whole blocks of 128, multiples of 8, and odd ones."""
    n = _log(rng, lo, hi)
    return rng.choice([max(128, n // 128 * 128), max(128, n // 128 * 128), max(8, n // 8 * 8), n])


def _channels(rng, lo, hi):
    """Channels that are summed over: whole groups of 128, or rows of 16 bytes that end inside a group."""
    n = _log(rng, lo, hi)
    return rng.choice([max(128, n // 128 * 128), max(128, n // 128 * 128), max(16, n // 16 * 16)])


def draw(rng):
    op = rng.choice(["matmul", "matmul", "matmul", "experts", "experts", "experts", "route", "silu", "sum"])
    dtype = rng.choice(["bf16", "bf16", "f16"])
    while True:
        if op == "matmul":
            c = dict(op=op, M=_log(rng, 1, 16384), N=_features(rng, 64, 16384), K=_channels(rng, 128, 16384),
                     row_scale=rng.random() < 0.25, dtype=dtype)
            if c["M"] * c["N"] * c["K"] <= 8191 * 5120 * 8192 and c["N"] * c["K"] <= 2 ** 27:
                return c
        elif op == "experts":
            E = rng.choice([8, 16, 32, 60, 64, 128, 256])
            c = dict(op=op, T=_log(rng, 1, 8192), k=rng.choice([1, 2, 4, 6, 8]), E=E, N=_features(rng, 128, 8192),
                     K=_channels(rng, 128, 8192), gather=rng.random() < 0.5, dtype=dtype)
            if c["T"] * c["k"] * c["N"] * c["K"] <= 4099 * 8 * 4096 * 2048 and E * c["N"] * c["K"] <= 2 ** 30:
                return c
        elif op == "route":
            E = rng.choice([8, 16, 32, 60, 64, 128, 256, _log(rng, 4, 512)])
            return dict(op=op, T=_log(rng, 1, 8192), E=E, k=min(E, rng.choice([1, 2, 4, 6, 8])), normalize=rng.random() < 0.5,
                        off=rng.choice([0, 0, E // 16, E - 2]), dtype=rng.choice(["f32", "bf16", "f16"]))
        elif op == "silu":
            c = dict(op=op, N=_log(rng, 1, 32768), d=rng.choice([512, 768, 1024, 2048, 3584, 8 * _log(rng, 8, 3584)]),
                     group=rng.choice([0, 128, 128]), dtype=dtype)
            if c["N"] * c["d"] <= 2 ** 26:
                return c
        else:
            c = dict(op=op, T=_log(rng, 1, 8192), k=rng.choice([1, 2, 4, 6, 8]), d=rng.choice([1024, 2048, 4096, 5120, 8192, 8 * _log(rng, 16, 1024)]),
                     dtype=dtype)
            if c["T"] * c["k"] * c["d"] <= 4099 * 8 * 4096:
                return c


def _counts(c):
    """Rows of each expert, the most wanted first: some want many, some none; never more than a token gives once."""
    R, E, T = c["T"] * c["k"], c["E"], c["T"]
    want = [math.exp(1.5 * ((i + 1) * GOLDEN % 1.0)) for i in range(E)]
    if E >= 16:
        for i in range(0, E, 16):
            want[i] = 0.0
    live = sum(w > 0 for w in want)
    if live < c["k"]:
        want = [1.0] * E
    total = sum(want)
    n = [min(T, int(R * w / total)) for w in want]
    i = 0
    while sum(n) < R:
        if want[i % E] > 0 and n[i % E] < T:
            n[i % E] += 1
        i += 5 if E % 5 else 1
    return n


def work(c):
    if c["op"] == "matmul":
        M, N, K = c["M"], c["N"], c["K"]
        g = -(-K // 128)
        return dict(bytes=M * K + 4 * M * (1 if c["row_scale"] else g) + N * K + 4 * g * -(-N // 128) + 2 * M * N, flops=2 * M * N * K)
    if c["op"] == "experts":
        R, N, K = c["T"] * c["k"], c["N"], c["K"]
        g, live, x = -(-K // 128), sum(n > 0 for n in _counts(c)), c["T"] if c["gather"] else R
        return dict(bytes=x * (K + 4 * g) + live * (N * K + 4 * g * -(-N // 128)) + 2 * R * N + 4 * (c["E"] + 1) + (4 * R if c["gather"] else 0),
                    flops=2 * R * N * K)
    if c["op"] == "route":
        size = 4 if c["dtype"] == "f32" else 2
        return dict(bytes=c["T"] * c["E"] * size + 16 * c["T"] * c["k"] + 4 * (c["E"] + 1), flops=4 * c["T"] * c["E"])
    if c["op"] == "silu":
        n = c["N"] * c["d"]
        return dict(bytes=5 * n + 4 * c["N"] * (-(-c["d"] // c["group"]) if c["group"] else 1), flops=10 * n)
    n = c["T"] * c["d"]
    return dict(bytes=2 * n * c["k"] + 8 * c["T"] * c["k"] + 2 * n, flops=2 * n * c["k"])


# ----------------------------------------------------------------- the inputs

def _eights(g, spread, *shape):
    """Normally distributed e4m3 values, as large as a group's (a block's) scale makes them."""
    n = math.prod(shape)
    out = torch.empty(n, dtype=F8, device="cuda")
    for i in range(0, n, 1 << 27):
        m = min(1 << 27, n - i)
        out[i:i + m] = torch.randn(m, device="cuda", generator=g, dtype=torch.float16).mul_(spread).clamp_(-448, 448).to(F8)
    return out.view(*shape)


def _scales(g, size, *shape):
    return torch.randn(*shape, device="cuda", generator=g).mul_(0.3).exp_().mul_(size)


def prepare(c, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    dev, dt = "cuda", DTYPES[c["dtype"]]
    if c["op"] == "matmul":
        M, N, K = c["M"], c["N"], c["K"]
        groups = -(-K // 128)
        return dict(c=c, x=_eights(g, 170, M, K), xs=_scales(g, 0.006, M, 1 if c["row_scale"] else groups), w=_eights(g, 107, N, K),
                    ws=_scales(g, K ** -0.5 / 107, -(-N // 128), groups))
    if c["op"] == "experts":
        T, k, E, N, K = c["T"], c["k"], c["E"], c["N"], c["K"]
        R, groups = T * k, -(-K // 128)
        counts = _counts(c)
        order = torch.randperm(E, device=dev, generator=g).tolist()              # which expert is how much wanted
        counts = [counts[i] for i in order]
        offsets = torch.tensor([0] + counts, device=dev).cumsum(0).int()
        rows = None
        if c["gather"]:
            # each expert's tokens, in order, k of them to each token: dealt out round by round
            token = torch.arange(R, device=dev) % T
            turn = torch.randperm(T, device=dev, generator=g)
            expert = torch.repeat_interleave(torch.arange(E, device=dev), torch.tensor(counts, device=dev))
            rows = turn[token]
            rows = rows[torch.argsort(expert * T + rows)].int()
        X = T if c["gather"] else R
        return dict(c=c, x=_eights(g, 170, X, K), xs=_scales(g, 0.006, X, groups), w=_eights(g, 107, E, N, K),
                    ws=_scales(g, K ** -0.5 / 107, E, -(-N // 128), groups), offsets=offsets, rows=rows, counts=counts)
    if c["op"] == "route":
        T, E = c["T"], c["E"]
        bias = torch.randn(E, device=dev, generator=g)
        logits = (torch.randn(T, E, device=dev, generator=g) * 1.5 + bias).to(dt)
        if c["off"]:
            logits[:, torch.randperm(E, device=dev, generator=g)[:c["off"]]] = -math.inf
        return dict(c=c, logits=logits)
    if c["op"] == "silu":
        x = torch.randn(c["N"], 2 * c["d"], device=dev, generator=g, dtype=torch.float32)
        return dict(c=c, x=(x * 1.7).to(dt))
    T, k, d = c["T"], c["k"], c["d"]
    x = torch.randn(T * k, d, device=dev, generator=g, dtype=torch.float32).to(dt)
    weights = torch.rand(T, k, device=dev, generator=g).add_(0.05)
    weights = weights / weights.sum(1, keepdim=True)
    place = torch.randperm(T * k, device=dev, generator=g).int().view(T, k)
    return dict(c=c, x=x, weights=weights, place=place)


# ------------------------------------------------------------- the plain forms

def _wide(x, scales):
    """e4m3 rows times their scales, binary32."""
    return x.float() * scales.repeat_interleave(128, 1)[:, :x.shape[1]] if scales.shape[1] > 1 else x.float() * scales


def _wide_weight(w, scales):
    return w.float() * scales.repeat_interleave(128, 0)[:w.shape[0]].repeat_interleave(128, 1)[:, :w.shape[1]]


def _plain_matmul(s):
    return (_wide(s["x"], s["xs"]) @ _wide_weight(s["w"], s["ws"]).T).to(DTYPES[s["c"]["dtype"]])


def _plain_experts(s):
    c = s["c"]
    x, xs = s["x"], s["xs"]
    if s["rows"] is not None:
        x, xs = x.view(torch.uint8)[s["rows"].long()].view(F8), xs[s["rows"].long()]
    out = torch.empty(x.shape[0], c["N"], dtype=DTYPES[c["dtype"]], device="cuda")
    at = 0
    for e, n in enumerate(s["counts"]):
        if n:
            out[at:at + n] = (_wide(x[at:at + n], xs[at:at + n]) @ _wide_weight(s["w"][e], s["ws"][e]).T).to(out.dtype)
        at += n
    return out


def _plain_route(s):
    c, x = s["c"], s["logits"].float()
    T, E, k = c["T"], c["E"], c["k"]
    v, i = torch.sort(x, dim=1, descending=True, stable=True)
    top, ids = v[:, :k], i[:, :k]
    live = top > -math.inf
    e = torch.where(live, (top - top[:, :1]).exp(), 0.0)
    total = e.sum(1, keepdim=True) if c["normalize"] else (x - top[:, :1]).exp().sum(1, keepdim=True)
    weights = torch.where(live, e / total, 0.0)
    flat = torch.where(live, ids, E).reshape(-1)
    order = torch.sort(flat, stable=True)[1]
    count = (flat[:, None] == torch.arange(E, device="cuda")[None]).sum(0)
    offsets = torch.zeros(E + 1, dtype=torch.int32, device="cuda")
    offsets[1:] = count.cumsum(0)
    place = torch.empty_like(flat)
    place[order] = torch.arange(T * k, device="cuda")
    there = torch.arange(T * k, device="cuda") < offsets[E]
    return dict(weights=weights, experts=torch.where(live, ids, -1).int(), offsets=offsets, rows=torch.where(there, order // k, -1).int(),
                place=torch.where(live, place.view(T, k), -1).int())


def _plain_silu(s):
    c, d, x = s["c"], s["c"]["d"], s["x"].float()
    gate, up = x[:, :d], x[:, d:]
    y = gate / (1 + (-gate).exp()) * up
    group = c["group"] or d
    full = -(-d // group)
    yg = torch.nn.functional.pad(y, (0, full * group - d)).view(-1, full, group)
    scale = yg.abs().amax(-1) / 448
    scale = torch.where(scale > 0, scale, 1.0)
    return (yg / scale[..., None]).clamp(-448, 448).view(-1, full * group)[:, :d].to(F8), scale


def _plain_sum(s):
    return (s["x"][s["place"].long()].float() * s["weights"][..., None]).sum(1).to(s["x"].dtype)


def run(s):
    c = s["c"]
    if not own:
        return {"matmul": _plain_matmul, "experts": _plain_experts, "route": _plain_route, "silu": _plain_silu, "sum": _plain_sum}[c["op"]](s)
    import tensor_decode_all_gb300 as tda
    if c["op"] == "matmul":
        return tda.matmul_fp8(s["x"], s["xs"], s["w"], s["ws"], dtype=DTYPES[c["dtype"]])
    if c["op"] == "experts":
        return tda.experts_matmul_fp8(s["x"], s["xs"], s["w"], s["ws"], s["offsets"], rows=s["rows"], dtype=DTYPES[c["dtype"]])
    if c["op"] == "route":
        r = tda.route_experts(s["logits"], c["k"], normalize=c["normalize"])
        return dict(weights=r.weights, experts=r.experts, offsets=r.offsets, rows=r.rows, place=r.place)
    if c["op"] == "silu":
        return tda.silu_mul_fp8(s["x"], group=c["group"])
    return tda.experts_sum(s["x"], s["weights"], s["place"])


# ----------------------------------------------------- the definitions, 64 bits

def _exact_product(x, xs, w, ws):
    """sum over the groups g of xs[m, g] ws[n / 128, g] (x_g . w_g), in 64 bits."""
    block = torch.arange(w.shape[0], device="cuda") // 128
    out = torch.zeros(x.shape[0], w.shape[0], dtype=torch.float64, device="cuda")
    for g in range(ws.shape[1]):
        cut = slice(128 * g, min(128 * g + 128, w.shape[1]))
        left = x[:, cut].double() * xs[:, min(g, xs.shape[1] - 1)].double()[:, None]
        right = w[:, cut].double() * ws[block, g].double()[:, None]
        out.addmm_(left, right.T)
    return out


def exact(c, seed):
    s = prepare(c, seed)
    if c["op"] == "matmul":
        return _exact_product(s["x"], s["xs"], s["w"], s["ws"])
    if c["op"] == "experts":
        parts, at = [], 0
        for e, n in enumerate(s["counts"]):
            if n:
                who = torch.arange(at, at + n, device="cuda") if s["rows"] is None else s["rows"][at:at + n].long()
                parts.append(_exact_product(s["x"].view(torch.uint8)[who].view(F8), s["xs"][who], s["w"][e], s["ws"][e]))
            at += n
        return torch.cat(parts)
    if c["op"] == "route":
        x = s["logits"].double()
        chosen = torch.zeros_like(x, dtype=torch.bool)
        picked = []
        for _ in range(c["k"]):
            left = x.masked_fill(chosen, -math.inf)
            best = (left == left.amax(1, keepdim=True)).int().argmax(1, keepdim=True)      # the first of the largest
            picked.append(left.gather(1, best))
            chosen.scatter_(1, best, True)
        top = torch.cat(picked, 1)
        z = torch.logsumexp(top if c["normalize"] else x, 1, keepdim=True)
        return dict(weights=(top - z).exp(), experts=None, offsets=None, rows=None, place=None)
    if c["op"] == "silu":
        x, d = s["x"].double(), c["d"]
        y = x[:, :d] * torch.sigmoid(x[:, :d]) * x[:, d:]
        scales, parts = [], []
        for a in range(0, d, c["group"] or d):
            part = y[:, a:a + (c["group"] or d)]
            top = part.abs().amax(1, keepdim=True)
            scales.append(torch.where(top > 0, top / 448, 1.0))
            parts.append(part / scales[-1])
        return torch.cat(parts, 1), torch.cat(scales, 1)
    out = torch.zeros(c["T"], c["d"], dtype=torch.float64, device="cuda")
    for j in range(c["k"]):
        out += s["weights"][:, j, None].double() * s["x"][s["place"][:, j].long()].double()
    return out
