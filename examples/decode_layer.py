"""Attention layers of a tensor-parallel decode, on R logical ranks of one GPU.

Each rank holds its share of the heads, its own 4-bit cache and its own stream.
A step: kv_plan says where the new tokens go; then per layer and rank the
projection of the 8-bit input, kv4_append, kv4_attend, the output projection's
partial sum, the all-reduce over the ranks, and add_norm_fp8, whose output is
the next layer's input.

    python examples/decode_layer.py [--ranks 2] [--requests 6] [--layers 3] [--steps 5]

prints how far the ranks' results are from a plain float32 computation on the
same cached values, and whether all ranks hold the same bits.
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import tensor_decode_all_gb300 as tda  # noqa: E402

D, PAGE = 128, 16


class Rank:
    """One rank's weights and caches, layer by layer, and its stream."""

    def __init__(self, gen, layers, dim, heads, kv_heads, pages):
        def weight(*shape):
            return (torch.randn(*shape, device="cuda", generator=gen) * shape[0] ** -0.5).to(torch.bfloat16)
        self.heads, self.kv_heads = heads, kv_heads
        self.qkv = [weight(dim, (heads + 2 * kv_heads) * D) for _ in range(layers)]
        self.out = [weight(heads * D, dim) for _ in range(layers)]
        self.pools = [tda.kv4_pool(pages, kv_heads, D, PAGE) for _ in range(layers)]
        self.stream = torch.cuda.Stream()


def layer(ranks, handle, norm, i, plan, table, xs, residuals, window=0, sinks=0):
    """Layer i of one step.  xs[r]: (e4m3 rows, scales) and residuals[r], on rank r's stream; returns the next ones."""
    partial, sums = [], []
    for rank, (x8, scale) in zip(ranks, xs):
        with torch.cuda.stream(rank.stream):
            x = (x8.to(torch.bfloat16) * scale).to(torch.bfloat16)
            qkv = (x @ rank.qkv[i]).view(len(x), -1, D)
            q, k, v = qkv.split((rank.heads, rank.kv_heads, rank.kv_heads), 1)
            tda.kv4_append(k, v, rank.pools[i], plan.slots)
            o = tda.kv4_attend(q, rank.pools[i], table, plan.lens, plan.cu, max_new=len(x), window=window, sinks=sinks)
            partial.append(o.view(len(x), -1) @ rank.out[i])
            sums.append(torch.empty_like(partial[-1]))
    handle.allreduce_each(partial, sums, [r.stream for r in ranks])
    nxt, after = [], []
    for rank, total, residual in zip(ranks, sums, residuals):
        with torch.cuda.stream(rank.stream):
            y, scale, h = tda.add_norm_fp8(total, norm[i], residual=residual)
            nxt.append((y, scale))
            after.append(h)
    return nxt, after


def plain_layer(ranks, norm, i, plan, table, x, residual, window=0, sinks=0):
    """The same in float32, over the values that the caches hold."""
    total = 0
    x = (x[0].float() * x[1]).to(torch.bfloat16).float()
    lens, cu = plan.lens.tolist(), plan.cu.tolist()
    for rank in ranks:
        qkv = (x @ rank.qkv[i].float()).to(torch.bfloat16).float().view(len(x), -1, D)
        rows = []
        for b, n in enumerate(lens):
            j = torch.arange(n, device="cuda")
            k, v = (t.float() for t in tda.kv4_load(rank.pools[i], table[b, j // PAGE].long() * PAGE + j % PAGE))
            for t in range(cu[b], cu[b + 1]):
                p = n - (cu[b + 1] - cu[b]) + t - cu[b]
                see = (j <= p) & ((j > p - window) | (j < sinks) if window else j >= 0)
                q = qkv[t, :rank.heads].view(rank.kv_heads, -1, D)
                w = (torch.einsum("hgd,lhd->hgl", q, k) * D ** -0.5).masked_fill(~see, -torch.inf).softmax(-1)
                rows.append(torch.einsum("hgl,lhd->hgd", w, v).reshape(-1))
        total = total + torch.stack(rows).to(torch.bfloat16).float() @ rank.out[i].float()
    h = total + residual.float()
    y = h * torch.rsqrt(h.square().mean(-1, keepdim=True) + 1e-6) * norm[i].float()
    return y, h


def main(argv=None):
    ap = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    for name, value in (("ranks", 2), ("requests", 6), ("layers", 3), ("steps", 5), ("dim", 1024), ("heads", 16), ("kv-heads", 4),
                        ("window", 24), ("sinks", 2)):
        ap.add_argument("--" + name, type=int, default=value)
    a = ap.parse_args(argv)
    tda.build()
    gen = torch.Generator(device="cuda").manual_seed(7)
    B, prompt = a.requests, [1 + 11 * b for b in range(a.requests)]
    width = -(-(max(prompt) + a.steps) // PAGE)
    ranks = [Rank(gen, a.layers, a.dim, a.heads // a.ranks, a.kv_heads // a.ranks, B * width) for _ in range(a.ranks)]
    norm = [torch.ones(a.dim, device="cuda", dtype=torch.bfloat16) for _ in range(a.layers)]
    table = torch.full((B, width), -1, dtype=torch.int32, device="cuda")
    free = torch.randperm(B * width, device="cuda", generator=gen).int()
    lens, used = torch.zeros(B, dtype=torch.int32, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")
    most = max(sum(prompt), B)
    worst, same = 0.0, True
    with tda.Handle(a.ranks, torch.bfloat16, most * a.dim, "hbm") as handle:
        for step in range(a.steps):
            # the prompts first, one token a request from then on
            new = torch.tensor(prompt if step == 0 else [1] * B, dtype=torch.int32, device="cuda")
            plan = tda.kv_plan(lens, new, table, free, used, page=PAGE, max_tokens=int(new.sum()))
            plan.check()
            lens, used = plan.lens, plan.free_used
            hidden = torch.randn(int(new.sum()), a.dim, device="cuda", generator=gen).to(torch.bfloat16)
            x0 = tda.add_norm_fp8(hidden, norm[0])
            xs, residuals = [x0[:2]] * a.ranks, [hidden] * a.ranks
            torch.cuda.synchronize()
            for i in range(a.layers):
                window, sinks = (a.window, a.sinks) if i % 2 else (0, 0)      # every other layer has a window
                before, residual = xs[0], residuals[0]
                xs, residuals = layer(ranks, handle, norm, i, plan, table, xs, residuals, window, sinks)
                torch.cuda.synchronize()
                y, h = plain_layer(ranks, norm, i, plan, table, before, residual, window, sinks)
                worst = max(worst, ((residuals[0].float() - h).norm() / h.norm()).item(),
                            ((xs[0][0].float() * xs[0][1] - y).norm() / y.norm()).item())
                same &= all(torch.equal(xs[0][0].view(torch.uint8), x[0].view(torch.uint8)) and torch.equal(residuals[0], r)
                            for x, r in zip(xs, residuals))
        handle.check()
        for workspace in tda.kv4_workspaces():
            workspace.check()
    print(f"{a.steps} steps of {a.layers} layers on {a.ranks} ranks: relative distance from float32 at most {worst:.2g}, "
          f"all ranks {'the same' if same else 'NOT the same'}")
    return worst, same


if __name__ == "__main__":
    main()
