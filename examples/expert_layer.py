"""Layers with experts of a tensor-parallel decode, on R logical ranks of one GPU.

Each rank holds its share of every expert's inner channels and its own stream.  A layer: the 8-bit input goes
through the router, whose choice is the same on all ranks; per rank the experts' gate and up products for the tokens that
chose them, the activation (8-bit again), the down products and their weighted sum, a partial sum of the layer's output; the
all-reduce over the ranks; and add_norm_fp8, whose output is the next layer's input.

    python examples/expert_layer.py [--ranks 2] [--tokens 5] [--experts 16] [--chosen 4] [--layers 3]

prints how far the ranks' results are from a plain float32 computation with the same 8-bit weights, and whether all
ranks hold the same bits.
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import tensor_decode_all_gb300 as tda  # noqa: E402

F8 = torch.float8_e4m3fn


def blocks_fp8(w):
    """A weight [..., features, channels] as e4m3, one scale to a block of 128 x 128: (w8, scales)."""
    *lead, n, k = w.shape
    rows, cols = -(-n // 128), -(-k // 128)
    padded = torch.nn.functional.pad(w.float(), (0, cols * 128 - k, 0, rows * 128 - n))
    tiles = padded.view(*lead, rows, 128, cols, 128)
    scales = tiles.abs().amax((-3, -1)) / 448
    scales = torch.where(scales > 0, scales, 1.0)
    w8 = (tiles / scales[..., :, None, :, None]).reshape(*lead, rows * 128, cols * 128)[..., :n, :k].to(F8)
    return w8.contiguous(), scales.contiguous()


def widened(w8, scales):
    wide = scales.repeat_interleave(128, -2).repeat_interleave(128, -1)
    return w8.float() * wide[..., :w8.shape[-2], :w8.shape[-1]]


class Rank:
    """One rank's share of the layers' experts, and its stream."""

    def __init__(self, gen, layers, experts, dim, inner):
        def weight(n, k):
            return blocks_fp8(torch.randn(experts, n, k, device="cuda", generator=gen) * k ** -0.5)
        self.gate_up = [weight(2 * inner, dim) for _ in range(layers)]
        self.down = [weight(dim, inner) for _ in range(layers)]
        self.stream = torch.cuda.Stream()


def layer(ranks, handle, norm, router, i, chosen, xs, residuals):
    """Layer i.  xs[r]: (e4m3 rows, scales) and residuals[r], on rank r's stream; returns the next ones and the routes."""
    partial, sums, routes = [], [], []
    for rank, (x8, scale), h in zip(ranks, xs, residuals):
        with torch.cuda.stream(rank.stream):
            r = tda.route_experts(h.float() @ router[i], chosen)
            y = tda.experts_matmul_fp8(x8, scale, *rank.gate_up[i], r.offsets, rows=r.rows)
            y8, ys = tda.silu_mul_fp8(y)
            y = tda.experts_matmul_fp8(y8, ys, *rank.down[i], r.offsets)
            partial.append(tda.experts_sum(y, r.weights, r.place))
            sums.append(torch.empty_like(partial[-1]))
            routes.append(r)
    # (one launch of all ranks: products of many rows take whole multiprocessors, and a rank that waited for another's on all of
    # them would keep it from running)
    handle.allreduce_all(partial, sums, [r.stream for r in ranks])
    nxt, after = [], []
    for rank, total, residual in zip(ranks, sums, residuals):
        with torch.cuda.stream(rank.stream):
            y, scale, h = tda.add_norm_fp8(total, norm[i], residual=residual, group=128)
            nxt.append((y, scale))
            after.append(h)
    return nxt, after, routes


def plain_layer(ranks, norm, i, x, residual, route):
    """The same in float32, with the 8-bit weights and the experts that were chosen."""
    wide = x[0].float() * x[1].repeat_interleave(128, 1)[:, :x[0].shape[1]]
    total = torch.zeros_like(wide)
    for rank in ranks:
        gate_up, down = widened(*rank.gate_up[i]), widened(*rank.down[i])
        for t in range(len(wide)):
            for j, e in enumerate(route.experts[t].tolist()):
                if e >= 0:
                    gate, up = (gate_up[e] @ wide[t]).chunk(2)
                    total[t] += route.weights[t, j] * (down[e] @ (torch.nn.functional.silu(gate) * up))
    h = total + residual.float()
    return h * torch.rsqrt(h.square().mean(-1, keepdim=True) + 1e-6) * norm[i].float(), h, total


def main(argv=None):
    ap = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    for name, value in (("ranks", 2), ("tokens", 5), ("experts", 16), ("chosen", 4), ("layers", 3), ("dim", 512), ("inner", 256)):
        ap.add_argument("--" + name, type=int, default=value)
    a = ap.parse_args(argv)
    tda.build()
    gen = torch.Generator(device="cuda").manual_seed(11)
    ranks = [Rank(gen, a.layers, a.experts, a.dim, a.inner // a.ranks) for _ in range(a.ranks)]
    norm = [torch.ones(a.dim, device="cuda", dtype=torch.bfloat16) for _ in range(a.layers)]
    router = [torch.randn(a.dim, a.experts, device="cuda", generator=gen) * a.dim ** -0.5 for _ in range(a.layers)]
    hidden = torch.randn(a.tokens, a.dim, device="cuda", generator=gen).to(torch.bfloat16)
    worst, same = 0.0, True
    with tda.Handle(a.ranks, torch.bfloat16, a.tokens * a.dim, "hbm") as handle:
        x0 = tda.add_norm_fp8(hidden, norm[0], group=128)
        xs, residuals = [x0[:2]] * a.ranks, [hidden] * a.ranks
        torch.cuda.synchronize()
        for i in range(a.layers):
            before, residual = xs[0], residuals[0]
            xs, residuals, routes = layer(ranks, handle, norm, router, i, a.chosen, xs, residuals)
            torch.cuda.synchronize()
            y, h, total = plain_layer(ranks, norm, i, before, residual, routes[0])
            got = residuals[0].float() - residual.float()
            worst = max(worst, ((got - total).norm() / total.norm()).item(), ((residuals[0].float() - h).norm() / h.norm()).item())
            same &= all(torch.equal(xs[0][0].view(torch.uint8), x[0].view(torch.uint8)) and torch.equal(residuals[0], r)
                        and torch.equal(routes[0].rows, k.rows) for x, r, k in zip(xs, residuals, routes))
        handle.check()
        tda.matmul_fp8_check()
    print(f"{a.layers} layers of {a.experts} experts on {a.ranks} ranks: relative distance from float32 at most {worst:.2g}, "
          f"all ranks {'the same' if same else 'NOT the same'}")
    return worst, same


if __name__ == "__main__":
    main()
