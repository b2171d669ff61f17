"""A 16-bit mixture-of-experts block around the library's operators, next to a 4-bit layer.

    h   = norm(r) * w_pre                                moe_block_norm (before the first block)
    ids, w = top-k of the router's logits                moe_router
    offsets, perm, slot_of = slots grouped by expert     moe_group
    u   = SwiGLU(W13[e] h[token])                        MoEGrouped, rows gathered by perm
    y   = W2[e] u                                        MoEGrouped, rows in place
    r'  = r + scale * gate * norm(sum_j w_j y[slot_j])   moe_block_norm (combine, norm after the
    h'  = norm(r') * w_next                              block, gate, residual scale, norm before
                                                         the next block)

The next block here is a 4-bit layer (MoELayer, MXFP4 weights and MXFP8 activations): it takes h' and
the router's ids and weights as they are, and its output goes through moe_block_norm again.

    python examples/block16.py [--tokens 16] [--experts 32] [--hidden 1024] [--inter 256] [--topk 4]
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import serving_route_count_gb300 as moe  # noqa: E402


class Block16:
    """One block's weights, plans and buffers for calls of up to max_tokens tokens."""

    def __init__(self, experts, hidden, inter, topk, max_tokens, dtype=torch.bfloat16, limit=7.0, scale=0.5, seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        rnd = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
        self.E, self.H, self.I, self.k, self.scale, self.limit = experts, hidden, inter, topk, scale, limit
        self.router = (rnd(experts, hidden) * hidden ** -0.5).to(dtype)
        self.bias = 0.1 * rnd(experts)
        self.w13 = (rnd(experts, 2 * inter, hidden) * hidden ** -0.5).to(dtype)
        self.w2 = (rnd(experts, hidden, inter) * inter ** -0.5).to(dtype)
        self.post = (1 + 0.1 * rnd(hidden)).to(dtype)
        self.next = (1 + 0.1 * rnd(hidden)).to(dtype)
        self.gate = torch.sigmoid(rnd(hidden)).to(dtype)
        rows = max_tokens * topk
        self.up = moe.MoEGrouped(experts, 2 * inter, hidden, rows, dtype, act=moe.MOE_ACT_SWIGLU, swiglu_limit=limit)
        self.down = moe.MoEGrouped(experts, hidden, inter, rows, dtype)

    def route(self, h):
        logits = h @ self.router.t()
        return moe.moe_router(logits, self.k, score=moe.MOE_SCORE_SIGMOID, bias=self.bias, scale=2.5)

    def __call__(self, r, h):
        """(r', h'): the residual stream after the block and the next block's input."""
        ids, w = self.route(h)
        offsets, perm, slot_of = moe.moe_group(ids, self.E)
        u = self.up(h, self.w13, offsets, perm=perm, topk=self.k)
        y = self.down(u, self.w2, offsets)
        return moe.moe_block_norm(r, y, slot_of=slot_of, topk_weights=w, post_weight=self.post, gate=self.gate, scale=self.scale,
                                  pre_weight=self.next)


def run(tokens=16, experts=32, hidden=1024, inter=256, topk=4, seed=0):
    """Both blocks once; (block, layer, r0, h0, r1, h1, r2, h2)."""
    from synth import moe_inputs as S
    block = Block16(experts, hidden, inter, topk, tokens, seed=seed)
    cfg = S.CONFIGS["tiny_w4a8"]
    layer = moe.MoELayer(S.make_checkpoint(cfg, seed=seed, E=experts, H=hidden, I=inter), topk, tokens, swiglu_limit=7.0, deterministic=True)
    g = torch.Generator(device="cuda").manual_seed(seed + 1)
    r0 = torch.randn((tokens, hidden), generator=g, device="cuda").bfloat16()
    w0 = torch.ones(hidden, device="cuda").bfloat16()
    _, h0 = moe.moe_block_norm(r0, pre_weight=w0)
    r1, h1 = block(r0, h0)
    ids, w = block.route(h1)
    r2, h2 = moe.moe_block_norm(r1, layer(h1, ids, w), post_weight=block.post, scale=block.scale, pre_weight=block.next)
    return block, layer, r0, h0, r1, h1, r2, h2


def main():
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    for name, value in (("tokens", 16), ("experts", 32), ("hidden", 1024), ("inter", 256), ("topk", 4)):
        ap.add_argument("--" + name, type=int, default=value)
    a = ap.parse_args()
    block, layer, r0, h0, r1, h1, r2, h2 = run(**vars(a))
    print("residual rms before / after the 16-bit block / after the 4-bit one: %.4f %.4f %.4f" % tuple(
        r.float().square().mean().sqrt() for r in (r0, r1, r2)))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        block(r0, h0)
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        rg, hg = block(r0, h0)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(rg, r1) and torch.equal(hg, h1)
    a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    a.record()
    for _ in range(20):
        graph.replay()
    b.record()
    b.synchronize()
    print("16-bit block, replayed as a graph: %.1f us" % (a.elapsed_time(b) / 20 * 1e3))
    print("device errors:", block.up.device_error(), block.down.device_error(), moe.moe_block_norm_get_device_error(), layer.device_error())


if __name__ == "__main__":
    main()
