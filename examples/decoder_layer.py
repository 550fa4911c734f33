"""A decoder layer on the library's operators: attention over a paged cache,
then MXFP4 routed experts.

    h = x + Wo attention(norm(x));   y = experts(norm(h)) + h

    python examples/decoder_layer.py

runs two prompts through the layer, then a few single-token steps, and prints
each step's time. The projections are plain matrix products (torch); the head
norms, the rotation and the cache write are one call (append_kv), the attention
another (paged_attention_prefill or paged_attention_decode), the router and
the experts two more (router_topk, mxfp4_swiglu_expert).
"""
from __future__ import annotations

import math
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import mxfp4_routed_expert_route_gb300 as lib  # noqa: E402


class DecoderLayer:
    """Random weights; `width` a multiple of 32, as the experts need."""

    def __init__(self, *, width=256, heads=8, kv_heads=2, head_dim=64, experts=8, picks=2,
                 hidden=128, window=None, sinks=0, pages=64, page_size=16, max_positions=1024,
                 dtype=torch.bfloat16, device="cuda", seed=0):
        g = torch.Generator(device=device).manual_seed(seed)
        self.heads, self.kv_heads, self.head_dim = heads, kv_heads, head_dim
        self.picks, self.window, self.sinks = picks, window, sinks

        def weight(*shape):
            return (torch.randn(*shape, generator=g, device=device) / math.sqrt(shape[0])).to(dtype)

        def mxfp4(rows, cols):
            packed = torch.randint(0, 256, (experts, rows, cols // 32, 16), generator=g,
                                   device=device, dtype=torch.uint8)
            scales = torch.randint(118, 122, (experts, rows, cols // 32), generator=g,
                                   device=device, dtype=torch.uint8)
            return packed, scales

        self.qkv = weight(width, (heads + 2 * kv_heads) * head_dim)
        self.out = weight(heads * head_dim, width)
        self.q_norm = torch.ones(head_dim, device=device, dtype=dtype)
        self.k_norm = torch.ones(head_dim, device=device, dtype=dtype)
        self.router = weight(width, experts).float()
        self.gate_up, self.down = mxfp4(2 * hidden, width), mxfp4(width, hidden)
        self.cache = lib.PagedKVCache.empty(pages, kv_heads, page_size, head_dim, dtype, device)
        inv = 10000.0 ** (-torch.arange(0, head_dim, 2, device=device) / head_dim)
        angle = torch.arange(max_positions, device=device)[:, None] * inv
        self.cos_sin = torch.cat([angle.cos(), angle.sin()], 1).float()

    @staticmethod
    def _norm(x):
        f = x.float()
        return (f * torch.rsqrt(f.square().mean(-1, keepdim=True) + 1e-6)).to(x.dtype)

    def __call__(self, x, seqs):
        """x: (tokens, width), the new tokens of `seqs` one after another."""
        T = x.shape[0]
        q, k, v = (self._norm(x) @ self.qkv).view(T, -1, self.head_dim).split(
            [self.heads, self.kv_heads, self.kv_heads], 1)
        q = lib.append_kv(q, k, v, self.cache, seqs, cos_sin=self.cos_sin, q_norm=self.q_norm,
                          k_norm=self.k_norm)
        attention = lib.paged_attention_decode if seqs.q_offsets is None \
            else lib.paged_attention_prefill
        a = attention(q, self.cache, seqs, window=self.window, sinks=self.sinks)
        h = x + a.view(T, -1) @ self.out
        z = self._norm(h)
        sel, p = lib.router_topk(z.float() @ self.router, None, self.picks)
        return lib.mxfp4_swiglu_expert(z, *self.gate_up, *self.down, sel, p, h)


def main():
    layer = DecoderLayer()
    prompts = [37, 130]
    # Each sequence owns pages for its prompt and the steps that follow.
    table = torch.arange(32, dtype=torch.int32, device="cuda").view(2, 16)
    lens = torch.tensor(prompts, dtype=torch.int32, device="cuda")
    offsets = torch.tensor([0, 37, 167], dtype=torch.int32, device="cuda")
    x = torch.randn(167, 256, device="cuda", dtype=torch.bfloat16)
    start, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))

    def timed(what, x, seqs):
        start.record()
        y = layer(x, seqs)
        end.record()
        end.synchronize()
        print(f"{what}: {x.shape[0]} tokens, {start.elapsed_time(end):.2f} ms, "
              f"|y| = {y.float().norm():.3f}")
        return y

    y = timed("prompts", x, lib.PagedSequences(table, lens, offsets))
    step = lib.PagedSequences(table, lens)
    x = y[offsets[1:].long() - 1]
    for i in range(4):
        lens += 1                      # read on the GPU: the handle stays
        x = timed(f"step {i}", x, step)
    assert lib.page_errors() == 0 and lib.wait_timeouts() == 0


if __name__ == "__main__":
    main()
