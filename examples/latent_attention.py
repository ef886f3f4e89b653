"""The attention half of the block with the package's latent-attention calls: prompts in
the expanded form, then single tokens in the absorbed form over the paged cache.

    python examples/latent_attention.py [--prompts 5,700,64] [--tokens 8] [--heads 64]

Both forms give the same attention, so the last prompt token, decoded again over the
cache, has to reproduce its prefill result; the script prints how near it comes and how
long a decode step takes in a CUDA graph.
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)

import routed_fp8_expert_gb300 as moe  # noqa: E402

LATENT, ROPE, NOPE, V = moe.MLA_LATENT, moe.MLA_ROPE, 128, 128
PAGE = 64


class LatentAttention:
    """One layer's latent attention for a batch of sequences: what a serving loop keeps."""

    def __init__(self, w_ukv, gamma, pages, max_pages, batch, device):
        """w_ukv [H, 128 + 128, 512]: the up-projection, each head's keys then its values."""
        self.w, self.gamma, self.H = w_ukv, gamma, w_ukv.shape[0]
        self.plan = moe.rope_plan(ROPE, base=50000.0, factor=32.0, original_ctx=4096, mscale=1.0, mscale_all_dim=1.0,
                                  device=device)
        self.scale = (NOPE + ROPE) ** -0.5 * self.plan.softmax_factor
        self.cache = torch.zeros(pages, PAGE, LATENT + ROPE, dtype=w_ukv.dtype, device=device)
        self.table = torch.arange(batch * max_pages, dtype=torch.int32, device=device).view(batch, max_pages)
        self.ctx = torch.zeros(batch, dtype=torch.int32, device=device)
        self.ws = moe.mla_paged_workspace(device)

    def prefill(self, q, kv, lens):
        """q [T, H, 192] and kv [T, 576] (latent, rotary key) of whole prompts, one after
        the other: their rows go to the cache, their attention runs expanded. -> [T, H, 128]"""
        dev = q.device
        cu = torch.tensor([0] + list(lens), device=dev).cumsum(0).to(torch.int32)
        pos = torch.cat([torch.arange(n, device=dev) for n in lens]).to(torch.int32)
        seq = torch.repeat_interleave(torch.arange(len(lens), device=dev), torch.tensor(list(lens), device=dev))
        slots = self.table[seq, (pos // PAGE).long()] * PAGE + pos % PAGE
        row = torch.empty_like(kv)
        q = q.clone()
        moe.mla_rope_append(q[..., NOPE:], kv, pos, self.plan, gamma=self.gamma, cache=self.cache,
                            slots=slots.to(torch.int32), q_out=q[..., NOPE:], kv_out=row)
        kvx = moe.mla_head_proj(row[:, None, :LATENT], self.w)
        self.ctx.copy_(torch.tensor(list(lens), dtype=torch.int32))
        return moe.mla_attn_ragged(q, kvx[..., :NOPE], row[:, LATENT:], kvx[..., NOPE:], cu, cu, max(lens), self.scale)

    def decode(self, q, kv, pos, q_abs=None):
        """q [B, H, 192], kv [B, 576]: one new token per sequence at positions pos [B] (the
        sequence's length so far, or less to decode a token again). -> [B, H, 128]"""
        if q_abs is None:
            q_abs = torch.empty(q.shape[0], self.H, LATENT + ROPE, dtype=q.dtype, device=q.device)
        slots = self.table.gather(1, (pos // PAGE).long()[:, None])[:, 0] * PAGE + pos % PAGE
        moe.mla_rope_append(q[..., NOPE:], kv, pos, self.plan, gamma=self.gamma, cache=self.cache, slots=slots,
                            q_out=q_abs[..., LATENT:])
        torch.add(pos, 1, out=self.ctx)
        moe.mla_head_proj(q[..., :NOPE], self.w[:, :NOPE], w_kn=True, out=q_abs[..., :LATENT])
        o = moe.mla_attn_paged(q_abs, self.cache, self.table, self.ctx, self.scale, ws=self.ws)
        return moe.mla_head_proj(o, self.w[:, NOPE:])


def main(prompts=(5, 700, 64), tokens=8, heads=64, device="cuda:0", seed=0):
    g = torch.Generator(device=device).manual_seed(seed)

    def rand(*shape, std=1.0):
        return (torch.randn(*shape, generator=g, device=device) * std).to(torch.bfloat16)

    B, T = len(prompts), sum(prompts)
    max_pages = (max(prompts) + tokens + PAGE - 1) // PAGE
    attn = LatentAttention(rand(heads, NOPE + V, LATENT, std=LATENT ** -0.5), (1 + rand(LATENT, std=0.1).float()).to(torch.bfloat16),
                           B * max_pages, max_pages, B, device)
    q, kv = rand(T, heads, NOPE + ROPE), rand(T, LATENT + ROPE, std=2.0)
    out = attn.prefill(q, kv, prompts)
    last = torch.tensor(list(prompts), device=device).cumsum(0) - 1
    pos = (attn.ctx - 1).clone()
    again = attn.decode(q[last].contiguous(), kv[last].contiguous(), pos)
    diff = ((again.float() - out[last].float()).norm() / out[last].float().norm()).item()
    print(f"prompts {list(prompts)}: decoding the last tokens again differs by {diff:.2e} (relative)")

    # a decode step in a CUDA graph: new tokens and positions go into the same tensors
    new_q, new_kv = rand(B, heads, NOPE + ROPE), rand(B, LATENT + ROPE, std=2.0)
    pos.copy_(torch.tensor(list(prompts), dtype=torch.int32))
    attn.decode(new_q, new_kv, pos)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step_out = attn.decode(new_q, new_kv, pos)
    start, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    start.record()
    for _ in range(tokens):
        new_q.normal_(generator=g)
        new_kv.normal_(generator=g)
        graph.replay()
        pos += 1
    end.record()
    torch.cuda.synchronize()
    moe.check_device_error(device)
    print(f"{tokens} tokens for {B} sequences: {start.elapsed_time(end) / tokens * 1e3:.0f} us a step, new inputs included; "
          f"finite: {bool(torch.isfinite(step_out).all())}")
    return diff


if __name__ == "__main__":
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--prompts", default="5,700,64")
    ap.add_argument("--tokens", type=int, default=8)
    ap.add_argument("--heads", type=int, default=64)
    a = ap.parse_args()
    main([int(x) for x in a.prompts.split(",")], a.tokens, a.heads)
