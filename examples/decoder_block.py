"""A decoder of attention and MoE blocks: several samples continue one prompt.

    python examples/decoder_block.py [--layers 2] [--prompt 1024] [--piece 400] [--samples 8] [--steps 32] [--dtype bf16]

The prompt is admitted in pieces of --piece tokens: the piece's keys are normed and turned by their positions on the way
into a paged cache, its queries in the same pass (KVCache.resize and .append, Rotary), and it attends everything admitted so
far (Attention.chunk). Each sample is a fork of the prompt's slot: it shares the prompt's full pages and has its own last
page. A step appends one token of every sample and attends the cache (Attention.decode), which reads the shared pages once
for all samples; MoELayer is the feed-forward part. At the end half of the samples are dropped and the pool is compacted. The
whole sequences without a cache (Rotary.apply, Attention.prompt) give the same numbers, which main() checks.

Weights and inputs are random; the dense projections and the blocks' norms are plain torch.
"""
from __future__ import annotations

import argparse
import os
import sys
import time

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)

import torch

import sparse_mixture_experts_moe_gb300 as moe


def rms_norm(x):
    y = x.float()
    return (y * torch.rsqrt(y.pow(2).mean(-1, keepdim=True) + 1e-6)).to(x.dtype)


class Block:
    """x + attention, then + MoE. d = heads * head_dim."""

    def __init__(self, layer, d, heads, kv_heads, experts, d_ff, rope, dtype, device, gen):
        self.layer, self.heads, self.kv_heads, self.head_dim, self.rope = layer, heads, kv_heads, d // heads, rope

        def weight(*shape):
            return (torch.randn(shape, generator=gen, device=device) * shape[-2] ** -0.5).to(dtype)

        self.w_qkv = weight(d, (heads + 2 * kv_heads) * self.head_dim)
        self.w_o = weight(d, d)
        self.norms = {name: (1 + 0.1 * torch.randn(self.head_dim, generator=gen, device=device)).to(dtype)
                      for name in ("q_weight", "k_weight")}  # of each head's queries and keys
        self.attn = moe.Attention(heads, kv_heads, self.head_dim, dtype)
        self.ffn = moe.MoELayer(weight(d, experts), weight(experts, d, d_ff), weight(experts, d_ff, d), k=2)

    def _qkv(self, x):
        # q, k and v are slices of one product: heads are dense within a token, tokens a row apart
        y = (rms_norm(x) @ self.w_qkv).view(len(x), self.heads + 2 * self.kv_heads, self.head_dim)
        return y.split([self.heads, self.kv_heads, self.kv_heads], dim=1)

    def _rest(self, x, a):
        x = x + a.reshape(x.shape) @ self.w_o
        return x + self.ffn(rms_norm(x))

    def prompt(self, x, offsets, positions):
        """Whole packed prompts, without a cache."""
        q, k, v = self._qkv(x)
        q, k = self.rope.apply(q, positions, k, **self.norms)
        return self._rest(x, self.attn.prompt(q, k, v, offsets))

    def _append(self, x, offsets, cache, slots, pos):
        q, k, v = self._qkv(x)
        return cache.append(k, v, slots, offsets, pos, self.rope, layer=self.layer, q=q, **self.norms)

    def piece(self, x, offsets, cache, slots, pos):
        """The next tokens of each slot, however many."""
        q = self._append(x, offsets, cache, slots, pos)
        return self._rest(x, self.attn.chunk(q, cache, slots, offsets, layer=self.layer))

    def step(self, x, offsets, cache, slots, pos, shared_len):
        """One more token of each slot."""
        q = self._append(x, offsets, cache, slots, pos)
        return self._rest(x, self.attn.decode(q, cache, slots, layer=self.layer, shared_len=shared_len))


class Decoder:
    def __init__(self, layers=2, d=1024, heads=16, kv_heads=4, experts=8, d_ff=2048, dtype=torch.bfloat16, device="cuda",
                 seed=0):
        gen = torch.Generator(device=device).manual_seed(seed)
        self.d, self.dtype, self.device, self.kv_heads, self.head_dim = d, dtype, device, kv_heads, d // heads
        rope = moe.Rotary(self.head_dim)
        self.blocks = [Block(i, d, heads, kv_heads, experts, d_ff, rope, dtype, device, gen) for i in range(layers)]

    def cache(self, n_pages, page_size, n_slots, max_len):
        return moe.KVCache.create(len(self.blocks), n_pages, page_size, n_slots, max_len, self.kv_heads, self.head_dim,
                                  self.dtype, self.device)

    def ints(self, values):
        return torch.tensor(values, dtype=torch.int32, device=self.device)

    def prompt(self, x, lengths):
        offsets = self.ints([sum(lengths[:i]) for i in range(len(lengths) + 1)])
        positions = torch.cat([torch.arange(n, dtype=torch.int32, device=self.device) for n in lengths])
        for b in self.blocks:
            x = b.prompt(x, offsets, positions)
        return x

    def piece(self, x, lengths, cache, slots):
        """The next lengths[i] tokens of each slot."""
        offsets = self.ints([sum(lengths[:i]) for i in range(len(lengths) + 1)])
        pos = cache.lens[slots]
        cache.resize(slots, pos + self.ints(lengths))
        for b in self.blocks:
            x = b.piece(x, offsets, cache, slots, pos)
        return x

    def step(self, x, cache, slots, shared_len=0):
        n = len(slots)
        offsets = torch.arange(n + 1, dtype=torch.int32, device=self.device)
        pos = cache.lens[slots]
        cache.resize(slots, pos + 1)
        for b in self.blocks:
            x = b.step(x, offsets, cache, slots, pos, shared_len)
        return x

    def check(self, cache):
        """Raises if a kernel has reported an error; synchronises."""
        for part in [cache] + [p for b in self.blocks for p in (b.attn, b.ffn)]:
            status, detail = part.device_status()
            if status != moe.MOE_OK:
                raise moe.MoeError(status, f"device status ({detail})")


def generate(dec, prompt, tokens, piece=400, page_size=64):
    """prompt [P, d], admitted `piece` tokens at a time; tokens [steps, samples, d], the embeddings that each sample goes
    on with. Returns the outputs [steps, samples, d] and the cache."""
    steps, n, _ = tokens.shape
    length = len(prompt) + steps
    full = len(prompt) // page_size            # pages that every sample shares
    own = -(-length // page_size) - full
    cache = dec.cache(full + 1 + n * own, page_size, n + 1, length)
    first, samples = dec.ints([n]), dec.ints(list(range(n)))
    for x in prompt.split(piece):
        dec.piece(x, [len(x)], cache, first)
    cache.fork(first.expand(n).contiguous(), samples)
    cache.resize(first, torch.zeros_like(first))  # the samples hold its pages now
    out = torch.stack([dec.step(tokens[t], cache, samples, shared_len=full * page_size) for t in range(steps)])
    return out, cache


def main():
    ap = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    ap.add_argument("--layers", type=int, default=2)
    ap.add_argument("--prompt", type=int, default=1024)
    ap.add_argument("--piece", type=int, default=400, help="tokens of the prompt admitted at a time")
    ap.add_argument("--samples", type=int, default=8)
    ap.add_argument("--steps", type=int, default=32)
    ap.add_argument("--dtype", choices=["bf16", "f32"], default="bf16")
    args = ap.parse_args()
    dtype = torch.bfloat16 if args.dtype == "bf16" else torch.float32

    dec = Decoder(layers=args.layers, dtype=dtype)
    gen = torch.Generator(device="cuda").manual_seed(1)
    prompt = torch.randn(args.prompt, dec.d, generator=gen, device="cuda").to(dtype)
    tokens = torch.randn(args.steps, args.samples, dec.d, generator=gen, device="cuda").to(dtype)

    generate(dec, prompt, tokens, args.piece)  # warm-up: workspaces
    torch.cuda.synchronize()
    t0 = time.perf_counter()
    out, cache = generate(dec, prompt, tokens, args.piece)
    torch.cuda.synchronize()
    ms = 1e3 * (time.perf_counter() - t0)
    dec.check(cache)

    # the same sequences as whole prompts
    whole = torch.cat([torch.cat([prompt, tokens[:, i]]) for i in range(args.samples)])
    want = dec.prompt(whole, [args.prompt + args.steps] * args.samples).view(args.samples, -1, dec.d)[:, args.prompt:]
    got, want = out.float(), want.transpose(0, 1).float()
    # bf16 rounds the two paths' scores differently, which now and then changes a token's experts: the median token
    err = ((got - want).norm(dim=-1) / want.norm(dim=-1)).median().item()
    print(f"{args.samples} samples of {args.steps} tokens after a prompt of {args.prompt}: {ms:.1f} ms; median difference from the "
          f"prompt path {err:.1e}")
    if not err < (2e-2 if dtype == torch.bfloat16 else 1e-4):
        raise SystemExit("the two paths differ")

    # half of the samples end: their pages are released and the others' moved to the front of the pool
    ended = dec.ints(list(range(0, args.samples, 2)))
    before = int((cache.refs > 0).sum())
    cache.resize(ended, torch.zeros_like(ended))
    live = int(cache.compact())
    dec.check(cache)
    print(f"pages in use: {before}, after half of the samples ended: {live}, the first {live} of the pool")


if __name__ == "__main__":
    main()
