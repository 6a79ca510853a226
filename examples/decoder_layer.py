"""One decoder layer of a mixture-of-experts model on the FP8 block-scaled path, served from a paged cache.

    python examples/decoder_layer.py [--dim 2048] [--sequences 3] [--prompt 100] [--decode 8]

The layer is what a serving program calls for every step, with whatever new tokens there are -- the rest of a
prompt, single tokens of other sequences, or both in one batch:

    act_quant + fp8_gemm    q, k and v of the normalised input
    qk_norm_rope            norm and rotation of q and k per head; keys and values into their cache slots
    paged_attention         the new tokens over all keys of their sequences
    act_quant + fp8_gemm    output projection
    moe_layer               router, experts and weighted sum, 64 tokens at a time

Weights are random, in the library's format: e4m3 codes with one fp32 scale per 128 x 128 block.
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)

import fp8_block_scaled_fp8bs_gb300 as fp8bs  # noqa: E402

BLOCK = 128


def quantised(g, *shape):
    """Random weights [..., N, K] of variance 1/K as e4m3 codes and block scales."""
    codes = (torch.randn(*shape, generator=g, device="cuda") * 32).to(torch.float8_e4m3fn)
    blocks = (*shape[:-2], shape[-2] // BLOCK, shape[-1] // BLOCK)
    scales = torch.exp2(torch.rand(*blocks, generator=g, device="cuda") - 0.5)
    return codes, scales / (32 * shape[-1] ** 0.5)


def rms_norm(x, w):
    y = x.float()
    return (y * torch.rsqrt(y.pow(2).mean(-1, keepdim=True) + 1e-6) * w.float()).bfloat16()


class DecoderLayer:
    def __init__(self, dim=2048, q_heads=16, k_heads=4, head_dim=128, experts=16, inter=512, top_k=4,
                 max_positions=4096, seed=0):
        g = torch.Generator(device="cuda")
        g.manual_seed(seed)
        self.q_heads, self.k_heads, self.head_dim, self.top_k = q_heads, k_heads, head_dim, top_k
        self.wqkv = quantised(g, (q_heads + 2 * k_heads) * head_dim, dim)
        self.wo = quantised(g, dim, q_heads * head_dim)
        self.w13 = quantised(g, experts, 2 * inter, dim)
        self.w2 = quantised(g, experts, dim, inter)
        self.router = (torch.randn(experts, dim, generator=g, device="cuda") * dim ** -0.5).bfloat16()
        self.router_bias = torch.zeros(experts, device="cuda")
        ones = lambda n: torch.ones(n, device="cuda", dtype=torch.bfloat16)  # noqa: E731
        self.attn_norm, self.moe_norm = ones(dim), ones(dim)
        self.q_norm, self.k_norm = ones(head_dim), ones(head_dim)
        inv = 10000.0 ** (-torch.arange(head_dim // 2, device="cuda", dtype=torch.float64) * 2 / head_dim)
        angle = torch.arange(max_positions, device="cuda", dtype=torch.float64)[:, None] * inv
        self.cos, self.sin = angle.cos().float(), angle.sin().float()

    def linear(self, x, w):
        return fp8bs.act_quant_gemm(x, *w, weights_constant=True)[0]

    def __call__(self, x, cache, batch):
        """x bf16 [T, dim] -> bf16 [T, dim]; the new tokens' keys and values go into the cache."""
        T = x.shape[0]
        hq, hk, d = self.q_heads, self.k_heads, self.head_dim
        qkv = self.linear(rms_norm(x, self.attn_norm), self.wqkv)
        q = qkv[:, :hq * d].unflatten(1, (hq, d))
        k = qkv[:, hq * d:(hq + hk) * d].unflatten(1, (hk, d))
        v = qkv[:, (hq + hk) * d:].unflatten(1, (hk, d))
        q = fp8bs.qk_norm_rope(q, k, self.cos, self.sin, batch["positions"], q_weight=self.q_norm,
                               k_weight=self.k_norm, cache=cache, v=v, slots=batch["slots"])
        o = fp8bs.paged_attention(q, cache, batch["page_table"], batch["q_start"], batch["kv_len"],
                                  max_q_len=batch["max_q_len"], max_kv_len=batch["max_kv_len"])
        x = x + self.linear(o.flatten(1), self.wo)
        h = rms_norm(x, self.moe_norm)
        most = fp8bs.MOE_MAX_TOKENS
        y = [fp8bs.moe_layer(h[t:t + most], self.router, *self.w13, *self.w2, self.top_k,
                             bias=self.router_bias) for t in range(0, T, most)]
        return x + torch.cat(y)


class Pages:
    """The host's side of a paged cache: which pages a sequence holds, and what a step's batch looks like."""

    def __init__(self, pages, page_size):
        self.free, self.page_size = list(range(pages)), page_size
        self.held, self.length = {}, {}

    def step(self, new):
        """new: {sequence: number of new tokens} -> the batch description of a layer call."""
        positions, slots, starts, lens, tables = [], [], [0], [], []
        for s, n in new.items():
            held, at = self.held.setdefault(s, []), self.length.get(s, 0)
            while len(held) * self.page_size < at + n:
                held.append(self.free.pop())
            for p in range(at, at + n):
                positions.append(p)
                slots.append(held[p // self.page_size] * self.page_size + p % self.page_size)
            self.length[s] = at + n
            starts.append(starts[-1] + n)
            lens.append(at + n)
            tables.append(held)
        width = max(len(t) for t in tables)
        dev = {"device": "cuda"}
        return {"positions": torch.tensor(positions, dtype=torch.int32, **dev),
                "slots": torch.tensor(slots, dtype=torch.int64, **dev),
                "q_start": torch.tensor(starts, dtype=torch.int32, **dev),
                "kv_len": torch.tensor(lens, dtype=torch.int32, **dev),
                "page_table": torch.tensor([t + [0] * (width - len(t)) for t in tables], dtype=torch.int32, **dev),
                "max_q_len": max(new.values()), "max_kv_len": max(lens)}

    def release(self, s):
        self.free += self.held.pop(s, [])
        self.length.pop(s, None)


def new_cache(layer, pages, page_size):
    shape = (pages, page_size, layer.k_heads, layer.head_dim)
    return fp8bs.PagedCache(*(torch.zeros(shape, dtype=torch.bfloat16, device="cuda") for _ in range(2)))


def main():
    ap = argparse.ArgumentParser()
    ap.add_argument("--dim", type=int, default=2048)
    ap.add_argument("--sequences", type=int, default=3)
    ap.add_argument("--prompt", type=int, default=100)
    ap.add_argument("--decode", type=int, default=8)
    a = ap.parse_args()
    layer = DecoderLayer(dim=a.dim)
    pages = Pages(256, 16)
    cache = new_cache(layer, 256, 16)
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    tokens = lambda n: torch.randn(n, a.dim, generator=g, device="cuda").bfloat16()  # noqa: E731
    # prompts one after another, the sequences before them decoding on in the same batch
    for s in range(a.sequences):
        new = {**{b: 1 for b in range(s)}, s: a.prompt + s}
        y = layer(tokens(sum(new.values())), cache, pages.step(new))
        print(f"prompt of sequence {s}: {tuple(y.shape)}, rms {y.float().pow(2).mean().sqrt().item():.3f}")
    step = {s: 1 for s in range(a.sequences)}
    x = tokens(a.sequences)
    for i in range(a.decode):
        y = layer(x, cache, pages.step(step))
    torch.cuda.synchronize()
    print(f"{a.decode} decode steps: lengths {pages.length}, rms {y.float().pow(2).mean().sqrt().item():.3f}")
    assert fp8bs.fp8bs_device_error() == 0


if __name__ == "__main__":
    main()
