"""One decoder layer with both halves from this package: attention over a paged
4-bit key/value cache, then the routed MoE FFN over its expert cache.

    python examples/decoder_layer.py [--steps 16] [--prompts 60,201,33]

Random weights of a small shape. Packed prompts go through the layer at once
(moe_kv_append, moe_attn_prompt, moe_layer_forward's prefill), then steps of one
token per sequence (moe_kv_append, moe_kv_attend, moe_layer_forward's decode);
the projections are plain matrix products. A program with several layers keeps
one KVCache and one MoECache for all of them and passes the layer's number.
"""
import argparse
import os
import sys
import time

import numpy as np

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))


class Sequences:
    """Which pages hold which tokens: every sequence's length, the block table,
    and the batches of a prompt or of one new token each."""

    def __init__(self, lens, most, page_tokens):
        import torch
        import paged_expert_cache_gb300 as pec
        self.pec, self.lens = pec, list(lens)
        per = -(-most // page_tokens)
        self.pages = per * len(lens)
        order = torch.randperm(self.pages, generator=torch.Generator().manual_seed(1)).to(torch.int32)
        self.table = order.view(len(lens), per).cuda()
        self.kv_lens = torch.tensor(self.lens, dtype=torch.int32).cuda()
        self.step_cu = torch.arange(len(lens) + 1, dtype=torch.int32).cuda()

    def prompt(self):
        import torch
        cu = torch.tensor([0] + self.lens).cumsum(0).to(torch.int32).cuda()
        return self.pec.KVBatch(cu, self.kv_lens, self.table)

    def step(self):
        """One more token in every sequence."""
        self.lens = [n + 1 for n in self.lens]
        self.kv_lens += 1
        return self.pec.KVBatch(self.step_cu, self.kv_lens, self.table)


class DecoderLayer:
    def __init__(self, seqs, hidden=256, inter=128, experts=16, top_k=2, slots=12, q_heads=8, kv_heads=2, head_dim=64,
                 page_tokens=16, max_tokens=512, max_positions=4096, seed=7):
        import torch
        import paged_expert_cache_gb300 as pec
        import synth
        self.pec, self.torch = pec, torch
        self.q_heads, self.kv_heads, self.dim, self.hidden = q_heads, kv_heads, head_dim, hidden
        g = torch.Generator().manual_seed(seed)

        def weight(rows, cols):
            return (torch.randn(rows, cols, generator=g) * cols ** -0.5).bfloat16().cuda()

        self.w_qkv = weight((q_heads + 2 * kv_heads) * head_dim, hidden)
        self.w_out = weight(hidden, q_heads * head_dim)
        self.kv = pec.KVCache(pec.make_kv_config(1, seqs.pages, q_heads, kv_heads, head_dim, page_tokens=page_tokens))
        inv = 10000.0 ** (-torch.arange(0, head_dim, 2, dtype=torch.float64) / head_dim)
        angle = torch.arange(max_positions, dtype=torch.float64)[:, None] * inv
        self.rope = torch.cat([angle.cos(), angle.sin()], 1).float().cuda()
        self.moe = pec.MoECache(pec.make_config(1, experts, top_k, hidden, inter, fmt="q4_0", slots_per_layer=slots,
                                                max_tokens=max_tokens, max_cache_tokens=slots // top_k))
        self.moe.load_experts(0, 0, synth.expert_records("q4_0", seed, 0, 0, experts, hidden, inter))
        self.router = torch.from_numpy(synth.router_weights(seed, 0, experts, hidden).view(np.int16)).cuda()

    def close(self):
        self.moe.close()
        self.kv.close()

    @staticmethod
    def norm(x):
        x = x.float()
        return (x * (x.square().mean(-1, keepdim=True) + 1e-6).rsqrt()).bfloat16()

    def project(self, x):
        """q, k, v: views of one fused projection's rows."""
        y = self.norm(x) @ self.w_qkv.T
        q, k, v = y.split([n * self.dim for n in (self.q_heads, self.kv_heads, self.kv_heads)], 1)
        return (t.unflatten(1, (-1, self.dim)) for t in (q, k, v))

    def ffn(self, x):
        h = self.norm(x)
        y = self.torch.empty(h.shape, dtype=self.torch.float32, device="cuda")
        self.moe.forward(h.view(self.torch.int16), self.router, 0, y)
        return x + y

    def prompt(self, x, batch):
        """x fp32 [T, hidden]: whole prompts, packed. Returns the layer's output."""
        torch = self.torch
        q, k, v = self.project(x)
        qr = torch.empty(q.shape, dtype=torch.bfloat16, device="cuda")
        kr = torch.empty(k.shape, dtype=torch.bfloat16, device="cuda")
        self.kv.append(0, q, k, v, batch, rope=self.rope, q_out=qr, k_out=kr)
        o = self.pec.attention_prompt(qr, kr, v, torch.empty_like(qr), batch.cu_tokens)
        return self.ffn(x + (o.flatten(1) @ self.w_out.T).float())

    def step(self, x, batch):
        """x fp32 [sequences, hidden]: one new token each."""
        torch = self.torch
        q, k, v = self.project(x)
        qr = torch.empty(q.shape, dtype=torch.bfloat16, device="cuda")
        self.kv.append(0, q, k, v, batch, rope=self.rope, q_out=qr)
        o = self.kv.attend(0, qr, batch, torch.empty_like(qr))
        return self.ffn(x + (o.flatten(1) @ self.w_out.T).float())


def main():
    import torch
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--prompts", default="60,201,33", help="lengths of the prompts")
    ap.add_argument("--steps", type=int, default=16)
    a = ap.parse_args()
    lens = [int(n) for n in a.prompts.split(",")]
    seqs = Sequences(lens, max(lens) + a.steps, 16)
    layer = DecoderLayer(seqs, max_tokens=max(sum(lens), 32), max_positions=max(lens) + a.steps)
    g = torch.Generator(device="cuda").manual_seed(3)
    y = layer.prompt(torch.randn(sum(lens), layer.hidden, generator=g, device="cuda"), seqs.prompt())
    last = y[torch.tensor(lens).cumsum(0) - 1]
    torch.cuda.synchronize()
    t = time.perf_counter()
    for _ in range(a.steps):
        last = layer.step(last, seqs.step())
    torch.cuda.synchronize()
    t = (time.perf_counter() - t) / max(a.steps, 1)
    layer.kv.status()
    hits = layer.moe.stats()["buckets"][0]
    print(f"{len(lens)} prompts of {lens} tokens, {a.steps} steps: {t * 1e6:.0f} us a step, "
          f"{layer.kv.info()['page_bytes']} bytes a page of 16 tokens, expert hits {hits['hits']} misses {hits['misses']}")
    layer.close()


if __name__ == "__main__":
    main()
