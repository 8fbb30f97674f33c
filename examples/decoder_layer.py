"""One decoder layer with both halves from this package: attention over a paged
4-bit key/value cache, then the routed MoE FFN over its expert cache.

    python examples/decoder_layer.py [--steps 16] [--prompts 60,201,33] [--samples 4]

Random weights of a small shape. Packed prompts go through the layer at once
(moe_kv_append, moe_attn_prompt, moe_layer_forward's prefill), then steps of one
token per sequence (moe_kv_append, moe_kv_attend, moe_layer_forward's decode),
with moe_residual_norm between the halves; the projections are plain matrix
products. With --samples, each prompt is continued so many times: the
continuations share its pages and attend over them together
(moe_kv_attend_shared), and their tokens are drawn by moe_sample. A program with
several layers keeps one KVCache and one MoECache for all of them and passes the
layer's number.
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


class Continuations:
    """samples continuations of every prompt of a Sequences: they name the pages
    that their prompt fills, and have a copy of the rest and new pages of their own."""

    def __init__(self, seqs, samples, most, page_tokens):
        import torch
        import paged_expert_cache_gb300 as pec
        self.pec, self.samples, self.prompts = pec, samples, list(seqs.lens)
        whole = [n // page_tokens for n in self.prompts]
        own = -(-most // page_tokens) - min(whole)
        count = len(self.prompts) * samples
        self.pages = seqs.pages + count * own
        self.table = seqs.table.repeat_interleave(samples, 0)
        width = max(self.table.shape[1], max(whole) + own)
        self.table = torch.nn.functional.pad(self.table, (0, width - self.table.shape[1]))
        for b in range(count):
            at = whole[b // samples]
            self.table[b, at:at + own] = seqs.pages + b * own + torch.arange(own, device="cuda")
        self.kv_lens = torch.tensor(self.prompts, dtype=torch.int32).repeat_interleave(samples).cuda()
        self.step_cu = torch.arange(count + 1, dtype=torch.int32).cuda()
        self.groups = pec.KVGroups(torch.arange(len(self.prompts) + 1, dtype=torch.int32).cuda() * samples,
                                   torch.tensor(self.prompts, dtype=torch.int32).cuda())
        # what each continuation writes again of its prompt: the rows of the page that it does not fill
        starts = torch.tensor([0] + self.prompts).cumsum(0).tolist()
        tails = [range(starts[i] + whole[i] * page_tokens, starts[i + 1]) for i in range(len(whole)) for _ in range(samples)]
        self.tail_rows = torch.tensor([r for t in tails for r in t], dtype=torch.int64).cuda()
        self.tail_cu = torch.tensor([0] + [len(t) for t in tails]).cumsum(0).to(torch.int32).cuda()

    def tail(self):
        return self.pec.KVBatch(self.tail_cu, self.kv_lens, self.table)

    def step(self):
        """One more token in every continuation."""
        self.kv_lens += 1
        return self.pec.KVBatch(self.step_cu, self.kv_lens, self.table)


class DecoderLayer:
    def __init__(self, seqs, hidden=256, inter=128, experts=16, top_k=2, slots=12, q_heads=8, kv_heads=2, head_dim=64,
                 page_tokens=16, max_tokens=512, max_positions=4096, seed=7, pages=None, vocab=1000):
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
        self.kv = pec.KVCache(pec.make_kv_config(1, pages or seqs.pages, q_heads, kv_heads, head_dim, page_tokens=page_tokens))
        self.w_head, self.embedding = weight(vocab, hidden), weight(vocab, hidden).float() * hidden ** 0.5
        self.workspace = None
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

    def norm(self, x):
        return self.pec.residual_norm(x, out=self.torch.empty(x.shape, dtype=self.torch.bfloat16, device="cuda"))

    def project(self, x):
        """q, k, v: views of one fused projection's rows."""
        y = self.norm(x) @ self.w_qkv.T
        q, k, v = y.split([n * self.dim for n in (self.q_heads, self.kv_heads, self.kv_heads)], 1)
        return (t.unflatten(1, (-1, self.dim)) for t in (q, k, v))

    def ffn(self, x):
        h = self.norm(x)
        y = self.torch.empty(h.shape, dtype=self.torch.float32, device="cuda")
        self.moe.forward(h.view(self.torch.int16), self.router, 0, y)
        return self.pec.residual_norm(x, y, x_out=self.torch.empty_like(x))

    def prompt(self, x, batch):
        """x fp32 [T, hidden]: whole prompts, packed. Returns the layer's output."""
        torch = self.torch
        q, k, v = self.project(x)
        qr = torch.empty(q.shape, dtype=torch.bfloat16, device="cuda")
        kr = torch.empty(k.shape, dtype=torch.bfloat16, device="cuda")
        self.kv.append(0, q, k, v, batch, rope=self.rope, q_out=qr, k_out=kr)
        self.last_prompt = kr, v
        o = self.pec.attention_prompt(qr, kr, v, torch.empty_like(qr), batch.cu_tokens)
        return self.ffn(x + (o.flatten(1) @ self.w_out.T).float())

    def fork(self, continuations):
        """Writes what the continuations have for themselves of the last prompts."""
        k, v = (t[continuations.tail_rows] for t in self.last_prompt)
        if len(k):
            self.kv.append(0, None, k.contiguous(), v.contiguous(), continuations.tail())

    def step(self, x, batch, groups=None):
        """x fp32 [sequences, hidden]: one new token each; groups: those that share
        their prompt's positions."""
        torch = self.torch
        q, k, v = self.project(x)
        qr = torch.empty(q.shape, dtype=torch.bfloat16, device="cuda")
        self.kv.append(0, q, k, v, batch, rope=self.rope, q_out=qr)
        if groups is None:
            o = self.kv.attend(0, qr, batch, torch.empty_like(qr))
        else:
            if self.workspace is None:
                self.workspace = self.kv.shared_workspace(len(qr))
            o = self.kv.attend_shared(0, qr, batch, groups, torch.empty_like(qr), self.workspace)
        return self.ffn(x + (o.flatten(1) @ self.w_out.T).float())

    def draw(self, x, uniform, **settings):
        """The next tokens of the layer's outputs x, and their rows of the embedding."""
        torch = self.torch
        logits = self.norm(x) @ self.w_head.T
        tokens = self.pec.sample(logits, torch.empty(len(x), dtype=torch.int32, device="cuda"), uniform, **settings)
        return tokens, self.embedding[tokens.long()]


def main():
    import torch
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--prompts", default="60,201,33", help="lengths of the prompts")
    ap.add_argument("--steps", type=int, default=16)
    ap.add_argument("--samples", type=int, default=0, help="continuations of each prompt, with tokens drawn")
    a = ap.parse_args()
    lens = [int(n) for n in a.prompts.split(",")]
    seqs = Sequences(lens, max(lens) + a.steps, 16)
    count = len(lens) * max(a.samples, 1)
    more = Continuations(seqs, a.samples, max(lens) + a.steps, 16) if a.samples else None
    layer = DecoderLayer(seqs, max_tokens=max(sum(lens), count, 32), max_positions=max(lens) + a.steps,
                         pages=more.pages if more else None)
    g = torch.Generator(device="cuda").manual_seed(3)
    y = layer.prompt(torch.randn(sum(lens), layer.hidden, generator=g, device="cuda"), seqs.prompt())
    last = y[torch.tensor(lens).cumsum(0) - 1]
    drawn = []
    if more:
        layer.fork(more)
        last = last.repeat_interleave(a.samples, 0)
        settings = dict(temperature=torch.full((count,), 0.8, device="cuda"), top_p=torch.full((count,), 0.9, device="cuda"))
    torch.cuda.synchronize()
    t = time.perf_counter()
    for _ in range(a.steps):
        if more:
            tokens, x = layer.draw(last, torch.rand(count, generator=g, device="cuda"), **settings)
            drawn.append(tokens)
            last = layer.step(x, more.step(), more.groups)
        else:
            last = layer.step(last, seqs.step())
    torch.cuda.synchronize()
    t = (time.perf_counter() - t) / max(a.steps, 1)
    layer.kv.status()
    hits = layer.moe.stats()["buckets"][0]
    print(f"{len(lens)} prompts of {lens} tokens, {a.steps} steps: {t * 1e6:.0f} us a step, "
          f"{layer.kv.info()['page_bytes']} bytes a page of 16 tokens, expert hits {hits['hits']} misses {hits['misses']}")
    if drawn:
        print("tokens of the first continuations:", torch.stack(drawn, 1)[: a.samples, :8].tolist())
    layer.close()


if __name__ == "__main__":
    main()
