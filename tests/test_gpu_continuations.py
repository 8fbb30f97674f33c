"""Continuations of shared prompts, as they are decoded: the example layer's steps
with moe_kv_attend_shared, moe_residual_norm and moe_sample, beside the same steps
with each operator's plain counterpart, and one step as a CUDA graph."""
import os
import subprocess
import sys

import pytest

from harness import cuda_available

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not cuda_available(), reason="needs a CUDA GPU")]

torch = pytest.importorskip("torch")
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
sys.path.insert(0, os.path.join(ROOT, "examples"))
from test_gpu_sample import reference as token_reference  # noqa: E402
import paged_expert_cache_gb300 as pec  # noqa: E402

LENS, SAMPLES, STEPS = [60, 5, 133], 4, 5


def decoder():
    from decoder_layer import Continuations, DecoderLayer, Sequences
    seqs = Sequences(LENS, 160, 16)
    more = Continuations(seqs, SAMPLES, 160, 16)
    layer = DecoderLayer(seqs, max_tokens=256, pages=more.pages)
    g = torch.Generator(device="cuda").manual_seed(9)
    y = layer.prompt(torch.randn(sum(LENS), layer.hidden, generator=g, device="cuda"), seqs.prompt())
    layer.fork(more)
    return layer, more, y[torch.tensor(LENS).cumsum(0) - 1].repeat_interleave(SAMPLES, 0), g


def test_steps_of_continuations():
    layer, more, last, g = decoder()
    n = len(LENS) * SAMPLES
    t, p = torch.full((n,), 0.9, device="cuda"), torch.full((n,), 0.95, device="cuda")
    seen = set()
    for _ in range(STEPS):
        u = torch.rand(n, generator=g, device="cuda")
        tokens, x = layer.draw(last, u, temperature=t, top_p=p)
        logits = layer.norm(last) @ layer.w_head.T
        want = [token_reference(logits[i], float(t[i]), 0, float(p[i]), 0.0, float(u[i]))[0] for i in range(n)]
        assert tokens.tolist() == want
        seen.add(tuple(want))
        # the norm, against its formula in 64 bits: half a step of bf16 and some fp32 roundings
        h = last.double() / (last.double().square().mean(-1, keepdim=True) + 1e-6).sqrt()
        assert ((layer.norm(last).double() - h).abs() <= h.abs() * (2 ** -8 + 2 ** -18)).all()
        batch = more.step()
        got = layer.step(x, batch, more.groups)
        # the same tokens once more without the groups (they are written again as they are)
        attend = layer.step(x, batch)
        # attention differs by two roundings of its output to bf16 and its own tolerance, 4e-3 each; the FFN routes
        # tokens, so single ones may take other experts where two are close
        err = ((got - attend).norm(dim=1) / attend.norm(dim=1)).sort().values
        assert float(err[: n * 3 // 4].max()) <= 2e-2, err
        assert torch.isfinite(got).all()
        last = got
    assert len(seen) == STEPS
    layer.kv.status()
    layer.close()


def test_a_step_as_a_graph_follows_lengths_and_draws():
    # append, attention, norm and draw captured once and replayed as the continuations grow
    layer, more, last, g = decoder()
    n, dim, hq = len(LENS) * SAMPLES, layer.dim, layer.q_heads
    u, x = torch.rand(n, generator=g, device="cuda"), last.clone()
    k = torch.empty(n, layer.kv_heads, dim, dtype=torch.bfloat16, device="cuda")
    q, v = torch.empty(n, hq, dim, dtype=torch.bfloat16, device="cuda"), torch.empty_like(k)
    qr, o, room = torch.empty_like(q), torch.empty_like(q), layer.kv.shared_workspace(n)
    h, tokens = torch.empty(n, layer.hidden, dtype=torch.bfloat16, device="cuda"), torch.empty(n, dtype=torch.int32, device="cuda")
    back, logits = torch.empty_like(h), torch.empty(n, 1000, dtype=torch.bfloat16, device="cuda")
    table = torch.nn.functional.pad(more.table, (0, 1 << 16), value=-1)  # wide: groups are read once though they are small
    batch = pec.KVBatch(more.step_cu, more.kv_lens, table)

    def step():
        layer.kv.append(0, q, k, v, batch, rope=layer.rope, q_out=qr)
        layer.kv.attend_shared(0, qr, batch, more.groups, o, room)
        pec.residual_norm(x, back, h)
        pec.sample(logits, tokens, u)

    def inputs():
        for t in (q, k, v, back, logits):
            t.copy_(torch.randn(t.shape, generator=g, device="cuda"))
        u.copy_(torch.rand(n, generator=g, device="cuda"))

    more.kv_lens += 1
    inputs()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for _ in range(3):
        more.kv_lens += 1
        inputs()
        before = x.clone()
        graph.replay()
        got = [t.clone() for t in (qr, o, x, h, tokens)]
        x.copy_(before)
        step()
        for a, b in zip(got, (qr, o, x, h, tokens)):
            assert torch.equal(a, b)
        plain = torch.empty_like(o)
        layer.kv.attend(0, qr, batch, plain)
        assert float((o.double() - plain.double()).norm() / plain.double().norm()) <= 8e-3
    layer.kv.status()
    layer.close()


FIRST = """
import torch, paged_expert_cache_gb300 as pec
B, n = torch.bfloat16, 2
kv = pec.KVCache(pec.make_kv_config(1, 16, 8, 2, 128, page_tokens=16))
i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")
table = torch.nn.functional.pad(i32([[0, 1, 2], [0, 1, 3]]), (0, 1 << 16))
k = torch.randn(80, 2, 128, device="cuda").to(B)
kv.append(0, None, k, k, pec.KVBatch(i32([0, 40, 80]), i32([40, 40]), table))
batch, groups = pec.KVBatch(i32([0, 1, 2]), i32([40, 40]), table), pec.KVGroups(i32([0, 2]), i32([32]))
q, x, z = torch.randn(n, 8, 128, device="cuda").to(B), torch.randn(n, 2048, device="cuda"), torch.randn(n, 50000, device="cuda")
o, h, t, room = torch.empty_like(q), torch.empty(n, 2048, dtype=B, device="cuda"), torch.empty(n, dtype=torch.int32, device="cuda"), kv.shared_workspace(n)
u = torch.rand(n, device="cuda")
def calls():
    kv.attend_shared(0, q, batch, groups, o, room)
    pec.residual_norm(x, out=h)
    pec.sample(z, t, u)
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    calls()
g.replay()
first = [v.clone() for v in (o, h, t)]
calls()
assert all(torch.equal(a, b) for a, b in zip(first, (o, h, t)))
kv.status()
print("same")
"""


def test_the_first_calls_of_a_process_may_be_captured():
    r = subprocess.run([sys.executable, "-c", FIRST], capture_output=True, text=True, timeout=300, cwd=ROOT)
    assert r.returncode == 0 and "same" in r.stdout, r.stderr


def test_the_example_runs():
    r = subprocess.run([sys.executable, os.path.join(ROOT, "examples", "decoder_layer.py"), "--steps", "4", "--samples", "3"],
                       capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr
    assert "tokens of the first continuations" in r.stdout
