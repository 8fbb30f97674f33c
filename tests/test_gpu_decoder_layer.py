"""The example decoder layer (examples/decoder_layer.py): attention over the
paged 4-bit cache and the MoE FFN in one layer, prompts then steps, against the
same layer computed step by step with attention from its 64-bit definition.

The FFN is the package's own on both sides (its parity is tested elsewhere), so
what is compared is the layer's input to it: x plus the attention's output
projection. Attention is within 4e-3 (relative L2, two bf16 roundings); its
projection to bf16 adds one more.
"""
import os
import sys

import pytest

from harness import cuda_available

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not cuda_available(), reason="needs a CUDA GPU")]

torch = pytest.importorskip("torch")
sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
import attn_reference as ref  # noqa: E402


def test_prompts_and_steps_of_the_example_layer():
    from decoder_layer import DecoderLayer, Sequences
    lens = [60, 5, 133]
    seqs = Sequences(lens, 160, 16)
    layer = DecoderLayer(seqs, max_tokens=256)
    seen = []
    ffn = layer.ffn
    layer.ffn = lambda x: (seen.append(x), ffn(x))[1]
    keys, values = [None] * 3, [None] * 3

    def expected(x, new, positions):
        q, k, v = layer.project(x)
        pos = torch.tensor(positions, device="cuda")
        qr, kr = ref.rotate(q, layer.rope, pos).bfloat16(), ref.rotate(k, layer.rope, pos).bfloat16()
        prompt = keys[0] is None
        at = 0
        ks, vs = [], []
        for b, n in enumerate(new):
            rows = slice(at, at + n)
            held = [ref.held(kr[rows]), ref.held(v[rows])]
            keys[b] = held[0] if prompt else torch.cat([keys[b], held[0]])
            values[b] = held[1] if prompt else torch.cat([values[b], held[1]])
            ks.append(kr[rows] if prompt else keys[b])  # a prompt attends to its own bf16 keys
            vs.append(v[rows] if prompt else values[b])
            at += n
        o, _ = ref.attend(qr, ks, vs, new, layer.dim ** -0.5)
        return o.flatten(1) @ layer.w_out.double().T

    g = torch.Generator(device="cuda").manual_seed(9)
    x = torch.randn(sum(lens), layer.hidden, generator=g, device="cuda")
    want = expected(x, lens, [p for n in lens for p in range(n)])
    y = layer.prompt(x, seqs.prompt())
    assert y.shape == x.shape and torch.isfinite(y).all()
    got = (seen[-1] - x).double()
    assert (got - want).norm() / want.norm() <= 8e-3
    last = y[torch.tensor(lens).cumsum(0) - 1]
    for _ in range(4):
        want = expected(last, [1, 1, 1], list(seqs.lens))
        y = layer.step(last, seqs.step())
        got = (seen[-1] - last).double()
        assert (got - want).norm() / want.norm() <= 8e-3
        assert torch.isfinite(y).all()
        last = y
    layer.kv.status()
    assert layer.moe.stats()["buckets"][0]["calls"] == 4
    layer.close()
