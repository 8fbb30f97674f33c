"""Edges of the attention operators' contracts.

Attention over the cache where value blocks lie far apart: between blocks of
dimensions, between tokens that some rows of a call see and others do not, and
in places that no row sees. Elementwise within the bound of the definition
(attn_reference.py), which counts a dimension's own values only; what a row does
not see must not change a bit of it. Then calls of fewer rows than the batch
describes, infinite values of prompts wherever they lie, and calls one behind
the other.
"""
import math

import pytest

from harness import cuda_available

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not cuda_available(), reason="needs a CUDA GPU")]

torch = pytest.importorskip("torch")
import attn_reference as ref  # noqa: E402
import paged_expert_cache_gb300 as pec  # noqa: E402
from test_gpu_attention import Paged, check, cumulative, prompt_inputs  # noqa: E402


def expect(P, q, new, scale, **kw):
    want, bound = ref.attend(q, P.split(ref.held(P.k)), P.split(ref.held(P.v)), new, scale)
    check(P.attend(q, new, scale=scale), want, bound, **kw)
    P.cache.status()


@pytest.mark.parametrize("quiet", [1.0, 0.05, 1e-4])
@pytest.mark.parametrize("dim", [64, 128])
def test_finite_values_past_the_lengths_do_not_touch_a_row(dim, quiet):
    # what an earlier sequence left behind in the last cell of a page
    P = Paged([100, 37, 64, 1], 8, 2, dim, page=32, seed=61, scale_v=quiet).fill()
    used = set(P.table.flatten().tolist())
    P.table[P.table < 0] = next(i for i in range(P.pages) if i not in used)
    q = P.q([1, 1, 1, 1])
    clean = P.attend(q, [1, 1, 1, 1])
    for loud in (4e5, 30.0, 1e-6):
        left = torch.full((4 * 4, 2, dim), loud, device="cuda").bfloat16()
        left[::2, :, ::3] *= -1
        P.lens.add_(4)
        P.cache.append(0, None, left, left, P.batch([4] * 4))
        P.lens.sub_(4)
        assert torch.equal(P.attend(q, [1, 1, 1, 1]), clean)


@pytest.mark.parametrize("dim,hq", [(64, 8), (128, 8), (128, 1)])
def test_values_of_a_later_row_do_not_touch_an_earlier_one(dim, hq):
    # rows of one call that share their tiles: the last token's values are 4e5, the earlier rows do not see it
    new = [4, 3]
    outs = []
    for loud in (1.0, 4e5, 1e-7):
        P = Paged([300, 43], hq, 1, dim, page=16, seed=62, scale_v=0.05)
        P.v[299] *= loud
        P.v[342] *= loud
        P.fill()
        q = P.q(new)
        expect(P, q, new, dim ** -0.5)
        outs.append(P.attend(q, new))
    for out in outs[1:]:
        assert torch.equal(out[:3], outs[0][:3]) and torch.equal(out[4:6], outs[0][4:6])


@pytest.mark.parametrize("loud", [30.0, 1e4, 1e5, 1e7])
@pytest.mark.parametrize("dim,hq,new", [(64, 8, 1), (128, 8, 1), (128, 8, 4), (64, 2, 1)])
def test_a_loud_block_of_dimensions_beside_quiet_ones(dim, hq, new, loud):
    P = Paged([700, 90, 5], hq, 1, dim, page=16, seed=63, scale_v=0.01)
    P.v[..., 32:64] *= loud
    P.fill()
    expect(P, P.q([new] * 3), [new] * 3, dim ** -0.5)


@pytest.mark.parametrize("quiet", [1e-3, 1e-5])
def test_quiet_blocks_in_a_long_context(quiet):
    # weights far apart as well: scores of spread 3, so that most of a row's mass may lie on light tokens
    P = Paged([6000], 4, 1, 128, page=64, seed=64)
    P.v[..., 64:] *= quiet
    P.fill()
    expect(P, P.q([1]), [1], 3 * 128 ** -0.5)


def test_loud_tokens_that_later_ones_outweigh():
    # the loud tokens come first, and the scores climb until their weight is nothing
    P = Paged([900, 900], 4, 1, 128, page=32, seed=65, scale_v=0.02)
    P.v[:40] *= 1e7
    P.v[900:940, :, :32] *= 1e6
    q = torch.zeros(2, 4, 128, device="cuda").bfloat16()
    q[..., 0] = 8.0
    P.k.zero_()
    P.k[:, 0, 0] = torch.linspace(-60, 60, 900, device="cuda").bfloat16().repeat(2)
    P.fill()
    expect(P, q, [1, 1], 0.125, l2=False)


@pytest.mark.parametrize("at", [3, 450])
def test_a_loud_token_that_one_head_weighs_and_another_does_not(at):
    P = Paged([800], 8, 1, 128, page=32, seed=66, scale_v=0.02)
    P.v[at] *= 1e7
    P.k[at, 0, 0] = 40.0
    P.fill()
    q = P.q([1])
    q[0, ::2, 0], q[0, 1::2, 0] = 8.0, -8.0
    expect(P, q, [1], 128 ** -0.5)


@pytest.mark.parametrize("loud", [100.0, 1e5])
def test_one_loud_dimension_of_one_token(loud):
    # its block's other dimensions are zero in that token, and keep the other tokens' precision
    P = Paged([500, 20], 8, 1, 64, page=16, seed=67, scale_v=0.05)
    P.v[7, 0, 3] = P.v[510, 0, 40] = loud
    P.fill()
    expect(P, P.q([1, 1]), [1, 1], 64 ** -0.5)


@pytest.mark.parametrize("dim,new", [(64, [1, 4, 2]), (128, [3, 4]), (128, [9])])
def test_the_first_rows_of_a_batch_see_what_they_see_in_the_whole_call(dim, new):
    P = Paged([100, 64, 9][:len(new)], 8, 2, dim, page=32, seed=70).fill()
    q = P.q(new)
    want, bound = ref.attend(q, P.split(ref.held(P.k)), P.split(ref.held(P.v)), new, dim ** -0.5)
    for T in range(1, sum(new) + 1):
        out = torch.full((T, 8, dim), 7.0, dtype=torch.bfloat16, device="cuda")
        P.cache.attend(0, q[:T], P.batch(new), out)
        check(out, want[:T], bound[:T])
        # the same rows are written and read back by calls of as many
        k, v = (x[P.cu_list[1] - new[0]:P.cu_list[1]][:T] for x in (P.k, P.v))
        kh, vh = torch.empty_like(k), torch.empty_like(v)
        P.cache.append(0, None, k, v, P.batch(new))
        P.cache.read(0, P.batch(new), kh, vh)
        assert torch.equal(kh, ref.held(k).bfloat16()) and torch.equal(vh, ref.held(v).bfloat16())
    P.cache.status()


@pytest.mark.parametrize("dim,hkv", [(64, 1), (64, 64), (128, 1), (128, 40)])  # halves of one tile's keys, and pairs
@pytest.mark.parametrize("low,what", [(-60.0, math.inf), (40.0, math.inf), (40.0, -math.inf), (-60.0, math.nan)])
def test_an_infinite_value_meets_its_weight_wherever_it_lies(dim, hkv, low, what):
    # token 10's score is 20 or 120 below the others': its weight is 2^-29, or 2^-173, which is 0 in fp32. Its value is
    # behind the diagonal of the first rows' tile, and in a tile that later rows see all of.
    n = 300
    q, k, v = prompt_inputs([n], [n], hkv, hkv, dim, seed=71)
    q.zero_(), k.zero_()
    q[..., 0] = 8.0
    k[..., 0] = 60.0
    k[10, :, 0] = low
    clean, out = torch.empty_like(q), torch.empty_like(q)
    pec.attention_prompt(q, k, v, clean, cumulative([n]), scale=0.125)
    v[10, :, 5] = what
    pec.attention_prompt(q, k, v, out, cumulative([n]), scale=0.125)
    assert torch.equal(out[:10], clean[:10])
    assert torch.equal(out[:, :, :5], clean[:, :, :5]) and torch.equal(out[:, :, 6:], clean[:, :, 6:])
    hit = out[10:, :, 5]
    assert (hit == what).all() if low > 0 else hit.isnan().all()


@pytest.mark.parametrize("dim,B", [(128, 1), (64, 24)])
def test_calls_in_a_row_read_what_the_call_before_wrote(dim, B):
    # 60 steps in one graph, each with its own lengths, pages and queries in the same buffers, as a decode loop has them
    steps, hq, hkv, page = 60, 8, 2, 16
    kv = [100 + 3 * b for b in range(B)]
    P = Paged([n + steps for n in kv], hq, hkv, dim, page, seed=72)
    tables = torch.stack([P.table[torch.randperm(B, generator=P.g, device="cuda")] for _ in range(steps)])
    lens = torch.randint(20, 100, (steps, B), generator=P.g, device="cuda").to(torch.int32)
    qkv = torch.randn(steps, B, hq + 2 * hkv, dim, generator=P.g, device="cuda").bfloat16()
    rope = ref.rope_table(400, dim).cuda()
    table, kv_lens, x = torch.empty_like(tables[0]), torch.empty_like(lens[0]), torch.empty_like(qkv[0])
    batch = pec.KVBatch(torch.arange(B + 1, dtype=torch.int32, device="cuda"), kv_lens, table)
    turned, out = (torch.empty(B, hq, dim, dtype=torch.bfloat16, device="cuda") for _ in range(2))

    def run(outs, wait):
        P.fill()
        for s in range(steps):
            table.copy_(tables[s]), kv_lens.copy_(lens[s]), x.copy_(qkv[s])
            wait()
            P.cache.append(0, x[:, :hq], x[:, hq:hq + hkv], x[:, hq + hkv:], batch, rope=rope, q_out=turned)
            wait()
            P.cache.attend(0, turned, batch, out)
            pec.attention_prompt(turned, x[:, hq:hq + hkv], x[:, hq + hkv:], x[:, :hq].contiguous(), batch.cu_tokens)
            wait()
            outs[s].copy_(out)

    want, got = (torch.zeros(steps, B, hq, dim, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    run(want, torch.cuda.synchronize)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run(got, lambda: None)
    for _ in range(5):
        got.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(got, want)
    P.cache.status()


@pytest.mark.skipif(cuda_available() and torch.cuda.device_count() < 2, reason="needs two CUDA devices")
@pytest.mark.parametrize("dim", [64, 128])
def test_one_process_runs_the_kernels_on_each_device(dim):
    outs = []
    for dev in (0, 1):
        with torch.cuda.device(dev):
            g = torch.Generator().manual_seed(80)
            q, k, v = (torch.randn(40, h, dim, generator=g).bfloat16().cuda() for h in (8, 2, 2))
            batch = pec.KVBatch(*(torch.tensor(x, dtype=torch.int32, device="cuda") for x in ([0, 40], [40], [[0]])))
            cache = pec.KVCache(pec.make_kv_config(1, 1, 8, 2, dim, device=dev))
            cache.append(0, None, k, v, batch)
            both = torch.empty(2, 40, 8, dim, dtype=torch.bfloat16, device="cuda")
            cache.attend(0, q, batch, both[0])
            pec.attention_prompt(q, k, v, both[1], batch.cu_tokens)
            outs.append(both.cpu())
    assert torch.equal(outs[0], outs[1])
    # a call on a cache of another device leaves the current one as it is
    with torch.cuda.device(0):
        cache.status()
        other = pec.KVCache(pec.make_kv_config(1, 1, 8, 2, dim, device=1))
        other.close()
        assert torch._C._cuda_getDevice() == 0
