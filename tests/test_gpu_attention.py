"""The paged Q4_0 key/value cache, attention over it and prompt attention, on
the GPU, against their definitions in 64 bits (attn_reference.py).

Stored blocks are compared value for value (their arithmetic is exact once the
rotated key is rounded); attention elementwise within the bound that the
reference derives from the roundings, and, where inputs are random, in relative
L2 within 4e-3: two roundings to bf16 (probabilities, output), each about
1.7e-3 in the mean square (2^-8 / sqrt 3 over the binade), give 2.4e-3.
"""
import math
import random

import pytest

from harness import cuda_available

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not cuda_available(), reason="needs a CUDA GPU")]

torch = pytest.importorskip("torch")
import attn_reference as ref  # noqa: E402
import paged_expert_cache_gb300 as pec  # noqa: E402

L2_TOL = 4e-3


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def cumulative(n):
    return i32([0] + list(torch.tensor(list(n)).cumsum(0)) if n else [0])


class Paged:
    """Sequences of random keys and values in a cache, pages in random order."""

    def __init__(self, kv, hq, hkv, dim, page=64, seed=0, spare=3, layers=1, scale_v=1.0, scale_k=1.0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.kv, self.hq, self.hkv, self.dim, self.page = kv, hq, hkv, dim, page
        self.g = g
        total = sum(kv)
        self.k = (torch.randn(total, hkv, dim, generator=g, device="cuda") * scale_k).bfloat16()
        self.v = (torch.randn(total, hkv, dim, generator=g, device="cuda") * scale_v).bfloat16()
        per = [-(-n // page) for n in kv]
        self.pages = sum(per) + spare
        ids = torch.randperm(self.pages, generator=g, device="cuda").to(torch.int32)
        width = max(max(per), 1) + 1
        self.table = torch.full((len(kv), width), -1, dtype=torch.int32, device="cuda")
        at = 0
        for b, n in enumerate(per):
            self.table[b, :n] = ids[at:at + n]
            at += n
        self.lens = i32(kv)
        self.cache = pec.KVCache(pec.make_kv_config(layers, self.pages, hq, hkv, dim, page_tokens=page))
        self.whole = pec.KVBatch(cumulative(kv), self.lens, self.table)
        self.cu_list = [0]
        for n in kv:
            self.cu_list.append(self.cu_list[-1] + n)

    def fill(self, layer=0):
        self.cache.append(layer, None, self.k, self.v, self.whole)
        return self

    def split(self, x):
        return [x[a:b] for a, b in zip(self.cu_list, self.cu_list[1:])]

    def batch(self, new):
        return pec.KVBatch(cumulative(new), self.lens, self.table)

    def q(self, new):
        return torch.randn(sum(new), self.hq, self.dim, generator=self.g, device="cuda").bfloat16()

    def attend(self, q, new, scale=None, layer=0):
        out = torch.full((q.shape[0], self.hq, self.dim), 7.0, dtype=torch.bfloat16, device="cuda")
        self.cache.attend(layer, q, self.batch(new), out, scale=scale)
        return out


def check(got, want, bound, l2=True):
    assert torch.isfinite(got).all()
    off = (got.double() - want).abs()
    worst = (off / bound.clamp_min(1e-30)).max().item() if off.numel() else 0.0
    assert worst <= 1.0, f"{worst:.3g} of the bound"
    if l2 and want.norm() > 0:
        err = ((got.double() - want).norm() / want.norm()).item()
        assert err <= L2_TOL, err


# ---------------------------------------------------------------------------
# append and read
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("dim,page,hq,hkv", [(128, 64, 32, 4), (64, 16, 7, 7), (128, 48, 5, 1), (64, 128, 12, 2)])
def test_append_rotates_and_stores_what_the_definition_says(dim, page, hq, hkv):
    new, ctx = [1, 0, 37, 5, 130], [0, 9, 15, 63, 77]
    kv = [a + b for a, b in zip(new, ctx)]
    P = Paged(kv, hq, hkv, dim, page, seed=1)
    T = sum(new)
    # parts of one fused projection: strided rows
    g = torch.Generator(device="cuda").manual_seed(5)
    fused = torch.randn(T, (hq + 2 * hkv) * dim, generator=g, device="cuda").bfloat16()
    q = fused[:, :hq * dim].unflatten(1, (hq, dim))
    k = fused[:, hq * dim:(hq + hkv) * dim].unflatten(1, (hkv, dim))
    v = fused[:, (hq + hkv) * dim:].unflatten(1, (hkv, dim))
    table = ref.rope_table(max(kv), dim).cuda()
    batch = P.batch(new)
    q_out, k_out, kh, vh = (torch.zeros(T, h, dim, dtype=torch.bfloat16, device="cuda") for h in (hq, hkv, hkv, hkv))
    assert P.cache.append(0, q, k, v, batch, rope=table, q_out=q_out, k_out=k_out) is q_out
    P.cache.read(0, batch, kh, vh)
    P.cache.status()
    pos = torch.cat([torch.arange(c, c + n) for c, n in zip(ctx, new)]).cuda()
    for got, x in ((q_out, q), (k_out, k)):
        want = ref.rotate(x, table, pos)
        big = x.double().abs()
        big = big + torch.cat([big[..., dim // 2:], big[..., :dim // 2]], -1)
        # three fp32 roundings of terms no larger than the pair, then one to bf16
        low, high = ((want + e).bfloat16() for e in (-2.0 ** -22 * big, 2.0 ** -22 * big))
        assert ((low <= got) & (got <= high)).all()
        # and the same bits as separate fp32 products and sums
        c, s = table[pos][:, None].chunk(2, -1)
        a, b = x.float().chunk(2, -1)
        assert torch.equal(got, torch.cat([a * c - b * s, b * c + a * s], -1).bfloat16())
    # the blocks of the rounded keys, exactly; read back rounded once to bf16
    assert torch.equal(kh, ref.held(k_out).bfloat16())
    assert torch.equal(vh, ref.held(v).bfloat16())


def test_append_leaves_every_other_token_as_it_was():
    P = Paged([100, 40], 4, 2, 64, page=32, seed=2).fill()
    before = [torch.empty(140, 2, 64, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    after = [torch.empty_like(b) for b in before]
    P.cache.read(0, P.whole, *before)
    assert torch.equal(before[0], ref.held(P.k).bfloat16())
    k2, v2 = torch.randn(4, 2, 64, device="cuda").bfloat16(), torch.randn(4, 2, 64, device="cuda").bfloat16()
    P.cache.append(0, None, k2, v2, P.batch([3, 1]))  # positions 97..99 of the first, 39 of the second
    P.cache.read(0, P.whole, *after)
    for b, a, x in zip(before, after, (k2, v2)):
        b = b.clone()
        b[97:100], b[139] = ref.held(x).bfloat16()[:3], ref.held(x).bfloat16()[3]
        assert torch.equal(a, b)


@pytest.mark.parametrize("scale", [1e-7, 1e-3, 1.0, 3e4, 1e30])
def test_blocks_of_any_magnitude(scale):
    # below fp16's range a block's scale rounds to a subnormal or zero, above it the values saturate
    P = Paged([33], 1, 1, 128, seed=3, scale_k=scale, scale_v=scale).fill()
    k, v = (torch.empty(33, 1, 128, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    P.cache.read(0, P.whole, k, v)
    assert torch.equal(k, ref.held(P.k).bfloat16()) and torch.equal(v, ref.held(P.v).bfloat16())


def test_special_blocks():
    P = Paged([8], 1, 1, 64, seed=4)
    x = P.k
    x[0] = 0.0                                 # a zero block
    x[1, 0, :32] = torch.linspace(-4, 4, 32)   # an exact tie of the extremes: the positive one
    x[2, 0, 5] = math.inf
    x[3, 0, 40] = math.nan
    x[4, 0, :32], x[4, 0, 32:] = 1.5, -1.5     # one value throughout
    P.v.copy_(x)
    P.fill()
    k, v = (torch.empty(8, 1, 64, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    P.cache.read(0, P.whole, k, v)
    want = ref.held(x).bfloat16()
    assert want[2, 0, :32].isnan().all() and not want[2, 0, 32:].isnan().any()
    for got in (k, v):
        assert torch.equal(got.nan_to_num(99.0), want.nan_to_num(99.0))


def test_rows_past_the_batch_and_empty_calls_change_nothing():
    P = Paged([10, 5], 2, 1, 64, seed=5).fill()
    q = P.q([2, 1])
    more = torch.cat([q, q])  # three rows of no sequence
    out = P.attend(more, [2, 1])
    assert (out[3:] == 7.0).all() and torch.equal(out[:3], P.attend(q, [2, 1]))
    k = torch.randn(6, 1, 64, device="cuda").bfloat16()
    q_out = torch.full((6, 2, 64), 3.0, dtype=torch.bfloat16, device="cuda")
    P.cache.append(0, more, k, k, P.batch([2, 1]), rope=ref.rope_table(16, 64).cuda(), q_out=q_out)
    assert (q_out[3:] == 3.0).all() and not (q_out[:3] == 3.0).all()
    empty = torch.empty(0, 2, 64, dtype=torch.bfloat16, device="cuda")
    P.cache.attend(0, empty, P.batch([0, 0]), empty)
    P.cache.status()


def test_rows_before_the_first_sequence_belong_to_none():
    P = Paged([10, 5], 2, 1, 64, seed=6).fill()
    q = P.q([2, 1])
    clean = P.attend(q, [2, 1])
    batch = pec.KVBatch(i32([1, 3, 4]), P.lens, P.table)
    out = torch.full((4, 2, 64), 7.0, dtype=torch.bfloat16, device="cuda")
    P.cache.attend(0, torch.cat([q[:1], q]), batch, out)
    assert (out[0] == 7.0).all() and torch.equal(out[1:], clean)
    before = [torch.empty(15, 1, 64, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    after = [torch.empty_like(b) for b in before]
    P.cache.read(0, P.whole, *before)
    k = torch.cat([P.k[:1] * 3, P.k[8:10], P.k[14:]])  # the row of no sequence, then what is there already
    v = torch.cat([P.v[:1] * 3, P.v[8:10], P.v[14:]])
    P.cache.append(0, None, k, v, batch)
    P.cache.read(0, P.whole, *after)
    assert torch.equal(before[0], after[0]) and torch.equal(before[1], after[1])
    P.cache.status()


def test_the_stride_of_a_single_row_does_not_matter():
    P = Paged([77], 8, 2, 128, seed=7).fill()
    q = P.q([1])
    odd = torch.empty(1, 1, 8, 131, dtype=torch.bfloat16, device="cuda")[..., :128]  # not rows of this layout
    with pytest.raises(pec.MoeError):
        P.attend(odd[0], [1])
    view = q.as_strided((1, 8, 128), (3, 128, 1))
    assert torch.equal(P.attend(view, [1]), P.attend(q, [1]))


def test_tensors_off_the_device_are_refused():
    P = Paged([20], 4, 2, 64, seed=10).fill()
    q, out = P.q([1]), torch.empty(1, 4, 64, dtype=torch.bfloat16, device="cuda")
    k = P.k[19:]
    batch = P.batch([1])
    calls = [lambda: P.cache.attend(0, q.cpu(), batch, out), lambda: P.cache.attend(0, q.cpu(), batch, out.cpu()),
             lambda: P.cache.append(0, None, k.cpu(), k.cpu(), batch), lambda: P.cache.append(0, q, k, k, batch, q_out=out.cpu()),
             lambda: P.cache.append(0, q, k, k, batch, rope=torch.zeros(32, 64), q_out=out),
             lambda: P.cache.read(0, batch, k.cpu(), k.cpu()), lambda: P.cache.attend(0, q, None, out),
             lambda: pec.attention_prompt(q, k, k, out, batch.cu_tokens.cpu()),
             lambda: pec.attention_prompt(q.cpu(), k.cpu(), k.cpu(), out.cpu(), batch.cu_tokens.cpu())]
    for call in calls:
        with pytest.raises(pec.MoeError) as e:
            call()
        assert e.value.status == pec.ERR_INVALID


def test_a_scale_of_zero_averages_what_is_seen():
    P = Paged([300, 20], 4, 2, 64, page=32, seed=8).fill()
    q = P.q([2, 1])
    want, bound = ref.attend(q, P.split(ref.held(P.k)), P.split(ref.held(P.v)), [2, 1], 0.0)
    check(P.attend(q, [2, 1], scale=0.0), want, bound)
    lens = [40, 150]
    q, k, v = prompt_inputs(lens, lens, 4, 2, 64, seed=9)
    out = torch.empty_like(q)
    pec.attention_prompt(q, k, v, out, cumulative(lens), scale=0.0)
    want, bound = ref.attend(q, parts(k, lens), parts(v, lens), lens, 0.0)
    check(out, want, bound)


# ---------------------------------------------------------------------------
# attention over the cache
# ---------------------------------------------------------------------------
ATTEND = [  # kv lengths, new tokens, hq, hkv, dim, page
    ([1], [1], 1, 1, 64, 64),
    ([1, 2, 15, 16, 17], [1] * 5, 8, 1, 128, 16),
    ([63, 64, 65, 127, 128, 129, 200], [1] * 7, 32, 4, 128, 64),
    ([300, 0, 5], [1, 0, 1], 28, 4, 128, 48),
    ([1000], [1], 16, 16, 64, 32),
    ([700, 31], [4, 3], 12, 2, 64, 128),
    ([40, 17, 90], [40, 17, 5], 6, 2, 128, 16),  # whole prompts through the cache
    ([5000], [1], 40, 1, 128, 64),               # more heads to a key head than a tile has rows
    ([2100, 1, 333, 4097], [2, 1, 7, 1], 64, 8, 128, 64),
    ([12345], [3], 9, 3, 64, 1024),
]


@pytest.mark.parametrize("kv,new,hq,hkv,dim,page", ATTEND)
def test_attend_matches_the_definition(kv, new, hq, hkv, dim, page):
    P = Paged(kv, hq, hkv, dim, page, seed=11).fill()
    q = P.q(new)
    want, bound = ref.attend(q, P.split(ref.held(P.k)), P.split(ref.held(P.v)), new, dim ** -0.5)
    got = P.attend(q, new)
    check(got, want, bound)
    P.cache.status()
    assert torch.equal(got, P.attend(q, new))  # the same bits again


def test_attend_rows_that_see_nothing_are_zero():
    # more rows than the cache holds: the first ones sit before position 0
    P = Paged([2, 40], 4, 2, 64, seed=12).fill()
    P.lens.copy_(i32([2, 0]))
    q = P.q([5, 3])
    out = P.attend(q, [5, 3])
    assert (out[:3] == 0).all() and (out[5:] == 0).all()
    want, bound = ref.attend(q[3:5], [ref.held(P.k[:2])], [ref.held(P.v[:2])], [2], 64 ** -0.5)
    check(out[3:5], want, bound)
    P.cache.status()


@pytest.mark.parametrize("q_scale,k_scale,v_scale", [(1e-6, 1.0, 1e-4), (1e6, 1e-5, 1e4), (30.0, 3.0, 1.0),
                                                     (1e-20, 1e4, 1e-6), (1e20, 1e-3, 30000.0)])
def test_attend_magnitudes(q_scale, k_scale, v_scale):
    # the scale brings the scores to a spread of about 4 (20 for the third)
    P = Paged([333, 1500], 16, 2, 128, seed=13, scale_v=v_scale, scale_k=k_scale).fill()
    q = (P.q([1, 2]).double() * q_scale).bfloat16()
    scale = 4 / (q_scale * k_scale * 128 ** 0.5) if q_scale != 30.0 else 20 / (90 * 128 ** 0.5)
    want, bound = ref.attend(q, P.split(ref.held(P.k)), P.split(ref.held(P.v)), [1, 2], scale)
    check(P.attend(q, [1, 2], scale=scale), want, bound)


def test_attend_values_that_grow_and_shrink_along_the_context():
    # each token's values 2^e apart, e from -12 to 8: the running scale of the value blocks has to follow
    P = Paged([800, 800], 8, 1, 128, seed=14)
    e = torch.linspace(-12, 8, 800, device="cuda")
    f = torch.cat([e, e.flip(0)]).exp2()[:, None, None]
    P.v.copy_((P.v.float() * f).bfloat16())
    P.fill()
    q = P.q([1, 1])
    want, bound = ref.attend(q, P.split(ref.held(P.k)), P.split(ref.held(P.v)), [1, 1], 128 ** -0.5)
    check(P.attend(q, [1, 1]), want, bound)


def test_attend_scores_that_climb_and_fall():
    # the running maximum moves in every step, up in one sequence and down in the other
    P = Paged([640, 640], 4, 1, 64, seed=15)
    ramp = torch.linspace(-60, 60, 640, device="cuda")
    q = torch.zeros(2, 4, 64, device="cuda").bfloat16()
    q[..., 0] = 8.0
    P.k.zero_()
    P.k[:640, 0, 0], P.k[640:, 0, 0] = ramp.bfloat16(), ramp.flip(0).bfloat16()
    P.fill()
    want, bound = ref.attend(q, P.split(ref.held(P.k)), P.split(ref.held(P.v)), [1, 1], 0.125)
    check(P.attend(q, [1, 1], scale=0.125), want, bound, l2=False)


def test_nan_and_infinity_in_places_a_row_does_not_see():
    P = Paged([100, 37, 64], 8, 2, 128, page=32, seed=16).fill()
    q = P.q([1, 1, 1])
    clean = P.attend(q, [1, 1, 1])
    bad = torch.full((4, 2, 128), math.nan, device="cuda").bfloat16()
    bad[1] = math.inf
    # positions past the lengths, in the tiles that the sequences end in and in pages of their own
    P.table[P.table < 0] = P.pages - 1
    used = set(P.table.flatten().tolist())
    P.lens.add_(4)
    P.table[2, 2] = next(i for i in range(P.pages) if i not in used)
    P.cache.append(0, None, torch.cat([bad] * 3), torch.cat([bad] * 3), P.batch([4, 4, 4]))
    P.lens.sub_(4)
    assert torch.equal(P.attend(q, [1, 1, 1]), clean)
    # a later drafted token's, for the earlier rows of the same call
    P.lens.add_(1)
    out = P.attend(q.repeat_interleave(2, 0), [2, 2, 2])
    assert torch.isfinite(out[0::2]).all() and out[1::2].isnan().all()
    off = (out[0::2].double() - clean.double()).norm() / clean.double().norm()
    assert off <= L2_TOL  # the same rows, perhaps split another way


def test_pages_out_of_range_are_reported_and_not_read():
    P = Paged([100, 100], 4, 2, 64, page=32, seed=17).fill()
    q = P.q([1, 1])
    clean = P.attend(q, [1, 1])
    for wrong in (-1, P.pages, 2 ** 30):
        keep = P.table[0, 1].item()
        P.table[0, 1] = wrong
        out = P.attend(q, [1, 1])
        assert out[0].isnan().all() and torch.equal(out[1], clean[1])
        with pytest.raises(pec.MoeError) as e:
            P.cache.status()
        assert e.value.status == pec.ERR_INVALID
        P.cache.status()  # reported once
        k = torch.empty(200, 2, 64, dtype=torch.bfloat16, device="cuda")
        v = torch.empty_like(k)
        P.cache.read(0, P.whole, k, v)
        assert k[32:64].isnan().all() and v[32:64].isnan().all() and torch.isfinite(k[64:]).all()
        P.cache.append(0, None, P.k, P.v, P.whole)
        with pytest.raises(pec.MoeError):
            P.cache.status()
        P.table[0, 1] = keep
    assert torch.equal(P.attend(q, [1, 1]), clean)
    # lengths past the table, and positions past the rotation table
    P.lens[0] = 32 * P.table.shape[1] + 1
    assert P.attend(q, [1, 1])[0].isnan().all()
    P.lens[0] = 100
    q_out = torch.empty_like(q)
    P.cache.append(0, q, P.k[:2], P.v[:2], P.batch([1, 1]), rope=ref.rope_table(99, 64).cuda(), q_out=q_out)
    assert q_out.isnan().all()
    with pytest.raises(pec.MoeError):
        P.cache.status()


def test_layers_and_pages_past_32_bit_offsets():
    # 3 layers of 18 KiB pages, 100000 of them: the last layer lies past 3.6e9 bytes
    P = Paged([150, 64], 8, 8, 64, page=64, seed=18)
    P.cache.close()
    pages = 100000
    P.cache = pec.KVCache(pec.make_kv_config(3, pages, 8, 8, 64, page_tokens=64))
    assert P.cache.info()["page_bytes"] * pages * 2 > 2 ** 32
    P.table[0, :3], P.table[1, :1] = i32([pages - 1, 0, pages - 2]), i32([pages - 3])
    P.fill(layer=2)
    q = P.q([1, 1])
    want, bound = ref.attend(q, P.split(ref.held(P.k)), P.split(ref.held(P.v)), [1, 1], 0.125)
    check(P.attend(q, [1, 1], layer=2), want, bound)
    assert (P.attend(q, [1, 1], layer=1) == 0).all()  # another layer's pages stay zero
    P.cache.close()


def test_many_sequences():
    r = random.Random(3)
    kv = [r.randint(1, 40) for _ in range(1500)]
    new = [r.randint(0, 1) for _ in kv]
    P = Paged(kv, 4, 2, 64, page=16, seed=19).fill()
    q = P.q(new)
    k, v = P.split(ref.held(P.k)), P.split(ref.held(P.v))
    want, bound = ref.attend(q, k, v, new, 0.125)
    check(P.attend(q, new), want, bound)


def test_strided_queries_side_stream_and_graph():
    P = Paged([500, 77], 8, 2, 128, seed=20).fill()
    wide = torch.randn(2, 12, 128, device="cuda").bfloat16()
    q = wide[:, 2:10]
    clean = P.attend(q.contiguous(), [1, 1])
    assert torch.equal(P.attend(q, [1, 1]), clean)
    s = torch.cuda.Stream()
    batch, out = P.batch([1, 1]), torch.zeros_like(clean)
    s.wait_stream(torch.cuda.current_stream())
    P.cache.attend(0, q, batch, out, stream=s)
    s.synchronize()
    assert torch.equal(out, clean)
    with torch.cuda.stream(s):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            P.cache.append(0, None, P.k[498:500].contiguous(), P.v[498:500].contiguous(), batch)
            P.cache.attend(0, q, batch, out)
    torch.cuda.synchronize()
    P.fill()
    P.lens.copy_(i32([490, 60]))  # a replay reads the lengths of the day
    graph.replay()
    torch.cuda.synchronize()
    k, v = P.k.clone(), P.v.clone()
    k[489], k[559], v[489], v[559] = P.k[498], P.k[499], P.v[498], P.v[499]
    want, bound = ref.attend(q, [ref.held(k[:490]), ref.held(k[500:560])], [ref.held(v[:490]), ref.held(v[500:560])],
                             [1, 1], 128 ** -0.5)
    check(out, want, bound)


# ---------------------------------------------------------------------------
# prompt attention
# ---------------------------------------------------------------------------
PROMPT = [  # queries, keys, hq, hkv, dim
    ([1], None, 1, 1, 64),
    ([1, 2, 3, 15, 16, 17], None, 8, 1, 128),
    ([127, 128, 129], None, 4, 4, 128),
    ([300], None, 32, 4, 128),
    ([257, 0, 31, 200], None, 28, 4, 64),
    ([64, 10], [64, 500], 12, 2, 128),           # a chunk over its context
    ([1, 1, 1], [700, 1, 129], 16, 2, 64),
    ([40, 7], [20, 0], 6, 3, 128),               # rows that see nothing
    ([90], None, 40, 1, 64),
    ([130], None, 128, 1, 128),
    ([520], [900], 5, 5, 128),
    ([1100], None, 2, 1, 64),
    ([700, 0, 300, 129], None, 16, 16, 64),      # enough pairs of tiles for every SM
    ([260, 400, 77], [900, 400, 1], 24, 12, 128),
]


def prompt_inputs(lq, lk, hq, hkv, dim, seed=30):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return [torch.randn(sum(n), h, dim, generator=g, device="cuda").bfloat16()
            for n, h in ((lq, hq), (lk, hkv), (lk, hkv))]


def parts(x, lens):
    return list(torch.split(x, list(lens)))


@pytest.mark.parametrize("lq,lk,hq,hkv,dim", PROMPT)
def test_prompt_matches_the_definition(lq, lk, hq, hkv, dim):
    q, k, v = prompt_inputs(lq, lk or lq, hq, hkv, dim)
    out = torch.full_like(q, 7.0)
    cu = cumulative(lq)
    got = pec.attention_prompt(q, k, v, out, cu, cumulative(lk) if lk else None)
    assert got is out
    want, bound = ref.attend(q, parts(k, lk or lq), parts(v, lk or lq), lq, dim ** -0.5)
    check(out, want, bound)
    again = torch.empty_like(out)
    pec.attention_prompt(q, k, v, again, cu, cumulative(lk) if lk else None)
    assert torch.equal(out, again)


@pytest.mark.parametrize("dim,hq,hkv", [(128, 8, 2), (64, 3, 3)])
def test_prompt_strided_rows_and_rows_of_no_sequence(dim, hq, hkv):
    g = torch.Generator(device="cuda").manual_seed(31)
    fused = torch.randn(200, (hq + 2 * hkv) * dim, generator=g, device="cuda").bfloat16()
    q, k, v = (x.unflatten(1, (-1, dim)) for x in fused.split([hq * dim, hkv * dim, hkv * dim], 1))
    lens = [70, 101]
    out = torch.full((200, hq, dim), 7.0, dtype=torch.bfloat16, device="cuda")
    pec.attention_prompt(q, k, v, out, cumulative(lens))
    want, bound = ref.attend(q[:171], parts(k[:171], lens), parts(v[:171], lens), lens, dim ** -0.5)
    check(out[:171], want, bound)
    assert (out[171:] == 7.0).all()


@pytest.mark.parametrize("dim,hq,hkv,what", [(128, 8, 2, math.nan), (64, 4, 4, math.inf), (128, 1, 1, -math.inf),
                                             (64, 32, 32, math.nan), (128, 24, 12, math.inf)])
def test_prompt_keys_and_values_a_row_does_not_see_do_not_touch_it(dim, hq, hkv, what):
    lens = [150, 90, 300]
    q, k, v = prompt_inputs(lens, lens, hq, hkv, dim, seed=32)
    cu = cumulative(lens)
    clean, out = torch.empty_like(q), torch.empty_like(q)
    pec.attention_prompt(q, k, v, clean, cu)
    for first in (149, 100, 37):  # from this token of the first sequence on, and all of the second
        k2, v2 = k.clone(), v.clone()
        for x in (k2, v2):
            x[first:240] = what
        pec.attention_prompt(q, k2, v2, out, cu)
        assert torch.equal(out[:first], clean[:first]) and torch.equal(out[240:], clean[240:])
        assert not torch.isfinite(out[first:240]).any()
    # values alone: a visible infinity arrives in its own dimension only
    v2 = v.clone()
    v2[200, :, 5] = what
    pec.attention_prompt(q, k, v2, out, cu)
    assert torch.equal(out[:200], clean[:200]) and torch.equal(out[240:], clean[240:])
    assert torch.equal(out[200:240, :, :5], clean[200:240, :, :5])
    assert torch.equal(out[200:240, :, 6:], clean[200:240, :, 6:])
    hit = out[200:240, :, 5]
    assert hit.isnan().all() if what != what else (hit == what).all()


@pytest.mark.parametrize("hkv", [1, 16])  # one tile with two halves of its keys, and two tiles an item
def test_prompt_scores_that_climb_and_fall(hkv):
    lens = [640, 640]
    q, k, v = prompt_inputs(lens, lens, 4 * hkv, hkv, 64, seed=33)
    ramp = torch.linspace(-60, 60, 640, device="cuda")
    q.zero_(), k.zero_()
    q[..., 0] = 8.0
    k[:640, :, 0], k[640:, :, 0] = ramp.bfloat16()[:, None], ramp.flip(0).bfloat16()[:, None]
    out = torch.empty_like(q)
    pec.attention_prompt(q, k, v, out, cumulative(lens), scale=0.125)
    want, bound = ref.attend(q, parts(k, lens), parts(v, lens), lens, 0.125)
    check(out, want, bound, l2=False)


@pytest.mark.parametrize("lq,lk,hq,hkv,dim", [
    ([1500], None, 28, 4, 64),            # 18 tokens a tile: some tiles straddle a multiple of 128 keys
    ([700, 400], None, 12, 4, 64),        # 42 tokens a tile
    ([640, 320], [717, 397], 16, 4, 64),  # 32 tokens a tile after a context of 77
    ([1500, 900], None, 28, 4, 128),
])
def test_prompt_tiles_that_clean_several_key_tiles(lq, lk, hq, hkv, dim):
    # The first tile of an item cleans the values of two key tiles in a row, while the second, whose maxima climb in
    # every key tile, lags behind it: each cleaning still has to be met by both.
    lk = lk or lq
    q, k, v = prompt_inputs(lq, lk, hq, hkv, dim, seed=36)
    tokens = 128 // (hq // hkv)
    q.zero_(), k.zero_()
    for n, at in zip(lq, [0] + lq):
        second = torch.arange(n, device="cuda") // tokens % 2 == 1
        q[at:at + n, :, 0] = torch.where(second, 8.0, 0.0).bfloat16()[:, None]
    at = 0
    for n in lk:
        k[at:at + n, :, 0] = torch.linspace(-n / 20, n / 20, n, device="cuda").bfloat16()[:, None]
        at += n
    out, again = torch.empty_like(q), torch.empty_like(q)
    cu, cu_k = cumulative(lq), cumulative(lk)
    pec.attention_prompt(q, k, v, out, cu, cu_k, scale=0.125)
    want, bound = ref.attend(q, parts(k, lk), parts(v, lk), lq, 0.125)
    check(out, want, bound, l2=False)
    for _ in range(30):
        pec.attention_prompt(q, k, v, again, cu, cu_k, scale=0.125)
        assert torch.equal(out, again)


@pytest.mark.parametrize("scale_q,scale_v", [(1e-6, 1e-6), (1e4, 1e4), (1e15, 1e30)])
def test_prompt_magnitudes(scale_q, scale_v):
    lens = [200, 77]
    q, k, v = prompt_inputs(lens, lens, 8, 2, 128, seed=34)
    q, v = (q.double() * scale_q).bfloat16(), (v.double() * scale_v).bfloat16()
    out = torch.empty_like(q)
    scale = 3 / (scale_q * 128 ** 0.5)
    pec.attention_prompt(q, k, v, out, cumulative(lens), scale=scale)
    want, bound = ref.attend(q, parts(k, lens), parts(v, lens), lens, scale)
    check(out, want, bound)


def test_prompt_many_short_sequences():
    r = random.Random(4)
    lens = [r.randint(0, 30) for _ in range(1300)]
    q, k, v = prompt_inputs(lens, lens, 4, 2, 64, seed=35)
    out = torch.empty_like(q)
    pec.attention_prompt(q, k, v, out, cumulative(lens))
    want, bound = ref.attend(q, parts(k, lens), parts(v, lens), lens, 0.125)
    check(out, want, bound)


def test_prompt_no_keys_and_no_queries():
    q, k, v = prompt_inputs([5], [0], 4, 2, 128)
    out = torch.full_like(q, 7.0)
    pec.attention_prompt(q, k, v, out, cumulative([5]), cumulative([0]))
    assert (out == 0).all()
    empty = q[:0]
    pec.attention_prompt(empty, k, v, empty, cumulative([0]), cumulative([0]))


# ---------------------------------------------------------------------------
# the operators together
# ---------------------------------------------------------------------------
def test_prompt_then_decode_through_the_cache():
    # a prompt's attention, its tokens into the cache, then steps of one token over the cache; a chunk read back
    # from the cache and attended as a prompt gives what attending the cache gives
    hq, hkv, dim, page = 8, 2, 128, 16
    lens = [50, 21]
    table = ref.rope_table(128, dim).cuda()
    P = Paged([64, 32], hq, hkv, dim, page, seed=40)
    q, k, v = prompt_inputs(lens, lens, hq, hkv, dim, seed=41)
    P.lens.copy_(i32(lens))
    batch = P.batch(lens)
    qr, kr, out = torch.empty_like(q), torch.empty_like(k), torch.empty_like(q)
    P.cache.append(0, q, k, v, batch, rope=table, q_out=qr, k_out=kr)
    pec.attention_prompt(qr, kr, v, out, batch.cu_tokens)
    want, bound = ref.attend(qr, parts(kr, lens), parts(v, lens), lens, dim ** -0.5)
    check(out, want, bound)
    keys, values = [list(parts(x, lens)) for x in (ref.held(kr), ref.held(v))]
    for step in range(3):
        P.lens.add_(1)
        q, k, v = prompt_inputs([1, 1], [1, 1], hq, hkv, dim, seed=50 + step)
        qr, kr, out = torch.empty_like(q), torch.empty_like(k), torch.empty_like(q)
        one = P.batch([1, 1])
        P.cache.append(0, q, k, v, one, rope=table, q_out=qr, k_out=kr)
        P.cache.attend(0, qr, one, out)
        for b in range(2):
            keys[b] = torch.cat([keys[b], ref.held(kr[b:b + 1])])
            values[b] = torch.cat([values[b], ref.held(v[b:b + 1])])
        want, bound = ref.attend(qr, keys, values, [1, 1], dim ** -0.5)
        check(out, want, bound)
    total = [n + 3 for n in lens]
    every = P.batch(total)
    kh, vh = (torch.empty(sum(total), hkv, dim, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    P.cache.read(0, every, kh, vh)
    again = torch.empty_like(out)
    pec.attention_prompt(qr, kh, vh, again, cumulative([1, 1]), every.cu_tokens)
    assert ((again.double() - want).norm() / want.norm()).item() <= 2 * L2_TOL  # keys and values rounded to bf16 as well
    P.cache.status()
