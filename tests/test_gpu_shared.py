"""Attention for groups of sequences that share their first positions
(moe_kv_attend_shared), against the definition in 64 bits and moe_kv_attend.

Bounds, elementwise, with mass = sum p |v|: the output's rounding to bf16, 2^-8 of
it; weights and values rounded to fp16, 2^-11 each (the rest of a sequence: weights
twice), 2^-9 mass in all; a key rounded to fp16 moves a score by at most ds = 2^-11
scale sum |q k|, and so its share of the weights by a factor within exp(+-2 ds).
fp16 ends at steps of 2^-24: a weight, held as 2^6 at the largest or more, is off by
at most 2^-25 / 2^6 of that beside its rounding, 2^-31 sum |v| over the keys a row
sees; in the rest, where weights are held as 2^10 and multiplied by a block's scale
before they meet codes of at most 8, by 2^-25 (|v| + 8) / 2^10 each, below 2^-35 |v|
+ 2^-32.
"""
import math

import pytest

from harness import cuda_available

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not cuda_available(), reason="needs a CUDA GPU")]

torch = pytest.importorskip("torch")
import attn_reference as ref  # noqa: E402
import paged_expert_cache_gb300 as pec  # noqa: E402

L2_TOL = 4e-3  # as for moe_kv_attend: two roundings to bf16 would give 2.4e-3


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def cumulative(n):
    return i32([0] + torch.tensor(list(n)).cumsum(0).tolist())


class Shared:
    """groups: (positions in common, [each sequence's own positions]); whole pages of the common part are the same pages, in
    random order, the page that it ends in is each sequence's own. room: the table is so wide that common positions are read
    once for their group even in these small batches."""

    def __init__(self, groups, hq, hkv, dim, page=64, seed=0, k_scale=1.0, v_scale=1.0, change=None, room=True):
        g = self.g = torch.Generator(device="cuda").manual_seed(seed)
        self.hq, self.hkv, self.dim, self.page = hq, hkv, dim, page

        def rows(n, scale):
            return (torch.randn(n, hkv, dim, generator=g, device="cuda") * scale).bfloat16()

        self.members = [len(own) for _, own in groups]
        self.prefix = [P for P, _ in groups]
        self.first = [0] + torch.tensor(self.members).cumsum(0).tolist()
        self.kv = [P + n for P, own in groups for n in own]
        self.keys, self.values = [], []
        for P, own in groups:
            kp, vp = rows(P, k_scale), rows(P, v_scale)
            if change:
                change(kp, vp)
            for n in own:
                self.keys.append(torch.cat([kp, rows(n, k_scale)]))
                self.values.append(torch.cat([vp, rows(n, v_scale)]))
        pages = sum(P // page for P in self.prefix) + sum(-(-n // page) for n in self.kv)
        ids = torch.randperm(pages + 2, generator=torch.Generator().manual_seed(seed)).tolist()
        self.pages = pages + 2
        width = max(-(-n // page) for n in self.kv) + 1
        if room:
            width = max(width, -(-4 * (1 << 16) * 16 * 64 // (hkv * dim * page)) + 1)
        self.table = torch.full((len(self.kv), width), -1, dtype=torch.int32)
        b = 0
        for P, own in groups:
            common = [ids.pop() for _ in range(P // page)]
            for n in own:
                mine = common + [ids.pop() for _ in range(-(-(P + n) // page) - len(common))]
                self.table[b, : len(mine)] = torch.tensor(mine, dtype=torch.int32)
                b += 1
        self.table = self.table.cuda()
        self.lens = i32(self.kv)
        self.cache = pec.KVCache(pec.make_kv_config(1, self.pages, hq, hkv, dim, page_tokens=page))
        if sum(self.kv):
            self.cache.append(0, None, torch.cat(self.keys), torch.cat(self.values),
                              pec.KVBatch(cumulative(self.kv), self.lens, self.table))
        self.groups = pec.KVGroups(i32(self.first), i32(self.prefix))

    def batch(self, new):
        return pec.KVBatch(cumulative(new), self.lens, self.table)

    def q(self, new, scale=1.0):
        return (torch.randn(sum(new), self.hq, self.dim, generator=self.g, device="cuda") * scale).bfloat16()

    def attend(self, q, new, scale=None, groups=None):
        T = q.shape[0]
        out = torch.full((T, self.hq, self.dim), 7.0, dtype=torch.bfloat16, device="cuda")
        n = self.cache.shared_workspace(T).numel()
        room = torch.full((n + 512,), 0xA5, dtype=torch.uint8, device="cuda")  # NaN-free garbage, and a margin behind
        assert self.cache.attend_shared(0, q, self.batch(new), groups or self.groups, out, room[:n], scale=scale) is out
        assert (room[n:] == 0xA5).all()
        return out

    def plain(self, q, new, scale=None):
        out = torch.full((q.shape[0], self.hq, self.dim), 7.0, dtype=torch.bfloat16, device="cuda")
        return self.cache.attend(0, q, self.batch(new), out, scale=scale)

    def reference(self, q, new, scale):
        keys, values = ([ref.held(x) if len(x) else x.double() for x in part] for part in (self.keys, self.values))
        out = torch.zeros(*q.shape, dtype=torch.float64, device="cuda")
        bound = torch.zeros_like(out)
        at, many = 0, self.hq // self.hkv
        for n, k, v in zip(new, keys, values):
            kk, vv = k.transpose(0, 1).repeat_interleave(many, 0), v.transpose(0, 1).repeat_interleave(many, 0)
            qq = q[at:at + n].double().transpose(0, 1)
            s = torch.matmul(qq, kk.transpose(1, 2)) * scale
            hidden = torch.arange(k.shape[0], device="cuda") > (k.shape[0] - n + torch.arange(n, device="cuda"))[:, None]
            s = s.masked_fill(hidden, -math.inf)
            big = torch.matmul(qq.abs(), kk.abs().transpose(1, 2)).masked_fill(hidden, 0).amax(2) * abs(scale) if k.shape[0] else \
                torch.zeros(self.hq, n, device="cuda")
            p = torch.softmax(s, 2).nan_to_num(0.0)  # rows that see nothing are zero
            o, mass = torch.matmul(p, vv), torch.matmul(p, vv.abs())
            ds = (2.0 ** -11 + 2.0 ** -19) * big[..., None]
            few = 2.0 ** -30 * vv.abs().sum(1, keepdim=True) + 2.0 ** -32 * vv.shape[1] + 1e-30
            out[at:at + n] = o.transpose(0, 1)
            bound[at:at + n] = (2.0 ** -8 * o.abs() + (2.0 ** -9 + torch.expm1(2 * ds)) * mass + few).transpose(0, 1)
            at += n
        return out, bound

    def check(self, new, scale=None, q=None, l2=True, groups=None):
        q = self.q(new) if q is None else q
        got = self.attend(q, new, scale, groups)
        want, bound = self.reference(q, new, self.dim ** -0.5 if scale is None else scale)
        assert torch.isfinite(got).all()
        off = (got.double() - want).abs()
        assert (off <= bound).all(), f"{float((off / bound).max()):.3g} of the bound"
        if l2 and want.norm() > 0:
            err = float((got.double() - want).norm() / want.norm())
            assert err <= L2_TOL, err
        self.cache.status()
        assert torch.equal(got, self.attend(q, new, scale, groups))  # the same bits again
        return q, got


CASES = [  # groups, new tokens of each sequence, hq, hkv, dim, page
    ([(16, [1])], 1, 1, 1, 64, 64),
    ([(15, [1, 2])], 1, 4, 2, 128, 16),                                  # less than a cell in common
    ([(0, [5, 0, 17])], 1, 8, 1, 64, 16),
    ([(128, [1, 1])], 1, 8, 2, 128, 64),
    ([(129, [3, 70])], 1, 8, 2, 128, 64),
    ([(600, [1, 100, 30, 64])], 1, 32, 4, 128, 64),
    ([(2451, [9, 300, 77, 1, 2, 45, 12, 80, 81, 500, 17, 16, 33, 128, 129, 250])], 1, 32, 4, 128, 64),
    ([(777, [5] * 40)], 1, 28, 4, 128, 16),                              # 280 rows: two tiles of 128 and one of 24
    ([(333, [40] * 50)], 1, 8, 1, 64, 32),                               # two items of rows
    ([(1000, [4, 8, 300])], 4, 16, 16, 64, 32),                          # drafts
    ([(500, [7, 20]), (0, [33]), (131, [7]), (64, [50, 7, 9]), (17, [9])], 7, 12, 2, 128, 48),
    ([(4000, [1]), (50, [20, 1, 3])], 1, 40, 1, 128, 64),                # 40 heads a key head
    ([(20000, [1, 5])], 1, 16, 1, 64, 128),                              # one item over the whole GPU
    ([(9001, [4] * 8)], 4, 16, 16, 64, 32),
    ([(300, [3])], 2, 128, 1, 128, 64),                                  # 256 rows
    ([(260, [2, 2, 2])], 1, 129, 3, 64, 16),                             # 43 heads a key head
]


@pytest.mark.parametrize("groups,new,hq,hkv,dim,page", CASES)
def test_matches_the_definition(groups, new, hq, hkv, dim, page):
    S = Shared(groups, hq, hkv, dim, page, seed=len(groups) + hq)
    news = [min(new, n) for n in S.kv]
    q, got = S.check(news)
    # moe_kv_attend differs by its own bound and this one's
    plain = S.plain(q, news)
    assert float((got.double() - plain.double()).norm() / plain.double().norm().clamp_min(1e-30)) <= 2 * L2_TOL


@pytest.mark.parametrize("groups,new,hq,hkv,dim,page", CASES[:9])
def test_small_batches_are_attended_over_each_sequence_by_itself(groups, new, hq, hkv, dim, page):
    S = Shared(groups, hq, hkv, dim, page, seed=len(groups) + hq, room=False)
    news = [min(new, n) for n in S.kv]
    q, got = S.check(news)
    assert torch.equal(got, S.plain(q, news))
    more = torch.cat([q, q[:1]])  # a row past the batch
    got = S.attend(more, news)
    assert torch.equal(got, S.plain(more, news)) and (got[len(q):] == 7).all()


def test_some_sequences_without_new_tokens_and_rows_of_none():
    S = Shared([(300, [9, 20, 1]), (200, [4, 4])], 8, 2, 128, seed=3)
    new = [1, 0, 2, 0, 0]
    q = S.q(new)
    want, bound = S.reference(q, new, 128 ** -0.5)
    more = torch.cat([q, q])  # three rows past the batch
    got = S.attend(more, new)
    assert ((got[:3].double() - want).abs() <= bound).all() and (got[3:] == 7).all()
    fewer = S.attend(q[:2], new)  # the call's rows end inside a sequence's
    assert ((fewer.double() - want[:2]).abs() <= bound[:2]).all()


@pytest.mark.parametrize("dim", [64, 128])
def test_rows_that_lie_among_the_common_positions(dim):
    # a second sequence that holds fewer positions than are named as common, and rows that see a part of them each
    S = Shared([(400, [6, 6])], 8, 2, dim, page=32, seed=4)
    for length in (1, 16, 100, 128, 129, 300, 399, 400):
        S.lens.copy_(i32([406, length]))
        for n in (1, min(length, 5)):
            new = [2, n]
            q = S.q(new)
            keep = S.keys, S.values
            S.keys, S.values = ([keep[i][0], keep[i][1][:length]] for i in (0, 1))
            want, bound = S.reference(q, new, dim ** -0.5)
            S.keys, S.values = keep
            got = S.attend(q, new)
            assert ((got.double() - want).abs() <= bound).all(), length


def test_rows_that_see_nothing_are_zero():
    S = Shared([(64, [2, 3])], 4, 2, 64, seed=5)
    S.lens.copy_(i32([66, 0]))
    q = S.q([1, 3])
    out = S.attend(q, [1, 3])
    assert (out[1:] == 0).all() and not (out[0] == 0).all()
    S.lens.copy_(i32([0, 67]))  # the first sequence holds nothing: nothing is in common
    out = S.attend(q, [1, 3])
    assert (out[0] == 0).all() and torch.equal(out[1:], S.plain(q, [1, 3])[1:])


def test_prefix_lens_beyond_what_is_held_and_groups_beyond_the_batch():
    S = Shared([(256, [9, 40]), (100, [5])], 8, 2, 128, seed=6)
    new = [1, 1, 1]
    q = S.q(new)
    plain = S.plain(q, new)

    def close(groups):
        got = S.attend(q, new, groups=groups)
        assert float((got.double() - plain.double()).norm() / plain.double().norm()) <= 2 * L2_TOL
        return got

    close(pec.KVGroups(i32([0, 1, 2, 3]), i32([10 ** 9, 2 ** 31 - 1, 0])))  # groups of one: all they hold is in common
    close(pec.KVGroups(i32([2, 3]), i32([100])))       # sequences before the first group
    close(pec.KVGroups(i32([0, 2]), i32([256])))       # and behind the last one
    assert torch.equal(close(pec.KVGroups(i32([0, 3]), i32([-5]))), plain)
    assert torch.equal(close(pec.KVGroups(i32([3, 9]), i32([64]))), plain)
    assert torch.equal(close(pec.KVGroups(i32([1, 1, 1]), i32([64, 64]))), plain)
    close(pec.KVGroups(i32([0, 2, 7]), i32([256, 96])))
    S.cache.status()


@pytest.mark.parametrize("q_scale,k_scale,v_scale", [(1e-6, 1.0, 1e-4), (1e6, 1e-5, 1e4), (30.0, 3.0, 1.0), (1e-20, 1e5, 1e-6),
                                                     (1e20, 1e-3, 30000.0), (1.0, 60000.0, 100000.0)])
@pytest.mark.parametrize("members", [2, 40])
def test_magnitudes(q_scale, k_scale, v_scale, members):
    S = Shared([(700, [3] * members)], 8, 2, 128, seed=7, k_scale=k_scale, v_scale=v_scale)
    spread = 12 if q_scale == 30.0 else 4
    S.check([1] * members, spread / (q_scale * k_scale * 128 ** 0.5), S.q([1] * members, q_scale))


@pytest.mark.parametrize("dim,hq", [(128, 8), (64, 4)])
@pytest.mark.parametrize("loud", [3e-6, 3e3, 9e4, 3e5])
def test_a_loud_block_of_dimensions_beside_quiet_ones(dim, hq, loud):
    def change(k, v):
        v[100:140, 0, :32] = (v[100:140, 0, :32].float() * loud).bfloat16()  # values past fp16's range / 8
        v[200, 0, 32:] = (v[200, 0, 32:].float() * loud).bfloat16()
        v[:, 1] = (v[:, 1].float() * 1e-5).bfloat16()
        v[199, 1, 5] = loud

    S = Shared([(600, [9, 30, 4]), (210, [5])], hq, 2, dim, page=32, seed=8, change=change)
    S.check([1] * 4, l2=False)


@pytest.mark.parametrize("loud", [3e4, 2e5])
def test_loud_keys_of_some_cells(loud):
    def change(k, v):
        k[70:75] = (k[70:75].float() * loud).bfloat16()
        k[400, 0, :5] = loud

    S = Shared([(600, [9, 30, 4])], 8, 2, 128, page=32, seed=9, change=change)
    q = S.q([1] * 3)
    q[..., :32] = 0  # rows do not see much of dims 0 .. 31
    S.check([1] * 3, 1e-4, q, l2=False)


def test_scores_that_climb_and_fall():
    def change(k, v):
        k.zero_()
        n = k.shape[0]
        k[:, :, 0] = torch.linspace(-60, 60, n, device="cuda")[:, None].bfloat16()
        k[: n // 2] = k[: n // 2].flip(0)

    S = Shared([(1500, [5, 9, 70])], 8, 2, 64, page=32, seed=10, change=change)
    q = torch.zeros(3, 8, 64, device="cuda").bfloat16()
    q[..., 0] = 8.0
    S.check([1] * 3, 0.125, q, l2=False)
    q[..., 0] = -8.0
    S.check([1] * 3, 0.125, q, l2=False)


def test_a_scale_of_zero_averages_what_is_seen():
    S = Shared([(300, [7, 20])], 4, 2, 64, page=32, seed=11)
    S.check([2, 1], 0.0)


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("what", [math.nan, math.inf])
def test_nan_and_infinities_touch_the_rows_that_see_them(dim, what):
    S = Shared([(300, [6, 6, 6])], 8, 2, dim, page=32, seed=12)
    new = [1, 1, 1]
    S.lens.copy_(i32([306, 200, 306]))
    q = S.q(new)
    clean = S.attend(q, new)
    k, v = S.keys[0][:300].clone(), S.values[0][:300].clone()
    v[250, 1, 40] = what  # a block's; the second sequence holds 200 positions
    k[290, 0, 3] = what
    S.cache.append(0, None, k, v, pec.KVBatch(i32([0, 300]), i32([300]), S.table[:1].contiguous()))
    S.cache.append(0, None, k[288:], v[288:], pec.KVBatch(i32([0, 12]), i32([300]), S.table[2:].contiguous()))
    got = S.attend(q, new)
    assert torch.equal(got[1], clean[1])
    for t in (0, 2):
        assert got[t, :4].isnan().all()                       # the key's head
        assert got[t, 4:, 32:64].isnan().all()                # the value's block of dims
        rest = [d for d in range(dim) if not 32 <= d < 64]
        assert torch.equal(got[t, 4:][:, rest], clean[t, 4:][:, rest])


def test_queries_with_nan_keep_to_their_rows():
    S = Shared([(500, [6] * 5)], 8, 2, 128, seed=13)
    q = S.q([1] * 5)
    clean = S.attend(q, [1] * 5)
    q[2, 3, 7], q[4, 0, 0] = math.nan, math.inf
    got = S.attend(q, [1] * 5)
    assert got[2, 3].isnan().all() and got[4, 0].isnan().all()
    got[2, 3], got[4, 0] = clean[2, 3], clean[4, 0]
    assert torch.equal(got, clean)


def test_pages_out_of_range_are_reported_and_not_read():
    S = Shared([(300, [6, 6, 6])], 8, 2, 128, page=32, seed=14)
    S.lens.copy_(i32([306, 150, 306]))
    new = [1, 1, 1]
    q = S.q(new)
    clean = S.attend(q, new)
    for bad in (-1, S.pages, 2 ** 31 - 1, -2 ** 31):
        S.table[0, 5] = bad  # positions 160 .. 191 of all
        got = S.attend(q, new)
        assert torch.equal(got[1], clean[1]) and got[0].isnan().all() and got[2].isnan().all()
        with pytest.raises(pec.MoeError):
            S.cache.status()
    S.cache.status()


def test_strided_queries_another_stream_and_graphs_with_other_contents():
    S = Shared([(700, [9, 40, 33]), (128, [70, 1])], 16, 4, 64, page=16, seed=15)
    new = [1] * 5
    q = S.q(new)
    clean = S.attend(q, new)
    wide = torch.randn(5, 20 * 64, device="cuda").bfloat16()
    wide[:, :16 * 64] = q.flatten(1)
    view = wide[:, :16 * 64].unflatten(1, (16, 64))
    assert torch.equal(S.attend(view, new), clean)
    side = torch.cuda.Stream()
    out, room = torch.empty_like(q), S.cache.shared_workspace(5)
    batch = S.batch(new)
    torch.cuda.synchronize()
    S.cache.attend_shared(0, q, batch, S.groups, out, room, stream=side)
    torch.cuda.synchronize()
    assert torch.equal(out, clean)
    graph = torch.cuda.CUDAGraph()
    qi = q.clone()
    with torch.cuda.graph(graph):
        S.cache.attend_shared(0, qi, batch, S.groups, out, room)
        S.cache.attend_shared(0, qi, batch, S.groups, out, room)  # twice in a row over one workspace
    for lens, cu, prefix in (([709, 740, 733, 198, 129], [0, 3, 5], [700, 128]), ([709, 40, 720, 150, 100], [0, 3, 5], [700, 128]),
                             ([709, 740, 733, 198, 129], [0, 2, 5], [640, 0])):
        S.lens.copy_(i32(lens))
        S.groups.cu_seqs.copy_(i32(cu))
        S.groups.prefix_lens.copy_(i32(prefix))
        qi.copy_(S.q(new))
        graph.replay()
        want = S.plain(qi, new)
        assert float((out.double() - want.double()).norm() / want.double().norm()) <= 2 * L2_TOL
    S.cache.status()


def test_many_groups_and_many_sequences():
    # more groups than a warp has lanes, more sequences than the kernel behind has threads
    S = Shared([(16 * (1 + i % 9), [1 + i % 5] * (1 + i % 11)) for i in range(70)], 4, 1, 64, page=16, seed=16)
    S.check([1] * len(S.kv))


def test_refusals_with_tensors_on_the_device():
    S = Shared([(100, [5, 5])], 4, 2, 64, seed=17)
    q = S.q([1, 1])
    out, room, batch = torch.empty_like(q), S.cache.shared_workspace(2), S.batch([1, 1])
    cpu = torch.zeros(2, dtype=torch.int32)
    calls = [(q, batch, S.groups, out, room[:-1]), (q, batch, S.groups, out, room[16:]), (q, batch, S.groups, out, room.cpu()),
             (q, batch, S.groups, out, None), (q, batch, None, out, room), (q, None, S.groups, out, room),
             (q.cpu(), batch, S.groups, out, room), (q.float(), batch, S.groups, out, room), (q, batch, S.groups, out[:1], room),
             (q, batch, S.groups, out, S.cache.shared_workspace(1)), (q, batch, S.groups, out, room[::2])]
    for args in calls:
        with pytest.raises(pec.MoeError) as e:
            S.cache.attend_shared(0, *args)
        assert e.value.status == pec.ERR_INVALID
    for scale in (-1.0, math.nan, math.inf):
        with pytest.raises(pec.MoeError):
            S.cache.attend_shared(0, q, batch, S.groups, out, room, scale=scale)
    with pytest.raises(pec.MoeError):
        S.cache.attend_shared(1, q, batch, S.groups, out, room)
    for cu, prefix in ((i32([0, 2, 2]), i32([1])), (i32([0]), i32([])), (i32([0, 2]).float(), i32([1])), (cpu, i32([1]))):
        with pytest.raises(pec.MoeError):
            pec.KVGroups(cu, prefix)
    empty = torch.empty(0, 4, 64, dtype=torch.bfloat16, device="cuda")
    S.cache.attend_shared(0, empty, S.batch([0, 0]), S.groups, empty, room)
