"""Sampling (moe_sample) against its definition in 64 bits: tokens have to be equal."""
import math

import pytest

import paged_expert_cache_gb300 as pec

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

B, F = torch.bfloat16, torch.float32


def reference(z, t, k, p, m, u):
    """One row on the host in fp64: (token, log of its share of the kept weights)."""
    z = z.double().cpu()
    rank = torch.argsort(z, descending=True, stable=True)
    if u is None or t == 0:
        return int(rank[0]), 0.0
    rank = rank[: int((z > -math.inf).sum())]
    if k > 0:
        rank = rank[:k]
    w = torch.exp((z[rank] - z[rank[0]]) / t)
    if p < 1:
        before = torch.cat([torch.zeros(1, dtype=torch.float64), w.cumsum(0)[:-1]])
        n = max(1, int((before < p * w.sum()).sum()))
        rank, w = rank[:n], w[:n]
    if m > 0:
        n = max(1, int((z[rank] >= z[rank[0]] + t * math.log(m)).sum()))
        rank, w = rank[:n], w[:n]
    upto = w.cumsum(0)
    i = min(int((upto <= u * upto[-1]).sum()), len(rank) - 1)
    return int(rank[i]), float((w[i] / upto[-1]).log())


def run(z, t=None, k=None, p=None, m=None, u=None, stream=None):
    T = z.shape[0]

    def array(v, dtype=F):
        return None if v is None else torch.as_tensor(v, dtype=dtype, device="cuda").expand(T).contiguous()

    a = dict(temperature=array(t), top_k=array(k, torch.int32), top_p=array(p), min_p=array(m), uniform=array(u))
    tokens = torch.full((T,), -7, dtype=torch.int32, device="cuda")
    logprobs = torch.full((T,), 7.0, device="cuda")
    pec.sample(z, tokens, a.pop("uniform"), logprobs=logprobs, stream=stream, **a)
    return tokens, logprobs


def check(z, t=None, k=None, p=None, m=None, u=None):
    tokens, logprobs = run(z, t, k, p, m, u)

    def row(v, default, i, dtype=F):
        if v is None:
            return default
        v = torch.as_tensor(v, dtype=dtype).expand(z.shape[0])[i]
        return v.item()  # as the kernel reads it, exact in fp64

    for i in range(z.shape[0]):
        token, lp = reference(z[i], row(t, 1.0, i), row(k, 0, i, torch.int32), row(p, 1.0, i), row(m, 0.0, i), row(u, None, i))
        assert int(tokens[i]) == token, (i, int(tokens[i]), token)
        # rounded once; sums of weights that are off by 2^-34 each
        assert abs(float(logprobs[i]) - lp) <= 2 ** -24 * abs(lp) + 2 ** -32, (i, float(logprobs[i]), lp)


def logits(T, V, dtype, seed, spread=2.0, peaks=True):
    g = torch.Generator(device="cuda").manual_seed(seed)
    z = torch.randn(T, V, generator=g, device="cuda") * spread - 3
    if peaks:
        z += (torch.rand(T, V, generator=g, device="cuda") < 30 / V) * 8 * torch.rand(T, V, generator=g, device="cuda")
    z[torch.rand(T, V, generator=g, device="cuda") < 0.02] = -math.inf
    z[:, 0] = 0.5  # a number in every row
    return z.to(dtype), torch.rand(T, generator=g, device="cuda")


@pytest.mark.parametrize("dtype", [B, F])
@pytest.mark.parametrize("V", [1, 2, 31, 1000, 4099, 50021, 131072])
@pytest.mark.parametrize("k,p,m", [(0, 1.0, 0.0), (40, 1.0, 0.0), (0, 0.9, 0.0), (0, 1.0, 0.05), (50, 0.95, 0.01), (3000, 0.99, 0.0),
                                   (1, 1.0, 0.0), (0, 0.0, 0.0), (0, 0.999, 0.001)])
def test_filters(dtype, V, k, p, m):
    z, u = logits(5, V, dtype, V + k)
    check(z, 0.8, k, p, m, u.cpu())


@pytest.mark.parametrize("dtype", [B, F])
@pytest.mark.parametrize("T,V", [(1, 200003), (3, 262144), (160, 3001), (700, 640)])
def test_settings_of_each_row(dtype, T, V):
    z, u = logits(T, V, dtype, T)
    g = torch.Generator().manual_seed(T)

    def choice(*v):
        return torch.tensor(v)[torch.randint(len(v), (T,), generator=g)]

    check(z, choice(0.0, 0.3, 1.0, 1.7), choice(0, 1, 7, 100, 2000, V, V + 5, -3), choice(1.0, 0.5, 0.9, 0.99, 2.0, -1.0),
          choice(0.0, 0.02, 0.5, 1.0, 3.0, -1.0), u.cpu())


@pytest.mark.parametrize("dtype", [B, F])
@pytest.mark.parametrize("V", [100, 70001])
def test_flat_rows_are_drawn_in_the_order_of_their_indexes(dtype, V):
    T = 64
    z = torch.full((T, V), -2.5, dtype=dtype, device="cuda")
    u = (torch.arange(T) + 0.5) / T
    tokens, logprobs = run(z, 0.7, u=u)
    assert tokens.tolist() == [int(float(x) * V) for x in u]
    assert (logprobs.double() + math.log(V)).abs().max() <= 2 ** -24 * math.log(V) + 1e-9
    tokens, _ = run(z, 0.7, k=10, u=u)  # the lowest indexes among equals
    assert tokens.tolist() == [int(float(x) * 10) for x in u]
    tokens, _ = run(z, 0.7, p=0.25, u=u)
    n = -(-V // 4)
    assert tokens.tolist() == [int(float(x) * n) for x in u]
    assert run(z)[0].tolist() == [0] * T


@pytest.mark.parametrize("dtype", [B, F])
@pytest.mark.parametrize("V", [300, 9000])
@pytest.mark.parametrize("spread", [1e-30, 1e-37, 1e-39])
def test_rows_that_are_nearly_flat(dtype, V, spread):
    T = 12
    g = torch.Generator(device="cuda").manual_seed(V)
    z = (torch.randn(T, V, generator=g, device="cuda") * 8).round().mul(spread).to(dtype)
    u = (torch.arange(T) + 0.3) / T
    for k, p, m in [(1, 1.0, 0.0), (3, 1.0, 0.0), (250, 0.7, 0.0), (0, 0.9, 0.0), (0, 1.0, 1.0), (0, 1.0, 0.0)]:
        check(z, 1.0, k, p, m, u)


@pytest.mark.parametrize("dtype", [B, F])
def test_a_cut_inside_a_run_of_equals(dtype):
    V = 9000
    z = torch.zeros(40, V, device="cuda")
    z[:, 100::7] = 1.0     # 1272 equal tokens behind two larger ones
    z[:, 5000] = z[:, 77] = 2.0
    u = (torch.arange(40) + 0.5) / 40
    for k in (1, 2, 3, 500, 1273, 1274, 1275, 4000):
        check(z.to(dtype), 1.0, k, 1.0, 0.0, u)
    for p in (0.001, 0.01, 0.2, 0.3, 0.31, 0.9):
        check(z.to(dtype), 1.0, 0, p, 0.0, u)


@pytest.mark.parametrize("dtype", [B, F])
def test_masks_of_the_lowest_value_and_of_minus_infinity(dtype):
    z, u = logits(6, 20000, F, 3)
    z[:, ::3] = torch.finfo(dtype).min
    z[1, 1:] = -math.inf                       # one token left
    z[2] = torch.finfo(dtype).min              # all equal, at the lowest
    z[3, 10:] = torch.finfo(dtype).min
    z[4] = -math.inf
    z[4, 19999] = -3e38
    z[5, 6] = torch.finfo(dtype).max
    z = z.to(dtype)
    for k, p, m in ((0, 1.0, 0.0), (50, 0.9, 0.0), (30, 1.0, 0.1), (0, 0.5, 0.0)):
        check(z, 1.0, k, p, m, u.cpu())


@pytest.mark.parametrize("dtype", [B, F])
def test_rows_without_a_distribution(dtype):
    z, u = logits(8, 3000, dtype, 4)
    z[0] = -math.inf
    z[1, 17] = math.nan
    z[2, 2999] = math.inf
    t = torch.ones(8)
    p, m = torch.ones(8), torch.zeros(8)
    t[3], t[4] = -1.0, math.nan
    p[5], m[6] = math.nan, math.nan
    for uniform in (u, None):
        tokens, logprobs = run(z, t, 20, p, m, uniform)
        assert tokens[:7].tolist() == [-1] * 7 and logprobs[:7].isnan().all()
        assert int(tokens[7]) == reference(z[7], 1.0, 20, 1.0, 0.0, None if uniform is None else float(u[7]))[0]
    t = torch.full((8,), math.inf)
    assert run(z, t, u=u)[0].tolist() == [-1] * 8
    u[7] = math.nan
    assert int(run(z, u=u)[0][7]) == -1


@pytest.mark.parametrize("t", [1e-30, 1e-6, 0.01, 30.0, 1e6, 1e30])
def test_temperatures(t):
    z, u = logits(6, 5000, F, 5)
    z[0, 7] = z[0, 4000] = 9.0  # two likeliest
    z[0].clamp_(max=9.0)
    check(z, t, 0, 1.0, 0.0, u.cpu())
    check(z, t, 0, 0.7, 0.0, u.cpu())


def test_the_ends_of_the_draw():
    z, _ = logits(4, 1000, F, 6)
    for u in (0.0, 1.0 - 2 ** -24, 1.0, -1.0, 2.0):
        tokens, _ = run(z, 1.0, 25, u=u)
        for i in range(4):
            rank = torch.argsort(z[i].cpu(), descending=True, stable=True)
            assert int(tokens[i]) == int(rank[0 if u <= 0 else 24]), u


def test_the_largest_vocabulary_is_right_beyond_what_shared_memory_holds():
    V = 1 << 20
    z, u = logits(2, V, F, 8, peaks=False)
    check(z, 1.0, 0, 1.0, 0.0, u.cpu())
    check(z, 1.0, 300000, 0.97, 0.0, u.cpu())


@pytest.mark.parametrize("dtype", [B, F])
@pytest.mark.parametrize("offset,pad", [(1, 0), (8, 8), (3, 2)])
def test_rows_of_wider_tensors(dtype, offset, pad):
    z, u = logits(5, 7001, dtype, 9)
    wide = torch.full((5, 7001 + offset + pad), 50.0, dtype=dtype, device="cuda")
    wide[:, offset:offset + 7001] = z
    check(wide[:, offset:offset + 7001], 0.9, 0, 0.9, 0.0, u.cpu())


def test_signed_zeros_are_equal():
    z = torch.zeros(32, 64, device="cuda")
    z[:, ::2] = -0.0
    u = (torch.arange(32) + 0.5) / 32
    assert run(z, u=u)[0].tolist() == [2 * i + 1 for i in range(32)]
    assert run(z, k=3, u=u)[0].tolist() == [int(float(x) * 3) for x in u]


def test_streams_graphs_and_repeats_give_the_same():
    z, u = logits(33, 40000, B, 10)
    first = run(z, 0.9, 0, 0.95, 0.0, u)
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    got = [run(z, 0.9, 0, 0.95, 0.0, u, stream=s) for s in streams for _ in range(3)]
    torch.cuda.synchronize()
    for tokens, logprobs in got:
        assert torch.equal(tokens, first[0]) and torch.equal(logprobs, first[1])
    zi, ui = z.clone(), u.clone()
    tokens = torch.empty(33, dtype=torch.int32, device="cuda")
    top_k = torch.full((33,), 60, dtype=torch.int32, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        pec.sample(zi, tokens, ui, top_k=top_k)
    for seed in (11, 12):
        z2, u2 = logits(33, 40000, B, seed)
        zi.copy_(z2)
        ui.copy_(u2)
        graph.replay()
        assert tokens.tolist() == run(z2, k=60, u=u2)[0].tolist()


def test_no_rows():
    z = torch.empty(0, 100, device="cuda")
    assert pec.sample(z, torch.empty(0, dtype=torch.int32, device="cuda")).shape == (0,)


def test_refusals_with_tensors_on_the_device():
    z, t, f = torch.zeros(4, 64, device="cuda"), torch.zeros(4, dtype=torch.int32, device="cuda"), torch.zeros(4, device="cuda")
    calls = [((z, t.long()), {}), ((z, t[:3]), {}), ((z, t.cpu()), {}), ((z, None), {}), ((z.half(), t), {}), ((z.cpu(), t), {}),
             ((z.t(), t), {}), ((z[:, :1].expand(4, 64), t), {}), ((z, t, f.double()), {}), ((z, t, f.cpu()), {}), ((z, t, f[::2]), {}),
             ((z, t), dict(top_k=f)), ((z, t), dict(temperature=t)), ((z, t), dict(top_p=0.9)), ((z, t), dict(min_p=f[:1])),
             ((z, t), dict(logprobs=t)), ((torch.zeros(1, (1 << 20) + 1, device="cuda"), t[:1]), {})]
    for args, kw in calls:
        with pytest.raises(pec.MoeError) as e:
            pec.sample(*args, **kw)
        assert e.value.status == pec.ERR_INVALID, (args, kw)
