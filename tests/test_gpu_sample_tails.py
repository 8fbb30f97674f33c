"""Sampling (moe_sample) of rows whose tokens are nearly all at the edge of what a
weight's unit holds: 29 to 31 below the top in units of the temperature.

A weight is off by at most 2^-34 of itself and 2^-44 of the row's largest, so a sum
of them by at most 2^-34 of itself and 2^-44 a token, with the largest weight 1. A
draw compares such a sum with `uniform` times another: the stretch of the token that
is drawn, made longer by three such bounds at either end (its own end's, the kept
sum's, and the rounding of their product, which is less), holds the point that exact
arithmetic gives.
"""
import math

import pytest

import paged_expert_cache_gb300 as pec

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


def rows(T, V, depth, temp, seed):
    """Two likely tokens, at random places, and all the others `depth` temperatures below the top."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    z = torch.full((T, V), -depth * temp, device="cuda")
    at = torch.rand(T, V, generator=g, device="cuda").topk(2).indices
    z[torch.arange(T, device="cuda"), at[:, 0]] = 0.0
    gap = torch.rand(T, generator=g, device="cuda") * temp
    z[torch.arange(T, device="cuda"), at[:, 1]] = -gap
    # the uniform number nearest to where the first token ends, as that looks without the tail
    w = torch.exp(-gap.double() / temp)
    u = (1 / (1 + w)).float()
    u[::4] = 1 - 2.0 ** -24  # and in the tail
    return z, u


def off(z, temp, u, p, tokens, logprobs):
    """Of each row, in units of the bound: how far the point lies out of the token's stretch, and the logprob's error."""
    worst = 0.0, 0.0
    for i in range(z.shape[0]):
        v = z[i].double()
        rank = torch.argsort(v, descending=True, stable=True)
        w = torch.exp((v[rank] - v[rank[0]]) / temp)
        upto = w.cumsum(0)
        if p < 1:
            keep = int((upto - w < p * upto[-1]).sum())
            upto, w = upto[:keep], w[:keep]
        bound = 2.0 ** -34 * float(upto[-1]) + 2.0 ** -44 * z.shape[1]
        at = int((rank == int(tokens[i])).nonzero())
        assert at < len(w), "a token that is not kept"
        point = float(u[i]) * float(upto[-1])
        out = max(float(upto[at] - w[at]) - point, point - float(upto[at]), 0.0)
        lp = float(torch.log(w[at] / upto[-1]))
        room = 2.0 ** -24 * abs(lp) + 2.0 ** -32 + bound / float(upto[-1])
        worst = max(worst[0], out / bound), max(worst[1], abs(float(logprobs[i]) - lp) / room)
    return worst


@pytest.mark.parametrize("V", [131072, 1 << 20])
@pytest.mark.parametrize("depth", [20.0, 29.0, 30.3, 30.5, 31.0])
@pytest.mark.parametrize("temp", [1.0, 0.25])
def test_long_tails(V, depth, temp):
    T = 24
    z, u = rows(T, V, depth, temp, V + int(10 * depth))
    tokens = torch.empty(T, dtype=torch.int32, device="cuda")
    logprobs = torch.empty(T, device="cuda")
    t = torch.full((T,), temp, device="cuda")
    pec.sample(z, tokens, u, temperature=t, logprobs=logprobs)
    out, err = off(z, temp, u, 1.0, tokens, logprobs)
    assert out <= 3 and err <= 1, (out, err)


def test_a_nucleus_of_all_but_the_tail():
    T, V = 8, 1 << 20
    z, u = rows(T, V, 20.0, 1.0, 5)  # the tail has 0.2% of the mass
    tokens = torch.empty(T, dtype=torch.int32, device="cuda")
    logprobs = torch.empty(T, device="cuda")
    pec.sample(z, tokens, u, top_p=torch.full((T,), 0.99, device="cuda"), logprobs=logprobs)
    out, err = off(z, 1.0, u, float(torch.tensor(0.99)), tokens, logprobs)
    assert out <= 3 and err <= 1, (out, err)
