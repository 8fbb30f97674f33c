"""Sampling (moe_sample) at the ends of the temperatures' range: those between 0 and 2^-99
count as 2^-99, for the weights, the filters and the log-probabilities alike."""
import pytest

from test_gpu_sample import B, F, reference, run

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

LEAST = 2.0 ** -99


def check(z, t, k, p, m, u):
    tokens, logprobs = run(z, t, k, p, m, u)
    t = max(float(torch.tensor(t, dtype=F)), LEAST)
    p, m = float(torch.tensor(p)), float(torch.tensor(m))
    for i in range(z.shape[0]):
        token, lp = reference(z[i], t, k, p, m, float(u[i]))
        assert int(tokens[i]) == token, (i, int(tokens[i]), token)
        assert abs(float(logprobs[i]) - lp) <= 2 ** -24 * abs(lp) + 2 ** -32, (i, float(logprobs[i]), lp)


@pytest.mark.parametrize("dtype", [B, F])
@pytest.mark.parametrize("V", [300, 9000])
@pytest.mark.parametrize("t,spread", [(1e-32, 1e-31), (1e-38, 1e-30), (1e-42, 1e-30), (2e-30, 1e-30), (1e38, 1e30), (1e29, 1e29), (1e33, 1e33),
                                      (3e33, 3e33), (1e38, 3e33)])
@pytest.mark.parametrize("k,p,m", [(0, 1.0, 0.0), (40, 0.9, 0.0), (0, 0.9, 0.0), (0, 1.0, 0.3)])
def test_logits_as_far_apart_as_the_temperature(dtype, V, t, spread, k, p, m):
    T = 12
    g = torch.Generator(device="cuda").manual_seed(V)
    z = (torch.randn(T, V, generator=g, device="cuda") * 4).round().div(2).clamp(-3, 3).mul(spread).to(dtype)
    check(z, t, k, p, m, (torch.arange(T) + 0.3) / T)
