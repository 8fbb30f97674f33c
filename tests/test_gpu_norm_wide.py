"""Residual norms of many rows in the forms that take a row a CTA: wider than 4096
values, and with a gate for each value; against the formula in 64 bits."""
import pytest

import paged_expert_cache_gb300 as pec
from test_gpu_norm import B, F, check, make, reference

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("xt,yt,wt", [(B, F, F), (F, B, B)])
@pytest.mark.parametrize("post,gate", [(True, "token"), (False, "full")])
@pytest.mark.parametrize("H", [4104, 4999, 5120, 7168, 8191, 8192, 12288, 16385])
def test_many_wide_rows(xt, yt, wt, post, gate, H):
    T = 700
    a = make(T, H, xt, yt, wt, post, gate, seed=H)
    out, xo = torch.empty(T, H, dtype=B, device="cuda"), torch.empty_like(a["x"])
    pec.residual_norm(a["x"], a["y"], out, weight=a["weight"], post_weight=a["post"], gate=a["gate"], scale=0.5, x_out=xo)
    check(xo, out, reference(a["x"], a["y"], a["weight"], a["post"], a["gate"], 0.5, 1e-6), xt)


@pytest.mark.parametrize("H", [64, 257, 2048, 4001, 4096])
@pytest.mark.parametrize("rows_apart", [0, 1])
def test_many_rows_with_a_gate_for_each_value(H, rows_apart):
    T = 1500
    a = make(T, H, B, B, F, True, "full", seed=H)
    gate = a["gate"] if rows_apart else a["gate"][:1].expand(T, H)  # one row of gates for all
    out, xo = torch.empty(T, H, dtype=B, device="cuda"), torch.empty_like(a["x"])
    pec.residual_norm(a["x"], a["y"], out, weight=a["weight"], post_weight=a["post"], gate=gate, x_out=xo)
    check(xo, out, reference(a["x"], a["y"], a["weight"], a["post"], gate, 1.0, 1e-6), B)
