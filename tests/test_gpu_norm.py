"""Residual norms (moe_residual_norm) against the formula in 64 bits."""
import pytest

import paged_expert_cache_gb300 as pec

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

B, F = torch.bfloat16, torch.float32
HALF_BF16, HALF_F32 = torch.finfo(B).eps / 2, torch.finfo(F).eps / 2


def reference(x, y, weight, post, gate, scale, eps):
    """s, out and, for the bounds, the size of what s is the sum of and the factor from s to out, fp64."""
    x = x.double()
    size = x.abs()
    if y is not None:
        y = y.double()
        if post is not None:
            y = y / (y.square().mean(-1, keepdim=True) + eps).sqrt() * post.double()
        if gate is not None:
            y = y * gate.double()
        x = x + scale * y
        size = size + (scale * y).abs()
    factor = 1 / (x.square().mean(-1, keepdim=True) + eps).sqrt()
    if weight is not None:
        factor = factor * weight.double()
    return x, x * factor, size, factor.abs()


def check(got_x, got_out, ref, x_type):
    s, out, size, factor = ref
    # fp32 on the way: the sum of squares of up to 32 values a thread and ten levels of a tree is off by at most 42 half
    # steps (half of that for the root), the other factors by ten or so
    work = 40 * HALF_F32
    if got_x is not None:
        half = HALF_BF16 if x_type is B else HALF_F32
        err = (got_x.double() - s).abs()
        assert (err <= half * s.abs() + work * size + 1e-37).all(), float((err / size).max())
    if got_out is not None:
        err = (got_out.double() - out).abs()
        assert (err <= HALF_BF16 * out.abs() + 2 * work * size * factor + 1e-37).all(), float((err / (size * factor)).max())


def make(T, H, xt, yt, wt, post, gate, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def n(*s):
        return torch.randn(*s, generator=g, device="cuda")

    x = (3 * n(T, H) * (1 + 30 * (torch.rand(H, generator=g, device="cuda") < 0.01))).to(xt)
    gates = {None: None, "token": lambda: n(T, 1).to(wt), "channel": lambda: n(H).to(wt), "full": lambda: n(T, H).to(wt)}[gate]
    return dict(x=x, y=n(T, H).to(yt), weight=(1 + n(H) / 4).to(wt), post=n(H).to(wt) if post else None,
                gate=gates() if gates else None)


@pytest.mark.parametrize("xt", [B, F])
@pytest.mark.parametrize("yt", [B, F])
@pytest.mark.parametrize("wt", [B, F])
@pytest.mark.parametrize("post,gate", [(False, None), (True, "token"), (False, "channel"), (True, "full")])
@pytest.mark.parametrize("T,H", [(3, 512), (5, 77), (2, 4001)])
def test_types_and_gates(xt, yt, wt, post, gate, T, H):
    a = make(T, H, xt, yt, wt, post, gate, seed=H)
    out, xo = torch.empty(T, H, dtype=B, device="cuda"), torch.empty_like(a["x"])
    got = pec.residual_norm(a["x"], a["y"], out, weight=a["weight"], post_weight=a["post"], gate=a["gate"], scale=0.7, eps=1e-5,
                            x_out=xo)
    assert got is out
    check(xo, out, reference(a["x"], a["y"], a["weight"], a["post"], a["gate"], 0.7, 1e-5), xt)
    # in place, and without the next block's input
    x = a["x"].clone()
    assert pec.residual_norm(x, a["y"], post_weight=a["post"], gate=a["gate"], scale=0.7, eps=1e-5) is x
    assert torch.equal(x, xo)


@pytest.mark.parametrize("H", [1, 2, 7, 8, 31, 64, 255, 256, 257, 264, 1000, 1024, 2048, 4096, 8192, 8193, 8200, 16384, 16391, 32760, 32768])
@pytest.mark.parametrize("T", [1, 6])
def test_widths(T, H):
    a = make(T, H, F, B, B, True, "token", seed=H)
    out = torch.empty(T, H, dtype=B, device="cuda")
    x = a["x"].clone()
    pec.residual_norm(x, a["y"], out, weight=a["weight"], post_weight=a["post"], gate=a["gate"])
    check(x, out, reference(a["x"], a["y"], a["weight"], a["post"], a["gate"], 1.0, 1e-6), F)


@pytest.mark.parametrize("T,H", [(1, 2048), (70000, 64), (4099, 257), (2451, 2048)])
def test_a_norm_alone(T, H):
    a = make(T, H, B, B, F, False, None, seed=T)
    out = torch.empty(T, H, dtype=B, device="cuda")
    assert pec.residual_norm(a["x"], out=out, weight=a["weight"]) is out
    check(None, out, reference(a["x"], None, a["weight"], None, None, 1.0, 1e-6), B)
    pec.residual_norm(a["x"], out=out)  # weights of one
    check(None, out, reference(a["x"], None, None, None, None, 1.0, 1e-6), B)


@pytest.mark.parametrize("xt,yt,wt", [(B, F, F), (F, B, B), (B, B, F), (F, F, B)])
@pytest.mark.parametrize("post,gate", [(True, "channel"), (False, "token"), (True, None)])
@pytest.mark.parametrize("H,offset,pad", [(264, 0, 0), (512, 8, 8), (261, 0, 0), (1000, 1, 2), (2047, 3, 0), (4095, 0, 1), (4096, 1, 7),
                                          (4096, 0, 0)])
def test_many_rows(xt, yt, wt, post, gate, H, offset, pad):
    # CTAs that take several rows each, whole vectors or not, all tensors with their own offset
    T = 1500
    a = make(T, H, xt, yt, wt, post, gate, seed=H + offset)

    def inside(t, shift):
        w = torch.full((T, H + offset + pad), 77.0, dtype=t.dtype, device="cuda")
        at = offset if shift else 0
        w[:, at:at + H] = t
        return w, w[:, at:at + H]

    (xw, x), (yw, y) = inside(a["x"], True), inside(a["y"], False)
    (ow, out), (xow, xo) = inside(torch.zeros(T, H, dtype=B, device="cuda"), True), inside(torch.zeros_like(a["x"]), False)
    pec.residual_norm(x, y, out, weight=a["weight"], post_weight=a["post"], gate=a["gate"], scale=0.5, x_out=xo)
    ref = reference(a["x"], a["y"], a["weight"], a["post"], a["gate"], 0.5, 1e-6)
    check(xo, out, ref, xt)
    assert (ow[:, :offset] == 77).all() and (ow[:, offset + H:] == 77).all() and (xow[:, H:] == 77).all()
    pec.residual_norm(x, y, weight=a["weight"], post_weight=a["post"], gate=a["gate"], scale=0.5)  # in place, without out
    assert torch.equal(x, xo) and (xw[:, :offset] == 77).all() and (xw[:, offset + H:] == 77).all()
    pec.residual_norm(x, out=out, weight=a["weight"])
    check(None, out, reference(x, None, a["weight"], None, None, 1.0, 1e-6), xt)


@pytest.mark.parametrize("offset,pad", [(0, 0), (8, 16), (1, 3), (0, 1), (4, 4)])
def test_rows_of_wider_tensors(offset, pad):
    T, H = 9, 264
    a = make(T, H, B, F, B, True, "full", seed=5)
    wide = {}

    def view(name, t):
        w = torch.full((T, H + offset + pad), 77.0, dtype=t.dtype, device="cuda")
        w[:, offset:offset + H] = t
        wide[name] = w
        return w[:, offset:offset + H]

    x, y, gate = view("x", a["x"]), view("y", a["y"]), view("gate", a["gate"])
    out = view("out", torch.zeros(T, H, dtype=B, device="cuda"))
    pec.residual_norm(x, y, out, weight=a["weight"], post_weight=a["post"], gate=gate)
    check(x, out, reference(a["x"], a["y"], a["weight"], a["post"], a["gate"], 1.0, 1e-6), B)
    for name, w in wide.items():  # nothing beside the rows is written
        assert (w[:, :offset] == 77).all() and (w[:, offset + H:] == 77).all(), name


@pytest.mark.parametrize("size", [1e-38, 1e-30, 1e-20, 1e-3, 1e10, 1e18, 1e25, 1e38])
@pytest.mark.parametrize("eps", [0.0, 1e-6])
def test_values_whose_squares_leave_fp32(size, eps):
    g = torch.Generator(device="cuda").manual_seed(3)
    x = (torch.rand(4, 512, generator=g, device="cuda") + 0.5) * size
    y = x.flip(1).contiguous()
    w = torch.ones(512, device="cuda")
    out, xo = torch.empty(4, 512, dtype=B, device="cuda"), torch.empty_like(x)
    pec.residual_norm(x, y, out, weight=w, post_weight=w, scale=0.25 * size, eps=eps, x_out=xo)
    check(xo, out, reference(x, y, w, w, None, float(torch.tensor(0.25 * size)), eps), F)


def test_rows_of_zeros_infinities_and_nan_keep_to_themselves():
    H = 320
    a = make(5, H, F, F, F, False, None, seed=1)
    x = a["x"].clone()
    x[1], x[2, 7], x[3, 9] = 0, float("inf"), float("nan")
    out = torch.empty(5, H, dtype=B, device="cuda")
    pec.residual_norm(x, out=out, weight=a["weight"])
    assert (out[1] == 0).all()
    assert out[2, 7].isnan() and (out[2, :7] == 0).all() and (out[2, 8:] == 0).all()
    assert out[3].isnan().all()
    check(None, out[[0, 4]], reference(x[[0, 4]], None, a["weight"], None, None, 1.0, 1e-6), F)


def test_no_rows_and_another_stream_and_a_graph():
    H = 2048
    a = make(7, H, F, B, B, False, None, seed=2)
    empty = torch.empty(0, H, device="cuda")
    pec.residual_norm(empty, torch.empty(0, H, device="cuda"), torch.empty(0, H, dtype=B, device="cuda"))
    out, x = torch.empty(7, H, dtype=B, device="cuda"), a["x"].clone()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        pec.residual_norm(x, a["y"], out, weight=a["weight"])  # the stream that is current
    torch.cuda.synchronize()
    ref = reference(a["x"], a["y"], a["weight"], None, None, 1.0, 1e-6)
    check(x, out, ref, F)
    xo, o2 = torch.empty_like(x), torch.empty_like(out)
    torch.cuda.synchronize()
    pec.residual_norm(a["x"], a["y"], o2, weight=a["weight"], x_out=xo, stream=s)
    torch.cuda.synchronize()
    assert torch.equal(o2, out) and torch.equal(xo, x)
    graph = torch.cuda.CUDAGraph()
    xi = a["x"].clone()
    with torch.cuda.graph(graph):
        pec.residual_norm(xi, a["y"], o2, weight=a["weight"], x_out=xo)
        pec.residual_norm(xo, a["y"], o2, weight=a["weight"])  # the next block's, in place
    for _ in range(2):  # with other contents
        xi.copy_(torch.randn_like(xi))
        graph.replay()
        torch.cuda.synchronize()
        s1 = reference(xi, a["y"], None, None, None, 1.0, 1e-6)[0]
        check(xo, o2, reference(s1, a["y"], a["weight"], None, None, 1.0, 1e-6), F)


def test_refusals_with_tensors_on_the_device():
    x, y, w = torch.zeros(4, 64, device="cuda"), torch.zeros(4, 64, device="cuda"), torch.ones(64, device="cuda")
    out = torch.empty(4, 64, dtype=B, device="cuda")
    calls = [((x,), dict()), ((x,), dict(out=out.float())), ((x,), dict(out=out[:3])), ((x,), dict(out=out.t())),
             ((x,), dict(out=out, x_out=x)), ((x,), dict(out=out, gate=w)), ((x,), dict(out=out, post_weight=w)),
             ((x, y[:, :32]), dict(out=out)), ((x, y.half()), dict(out=out)), ((x, y.cpu()), dict(out=out)),
             ((x, y), dict(weight=w[:63], out=out)), ((x, y), dict(weight=w, post_weight=w.bfloat16(), out=out)),
             ((x, y), dict(gate=w[:, None])), ((x, y), dict(gate=torch.ones(3, 1, device="cuda"))),
             ((x, y), dict(x_out=torch.empty(4, 64, dtype=B, device="cuda"))), ((x, y), dict(x_out=torch.empty(4, 64))),
             ((x, y), dict(scale=1e39)), ((x, y), dict(scale=float("nan"))), ((x, y), dict(eps=-1.0)), ((x, y), dict(scale="2")),
             ((x[:, :1].expand(4, 64), y), dict()), ((x.t(), y.t()), dict()), ((torch.zeros(1, 40000, device="cuda"),), dict(out=torch.empty(1, 40000, dtype=B, device="cuda")))]
    for args, kw in calls:
        with pytest.raises(pec.MoeError) as e:
            pec.residual_norm(*args, **kw)
        assert e.value.status == pec.ERR_INVALID, (args, kw)


@pytest.mark.parametrize("H,odd", [(264, False), (512, False), (261, True), (520, True)])
def test_fewer_rows_than_ctas_fit(H, odd):
    # between two rows an SM and as many CTAs as run at once: every CTA has a row of its own, and no CTA one past the last
    for T in (310, 608, 1500):
        wide = torch.full((T, H + (1 if odd else 0)), 1.0, device="cuda")
        x, y = wide[:, :H], torch.randn(T, H, device="cuda").bfloat16()
        out = torch.empty(T, H, dtype=B, device="cuda")
        ref = reference(x, y, None, None, None, 1.0, 1e-6)
        pec.residual_norm(x, y, out)
        check(x, out, ref, F)


@pytest.mark.parametrize("xt,yt", [(B, F), (F, B)])
@pytest.mark.parametrize("H,offset,pad", [(257, 0, 0), (4001, 0, 0), (4089, 3, 1), (2048, 5, 6), (1001, 7, 8), (264, 1, 7)])
def test_rows_of_one_phase_and_what_lies_between_them(xt, yt, H, offset, pad):
    # tensors of one offset and distance, whose rows' edges lie in the same 16 bytes as NaN that are no one's
    T = 1203
    a = make(T, H, xt, yt, F, True, "token", seed=H)

    def inside(t, fill):
        w = torch.full((T, offset + H + pad), fill, dtype=t.dtype, device="cuda")
        w[:, offset:offset + H] = t
        return w, w[:, offset:offset + H]

    (xw, x), (_, y) = inside(a["x"], float("nan")), inside(a["y"], float("nan"))
    (ow, out), (xow, xo) = inside(torch.zeros(T, H, dtype=B, device="cuda"), 77.0), inside(torch.zeros_like(a["x"]), 77.0)
    args = dict(weight=a["weight"], post_weight=a["post"], gate=a["gate"], scale=0.5)
    pec.residual_norm(x, y, out, x_out=xo, **args)
    check(xo, out, reference(a["x"], a["y"], a["weight"], a["post"], a["gate"], 0.5, 1e-6), xt)
    for w in (ow, xow):
        assert (w[:, :offset] == 77).all() and (w[:, offset + H:] == 77).all()
    first = out.clone()
    pec.residual_norm(x, y, out, **args)  # in place
    assert torch.equal(x, xo) and torch.equal(out, first)
    assert xw[:, :offset].isnan().all() and xw[:, offset + H:].isnan().all()
