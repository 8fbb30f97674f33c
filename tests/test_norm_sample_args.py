"""Refusals of moe_residual_norm and moe_sample on the host (no GPU needed): a
message and MOE_ERR_INVALID, before anything is launched."""
import ctypes

import pytest

import paged_expert_cache_gb300 as pec

torch = pytest.importorskip("torch")

B, F = torch.bfloat16, torch.float32


def norm_args(**change):
    a = dict(rows=2, hidden=64, x_type=1, y_type=0, w_type=0, gate_wide=0, scale=1.0, eps=1e-6, x=64, x_stride=64, y=64,
             y_stride=64, x_out=64, x_out_stride=64, out=64, out_stride=64, weight=64, post_weight=64, gate=64, gate_stride=1)
    a.update(change)
    n = pec.NormArgs()
    for name, v in a.items():
        setattr(n, name, v)
    return n


@pytest.mark.parametrize("change,what", [
    (dict(rows=-1), "rows"), (dict(hidden=0), "hidden"), (dict(hidden=32769), "hidden"), (dict(x_type=2), "types"),
    (dict(y_type=-1), "types"), (dict(w_type=3), "types"), (dict(scale=float("nan")), "scale"), (dict(scale=float("inf")), "scale"),
    (dict(eps=-1e-6), "eps"), (dict(eps=float("inf")), "eps"), (dict(gate_wide=2), "gate_wide"), (dict(x=None), "NULL x"),
    (dict(y=None), "need y"), (dict(y=None, x_out=None, gate=None), "need y"), (dict(out=None, x_out=None), "neither"),
    (dict(x=66), "aligned to its type"), (dict(out=65), "aligned to its type"), (dict(gate=65), "aligned to its type"),
    (dict(x_stride=63), "apart"), (dict(x_out_stride=0), "apart"), (dict(out_stride=-64), "apart"),
    (dict(gate_wide=1, gate_stride=8), "apart"), (dict(gate_stride=-1), "gate_stride"),
])
def test_norm_entry_refuses_bad_arguments(change, what):
    lib = pec.load()
    assert lib.moe_residual_norm(ctypes.addressof(norm_args(**change)), None) == pec.ERR_INVALID
    assert what in lib.moe_last_error(None).decode()


def test_norm_entry_takes_no_rows_and_refuses_null():
    lib = pec.load()
    assert lib.moe_residual_norm(ctypes.addressof(norm_args(rows=0, x=None, y=None, out=None)), None) == pec.OK
    assert lib.moe_residual_norm(None, None) == pec.ERR_INVALID


def test_norm_wrapper_refuses_mismatched_tensors():
    x, w = torch.zeros(3, 64), torch.ones(64)
    for args, kw in (((x[0],), {}), ((x.double(),), {}), (([1.0],), {}), ((x,), dict(out=x))):
        with pytest.raises(pec.MoeError) as e:
            pec.residual_norm(*args, **kw)
        assert e.value.status == pec.ERR_INVALID
    with pytest.raises(pec.MoeError) as e:
        pec.residual_norm(x, x, weight=w)
    assert "CUDA device" in str(e.value)


@pytest.mark.parametrize("change,what", [
    (dict(rows=-1), "rows"), (dict(rows=(1 << 24) + 1), "rows"), (dict(vocab=0), "vocab"), (dict(vocab=(1 << 20) + 1), "vocab"),
    (dict(type=2), "type"), (dict(settings=None), "settings"), (dict(logits=None), "NULL"), (dict(tokens=None), "NULL"),
    (dict(stride=99), "apart"), (dict(logits=65), "aligned"), (dict(tokens=66), "aligned"), (dict(logprobs=66), "aligned"),
])
def test_sample_entry_refuses_bad_arguments(change, what):
    lib = pec.load()
    s = pec.SamplingArgs(64, 64, 64, 64, 64)
    a = dict(logits=64, type=0, stride=100, rows=2, vocab=100, settings=ctypes.addressof(s), tokens=64, logprobs=64)
    a.update(change)
    st = lib.moe_sample(a["logits"], a["type"], a["stride"], a["rows"], a["vocab"], a["settings"], a["tokens"], a["logprobs"], None)
    assert st == pec.ERR_INVALID
    assert what in lib.moe_last_error(None).decode()


@pytest.mark.parametrize("name", ["temperature", "top_k", "top_p", "min_p", "uniform"])
def test_sample_entry_refuses_misaligned_settings(name):
    lib = pec.load()
    s = pec.SamplingArgs()
    setattr(s, name, 66)
    assert lib.moe_sample(64, 0, 100, 2, 100, ctypes.addressof(s), 64, None, None) == pec.ERR_INVALID


def test_sample_takes_no_rows():
    s = pec.SamplingArgs()
    assert pec.load().moe_sample(None, 0, 100, 0, 100, ctypes.addressof(s), None, None, None) == pec.OK


def test_sample_wrapper_refuses_mismatched_tensors():
    z, t = torch.zeros(3, 64), torch.zeros(3, dtype=torch.int32)
    for args in ((z[0], t), (z.double(), t), (z, t)):
        with pytest.raises(pec.MoeError) as e:
            pec.sample(*args)
        assert e.value.status == pec.ERR_INVALID


def test_packed_arguments_are_the_structures():
    assert len(pec._norm_args(*([0] * 6), 0.0, 0.0, *([0] * 12))) == ctypes.sizeof(pec.NormArgs)
    assert len(pec._sampling_args(*([0] * 5))) == ctypes.sizeof(pec.SamplingArgs)
    n = pec.NormArgs.from_buffer_copy(pec._norm_args(1, 2, 3, 4, 5, 6, 0.5, 0.25, *range(11, 23)))
    assert [getattr(n, f) for f, _ in pec.NormArgs._fields_] == [1, 2, 3, 4, 5, 6, 0.5, 0.25, *range(11, 23)]
