"""Refusals of the attention entry points on the host (no GPU needed): bad
configurations and mismatched tensors raise MoeError(ERR_INVALID) with a
message, before anything is launched."""
import ctypes

import pytest

import paged_expert_cache_gb300 as pec

torch = pytest.importorskip("torch")


@pytest.mark.parametrize("kw", [
    dict(L=0), dict(pages=0), dict(page_tokens=8), dict(page_tokens=24), dict(page_tokens=2048), dict(head_dim=96),
    dict(kv_heads=0), dict(q_heads=0), dict(q_heads=6, kv_heads=4), dict(q_heads=129, kv_heads=1),
])
def test_bad_cache_configurations_are_refused(kw):
    c = pec.make_kv_config(**{**dict(L=1, pages=4, q_heads=8, kv_heads=2, head_dim=128), **kw})
    with pytest.raises(pec.MoeError) as e:
        pec.KVCache(c)
    assert e.value.status == pec.ERR_INVALID and str(e.value)


def test_a_pool_whose_size_overflows_is_refused():
    # 2^31 - 1 layers of pages of 150 MB: the product does not fit 64 bits
    c = pec.make_kv_config(2 ** 31 - 1, 2 ** 31 - 1, 1024, 1024, 128, page_tokens=1024)
    with pytest.raises(pec.MoeError) as e:
        pec.KVCache(c)
    assert e.value.status in (pec.ERR_OOM, pec.ERR_CUDA)  # no device here, or no such memory


def test_config_defaults():
    c = pec.KvConfig()
    pec.load().moe_kv_config_default(ctypes.byref(c))
    assert c.page_tokens == 64 and c.num_layers == 1 and c.device == 0


def test_null_handles_are_refused():
    lib = pec.load()
    b = pec.KvBatchArgs()
    ref = ctypes.addressof(b)
    assert lib.moe_kv_append(None, 0, None, 0, None, 0, None, 0, 1, ref, None, 0, None, None, None) == pec.ERR_INVALID
    assert lib.moe_kv_attend(None, 0, None, 0, 1, ref, 1.0, None, None) == pec.ERR_INVALID
    assert lib.moe_kv_read(None, 0, 1, ref, None, None, None) == pec.ERR_INVALID
    assert lib.moe_kv_info(None, None) == pec.ERR_INVALID
    assert lib.moe_kv_status(None) == pec.ERR_INVALID
    assert lib.moe_kv_create(None, None) == pec.ERR_INVALID
    assert lib.moe_kv_destroy(None) == pec.OK
    assert b"NULL" in lib.moe_last_error(None)


@pytest.mark.parametrize("change,what", [
    (dict(Tq=-1), "Tq"), (dict(B=0), "num_seqs"), (dict(cu_q=None), "cu_q"), (dict(dim=80), "head_dim"),
    (dict(hq=3, hkv=2), "kv_heads"), (dict(hq=130, hkv=1), "kv_heads"), (dict(q=None), "NULL"), (dict(v=None), "NULL"),
    (dict(scale=-1.0), "scale"), (dict(scale=float("nan")), "scale"), (dict(scale=float("inf")), "scale"),
    (dict(q=8), "aligned"), (dict(qs=64), "aligned"), (dict(ks=260), "aligned"), (dict(out=24), "aligned"),
])
def test_prompt_entry_refuses_bad_arguments_before_any_launch(change, what):
    a = dict(q=16, qs=1024, k=16, ks=256, v=16, vs=256, Tq=4, Tk=4, B=1, cu_q=16, cu_k=16, hq=8, hkv=2, dim=128, out=16, scale=1.0)
    a.update(change)
    st = pec.load().moe_attn_prompt(a["q"], a["qs"], a["k"], a["ks"], a["v"], a["vs"], a["Tq"], a["Tk"], a["B"],
                                    a["cu_q"], a["cu_k"], a["hq"], a["hkv"], a["dim"], a["scale"], a["out"], None)
    assert st == pec.ERR_INVALID
    assert what in pec.load().moe_last_error(None).decode()


def test_prompt_wrapper_refuses_mismatched_tensors():
    q, k = torch.zeros(4, 8, 64).bfloat16(), torch.zeros(4, 2, 64).bfloat16()
    cu = torch.zeros(2, dtype=torch.int32)
    bad = [
        ((q[0], k, k, q, cu), "[T, heads, head_dim]"),
        ((q.float(), k, k, q, cu), "bfloat16"),
        ((q, k, k[:3], q, cu), "rows"),
        ((q, k[..., :32], k, q, cu), "v must be"),
        ((q, k.transpose(1, 2).contiguous().transpose(1, 2), k, q, cu), "contiguous"),
        ((q, k, k, q, cu), "CUDA device"),
    ]
    for args, what in bad:
        with pytest.raises(pec.MoeError) as e:
            pec.attention_prompt(*args)
        assert e.value.status == pec.ERR_INVALID
        if what != "v must be":
            assert what in str(e.value) or "CUDA device" in str(e.value), (what, str(e.value))


def test_dense_tensors_off_the_device_are_not_taken_for_usable_ones():
    x = torch.zeros(4, 2, 64).bfloat16()
    pec._need_torch()
    assert not pec._all_dense(torch.bfloat16, 0, (x, (4, 2, 64)), (x, (4, 2, 64)))
    assert pec._all_dense(torch.bfloat16, 0, (None, (4, 2, 64)))


def test_batch_refuses_wrong_arrays():
    cu, lens, table = (torch.zeros(3, dtype=torch.int32), torch.zeros(2, dtype=torch.int32),
                       torch.zeros(2, 4, dtype=torch.int32))
    for bad, what in (((cu.long(), lens, table), "CUDA device"), ((cu, lens.float(), table), "int32"),
                      ((cu, lens, table[:, ::2]), "CUDA device"), ((cu, lens, table), "CUDA device")):
        with pytest.raises(pec.MoeError) as e:
            pec.KVBatch(*bad)
        assert e.value.status == pec.ERR_INVALID and what in str(e.value)


def test_a_batch_of_another_device_is_refused():
    # made without tensors, as one whose arrays are on device 1
    batch = pec.KVBatch.__new__(pec.KVBatch)
    batch._ref, batch._device = 16, 1
    assert pec._batch(batch, 1) == 16
    with pytest.raises(pec.MoeError) as e:
        pec._batch(batch, 0)
    assert e.value.status == pec.ERR_INVALID and "batch is on CUDA device 1" in str(e.value)
