"""Refusals of the shared-prefix attention on the host (no GPU needed)."""
import ctypes

import pytest

import paged_expert_cache_gb300 as pec

torch = pytest.importorskip("torch")


def test_null_handles_are_refused():
    lib = pec.load()
    b, g, n = pec.KvBatchArgs(), pec.KvGroupArgs(), ctypes.c_uint64(0)
    ref = ctypes.addressof
    assert lib.moe_kv_attend_shared(None, 0, None, 0, 1, ref(b), ref(g), 1.0, None, None, 0, None) == pec.ERR_INVALID
    assert b"NULL" in lib.moe_last_error(None)
    assert lib.moe_kv_shared_bytes(None, 1, ctypes.byref(n)) == pec.ERR_INVALID


def test_groups_refuse_wrong_arrays():
    cu, prefix = torch.zeros(3, dtype=torch.int32), torch.zeros(2, dtype=torch.int32)
    for bad, what in (((cu, prefix.long()), "int32"), ((cu, prefix[:0]), "CUDA device"), ((cu[None], prefix), "CUDA device"),
                      (([0, 2], [64]), "int32"), ((cu, prefix), "CUDA device")):
        with pytest.raises(pec.MoeError) as e:
            pec.KVGroups(*bad)
        assert e.value.status == pec.ERR_INVALID and what in str(e.value)
