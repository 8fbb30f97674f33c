"""Shared-prefix attention (moe_kv_attend_shared) with so many groups that looking
through them takes longer than a wait of the kernel has for anything else."""
import pytest

from test_gpu_shared import CASES, Shared, i32

import paged_expert_cache_gb300 as pec

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


def test_groups_behind_millions_of_empty_ones():
    groups, _, hq, hkv, dim, page = CASES[5]
    s = Shared(groups, hq, hkv, dim, page)
    new = [1] * len(s.kv)
    q, want = s.check(new)
    empty = 1 << 25  # half a second of them
    cu = torch.zeros(empty + len(s.first), dtype=torch.int32, device="cuda")
    cu[empty:] = i32(s.first)
    prefix = torch.zeros(empty + len(s.prefix), dtype=torch.int32, device="cuda")
    prefix[empty:] = i32(s.prefix)
    assert torch.equal(s.attend(q, new, groups=pec.KVGroups(cu, prefix)), want)
    assert torch.equal(s.attend(q, new), want)  # and the next call is as ever
