"""Grouped decode where the workspace's counters do not suffice for merging many ranges in two
steps (many requests cut into many ranges each): one step merges them all."""
import random

import pytest
import torch

import scored_ref as R
from paged_kv_cache_214_gb300 import pkv
from test_grouped_decode import Group, prompt

COUNTERS = (1 << 20) // 4   # of a workspace: one a request, two a range for the first step


@pytest.mark.gpu
@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("requests,width,Hq,Hkv,splits", [(300, 1, 1, 1, 500), (100, 2, 4, 2, 700)])
def test_many_ranges_without_counters_for_groups(requests, width, Hq, Hkv, splits, fp8):
    assert Hkv * (requests + 2 * requests * splits) > COUNTERS
    r = random.Random(requests)
    lens = [r.choice([0, 1, 64, 90]) for _ in range(requests * width)]
    for b in (0, 3, requests - 1):   # 17 and more ranges of one tile each
        lens[b * width:(b + 1) * width] = [1100 + 700 * (b > 0) + w for w in range(width)]
    g = Group(lens, width, Hq, Hkv, 5 + requests, prompt(2), fp8)
    want = g.want()
    need = pkv.paged_decode_grouped_workspace_bytes(len(lens), width, Hq, Hkv, 128, g.tables.shape[1],
                                                    fp8=fp8, num_splits=splits)
    ws = torch.zeros(need, dtype=torch.uint8, device="cuda")
    for _ in range(2):
        out, lse = g.run(num_splits=splits, workspace=ws)
        R.check(out, lse, want, "one step")
    assert not ws[:1 << 20].any()
    assert pkv.get_device_error() == pkv.PKV_OK
