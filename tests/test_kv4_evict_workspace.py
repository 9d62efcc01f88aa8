"""Eviction's workspace where the budget covers the block table's room: no sequence can be cut,
so none is needed (on the host, before any HIP call)."""

import os

import pytest

from gated_delta_rule_kla_amd import kla

pytestmark = pytest.mark.skipif(not os.path.exists(kla.lib_path()), reason="libkla.so not built")


@pytest.mark.parametrize("N,Hkv,D,page,M", [(64, 4, 128, 64, 64), (1, 1, 64, 16, 1), (1, 2, 128, 64, 2048), (3, 8, 64, 48, 5)])
def test_none_where_the_budget_covers_the_room(N, Hkv, D, page, M):
    room = M * page
    for budget in (room, room + 1, 131072):
        assert kla.kv4_evict_workspace_bytes(N, Hkv, D, budget, page, M) == 0
    assert kla.kv4_evict_workspace_bytes(N, Hkv, D, room - 1, page, M) >= N * Hkv * (room - 1) * (D + 32)
