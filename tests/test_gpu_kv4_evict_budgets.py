"""Eviction with a budget that covers the block table's room, on the GPU: without a workspace, and
nothing changes."""

import pytest
import torch

from gated_delta_rule_kla_amd import kla
from test_gpu_kv4 import i32
from test_gpu_kv4_evict import check, make

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a GPU")]


@pytest.mark.parametrize("lens", [[0, 1, 64, 300], [20000, 3], [13000]])
@pytest.mark.parametrize("more", [0, 1, 5000])
def test_budgets_of_the_room_and_more(lens, more):
    """One piece and parts; lengths of the whole room, and longer than it."""
    budget = -(-max(lens) // 64) * 64 + more
    check(lens, 2, 64, 64, budget, min(budget, 10))
    codes, scales, table, w = make(lens, 2, 64, 64)
    room = table.shape[1] * 64
    keep = [x.clone() for x in (codes, scales, w)]
    assert kla.kv4_evict_workspace_bytes(len(lens), 2, 64, budget, 64, table.shape[1]) == 0
    empty = torch.empty(0, dtype=torch.uint8, device=codes.device)
    new, kept = kla.kv4_evict(codes, scales, table, i32([n + 2 ** 20 for n in lens]), w, budget, 5, empty)
    assert new.tolist() == [room] * len(lens)
    assert (kept[..., :room].cpu() == torch.arange(room, dtype=torch.int32)).all() and (kept[..., room:] == -1).all()
    assert all(torch.equal(a, b) for a, b in zip((codes, scales, w), keep))
