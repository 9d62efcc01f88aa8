"""Eviction's choice by one workgroup that reads the weights again on every pass: more tokens to
choose from than its registers hold, in batches too large for a choice in parts."""

import numpy as np
import pytest
import torch

from gated_delta_rule_kla_amd import kla
from oracle.kv4_oracle import evict
from test_gpu_kv4 import DEV, i32
from test_gpu_kv4_evict import check, hard, make

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a GPU")]

HELD = 32768  # tokens whose weights a workgroup keeps in registers
HKV, D, PAGE = 8, 64, 64


def lengths(recent):
    """Around what the registers hold beside `recent` tokens, far beyond it, and short ones."""
    return [37000, HELD + recent, HELD + recent + 1, 33001 + recent, 5, 3000]


def in_one_piece(N, budget, max_pages):
    """The workspace of a choice in parts has histograms behind the kept rows."""
    rows = N * HKV * budget * (D + 32)
    return kla.kv4_evict_workspace_bytes(N, HKV, D, budget, PAGE, max_pages) == -(-rows // 256) * 256


@pytest.mark.parametrize("f", [None, hard, torch.zeros_like, lambda w: (w * 2).round() / 2])
@pytest.mark.parametrize("budget,recent", [(1, 0), (4000, 700), (30000, 30000), (36999, 1)])
def test_weights_read_on_every_pass(f, budget, recent):
    lens = lengths(recent)
    assert max(lens) - recent > HELD or recent == budget
    assert in_one_piece(len(lens), budget, -(-max(lens) // PAGE))
    check(lens, HKV, D, PAGE, budget, recent, f)


def test_weights_read_on_every_pass_of_odd_rows():
    """Rows of weights that do not begin at 16 bytes: read one by one."""
    lens, budget, recent = lengths(20), 5000, 20
    codes, scales, table, w = make(lens, HKV, D, PAGE)
    assert in_one_piece(len(lens), budget, table.shape[1])
    odd = torch.zeros(len(lens), HKV, w.shape[2] + 3, device=DEV)
    odd[..., :w.shape[2]] = hard(w)
    before = odd.clone()
    kept = kla.kv4_evict(codes, scales, table, i32(lens), odd, budget, recent)[1].cpu().numpy()
    for n, L in enumerate(lens):
        for h in range(HKV):
            keep = evict(before[n, h, :L].cpu().double().numpy(), L, budget, recent)
            np.testing.assert_array_equal(kept[n, h, :len(keep)], keep)
            assert (kept[n, h, len(keep):] == -1).all()
