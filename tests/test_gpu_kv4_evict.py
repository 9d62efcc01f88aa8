"""Eviction from the 4-bit cache by accumulated weight, on the GPU: positions, codes, scales and
weights have to equal the oracle's."""

import numpy as np
import pytest
import torch

from gated_delta_rule_kla_amd import kla
from oracle.kv4_oracle import evict
from test_gpu_kv4 import DEV, i32, pages

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a GPU")]


def make(lens, Hkv, D, page, seed=0):
    gen = torch.Generator().manual_seed(seed)
    table, P = pages([max(n, 1) for n in lens], page, seed)
    codes = torch.randint(0, 256, (P, 2, Hkv, page, D // 2), generator=gen, dtype=torch.uint8).to(DEV)
    scales = torch.randint(0, 256, (P, 2, Hkv, page, D // 32), generator=gen, dtype=torch.uint8).to(DEV)
    w = torch.exp(2 * torch.randn(len(lens), Hkv, table.shape[1] * page, generator=gen)).to(DEV)
    return codes, scales, table, w


def rows(x, table, n, h, page):
    """A head's rows of sequence n, in the table's order: [positions, 2, ...]."""
    t = table[n].cpu()
    t = t[t >= 0].long().to(x.device)
    return x[t, :, h].permute(0, 2, 1, 3).flatten(0, 1)


def check(lens, Hkv, D, page, budget, recent, w=None, seed=0, workspace=None):
    codes, scales, table, weights = make(lens, Hkv, D, page, seed)
    if w is not None:
        weights = w(weights)
    c0, s0, w0 = codes.clone(), scales.clone(), weights.clone()
    new, kept = kla.kv4_evict(codes, scales, table, i32(lens), weights, budget, recent, workspace)
    assert new.tolist() == [min(n, budget) for n in lens]
    expect_c, expect_s, expect_w = c0.clone(), s0.clone(), w0.clone()
    for n, L in enumerate(lens):
        t = table[n].cpu().tolist()
        for h in range(Hkv):
            keep = evict(w0[n, h, :L].cpu().double().numpy(), L, budget, recent)
            want = np.full(budget, -1)
            want[:len(keep)] = keep
            np.testing.assert_array_equal(kept[n, h].cpu().numpy(), want)
            if L <= budget:
                continue
            to = np.arange(budget)
            pf, pt = ([t[i // page] for i in x] for x in (keep, to))
            for a, b in ((expect_c, c0), (expect_s, s0)):
                a[pt, :, h, to % page] = b[pf, :, h, keep % page]
            expect_w[n, h, :budget] = w0[n, h, torch.from_numpy(keep).to(DEV)]
            expect_w[n, h, budget:L] = 0
    assert torch.equal(codes, expect_c) and torch.equal(scales, expect_s)
    assert torch.equal(weights.nan_to_num(-1.0), expect_w.nan_to_num(-1.0))


@pytest.mark.parametrize("D,page,Hkv", [(128, 64, 2), (64, 16, 3), (128, 48, 1)])
@pytest.mark.parametrize("budget,recent", [(1, 0), (1, 1), (63, 7), (64, 64), (65, 0), (300, 299), (257, 100)])
def test_budgets(D, page, Hkv, budget, recent):
    check([0, 1, 64, 65, 66, 300, 301, 1000, 2500], Hkv, D, page, budget, recent)


@pytest.mark.parametrize("budget", [1, 100, 999])
def test_equal_weights(budget):
    """All equal, few values, zeros of both signs: the earlier tokens stay."""
    for f in (torch.zeros_like, torch.ones_like, lambda w: (w * 2).round() / 2,
              lambda w: torch.where(w > 1, 0.0, -0.0)):
        check([1000, 1024, 1500], 2, 64, 32, budget, min(budget, 10), f)


def test_any_numbers():
    """Negative, infinite, the smallest, NaN (the largest)."""
    def f(w):
        w = w - 3
        w[..., 3::17] = float("nan")
        w[..., 5::31] = float("inf")
        w[..., 6::31] = -float("inf")
        w[..., 7::29] = 1e-42
        return w

    for budget in (5, 200, 700):
        check([1000, 3000], 2, 64, 16, budget, 3, f)


def test_many_tokens():
    check([40000, 7, 25001], 2, 128, 64, 20000, 500)
    check([3000] * 150, 2, 64, 64, 1024, 64)


def test_again_after_more_tokens():
    """Cut, filled and cut again: the weights moved with their tokens."""
    codes, scales, table, w = make([500], 1, 64, 16)
    lens, kept = kla.kv4_evict(codes, scales, table, i32([500]), w, 100, 10)
    first = w.clone()
    lens += 60
    w[0, 0, 100:160] = 1e-3
    lens, kept = kla.kv4_evict(codes, scales, table, lens, w, 100, 60)
    assert lens.tolist() == [100]
    k = kept[0, 0].cpu().numpy()
    assert (k[40:] == np.arange(100, 160)).all()
    np.testing.assert_array_equal(k[:40], evict(first[0, 0, :160].cpu().double().numpy(), 160, 100, 60)[:40])


def test_missing_pages():
    """A token of a missing page moves as zero, one that would move to one is lost."""
    codes, scales, table, w = make([400], 1, 64, 16)
    table[0, 0], table[0, 5] = -1, 1 << 30
    w.fill_(0.0)
    w[0, 0, 80:100] = 1.0  # 80 .. 95 are of the missing page
    c0, s0, t = codes.clone(), scales.clone(), table.tolist()[0]
    kla.kv4_evict(codes, scales, table, i32([400]), w, 30, 10)
    c, s = rows(codes, table[:, 1:5], 0, 0, 16), rows(scales, table[:, 1:5], 0, 0, 16)
    old_c, old_s = rows(c0, table[:, 6:], 0, 0, 16), rows(s0, table[:, 6:], 0, 0, 16)
    assert torch.equal(c[0:4], old_c[0:4]) and torch.equal(s[0:4], old_s[0:4])       # 96 .. 99, at 16 .. 19
    assert torch.equal(c[4:14], old_c[294:304]) and torch.equal(s[4:14], old_s[294:304])  # 390 .. 399
    changed = (codes != c0).flatten(1).any(1)
    assert changed.sum() == 1 and changed[t[1]]
    w2 = make([400], 1, 64, 16)[3]
    table[0, 0], table[0, 5] = t[1], -1
    table[0, 1] = int(set(range(codes.shape[0])).difference(table[0].tolist()).pop())
    w2.fill_(0.0)
    w2[0, 0, 80:100] = 1.0
    kla.kv4_evict(codes, scales, table, i32([400]), w2, 30, 10)
    head = rows(codes, table[:, :1], 0, 0, 16)
    assert not head.any() and (rows(scales, table[:, :1], 0, 0, 16) == 1).all()


@pytest.mark.parametrize("N", [1, 40])
def test_captured_and_replayed(N):
    codes, scales, table, w = make([900] * N, 2, 64, 64)
    lens = i32([900] * N)
    keep = [x.clone() for x in (codes, scales, w)]

    def call():
        return kla.kv4_evict(codes, scales, table, lens, w, 300, 20)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        call()
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        got = call()
    for i in range(3):
        out = []
        for run in (graph.replay, call):
            for x, s in zip((codes, scales, w), keep):
                x.copy_(s)
            w.mul_(torch.rand(w.shape, generator=torch.Generator(device=DEV).manual_seed(i), device=DEV))
            lens.fill_(900 - 250 * i)
            r = run()
            torch.cuda.synchronize()
            out.append([x.clone() for x in (codes, scales, w, *(got if r is None else r))])
        assert all(torch.equal(a, b) for a, b in zip(*out))


def hard(w):
    w = w - 3
    w[..., 3::17] = float("nan")
    w[..., 5::31] = float("inf")
    w[..., 6::31] = -float("inf")
    w[..., 7::29] = 1e-42
    return w


@pytest.mark.parametrize("f", [None, hard, torch.zeros_like, lambda w: (w * 2).round() / 2])
@pytest.mark.parametrize("budget,recent", [(1, 0), (3000, 3000), (5000, 700), (11999, 1)])
def test_choices_in_parts(f, budget, recent):
    """Few sequences of many tokens, in parts of 4,096; also ones that end in an earlier part."""
    check([20000, 300, 12000, 12288, 8193], 1, 64, 64, budget, recent, f)


def test_choices_of_large_batches_and_odd_rows():
    check([9000] * 40, 4, 64, 16, 2000, 5, hard)
    codes, scales, table, w = make([9001, 5000], 1, 64, 16)
    odd = torch.zeros(2, 1, w.shape[2] + 3, device=DEV)
    odd[..., :w.shape[2]] = w
    got = [kla.kv4_evict(codes.clone(), scales.clone(), table, i32([9001, 5000]), x, 1234, 56) for x in (w.clone(), odd)]
    assert torch.equal(got[0][1], got[1][1])
