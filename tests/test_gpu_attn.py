"""Attention over whole prompts on the GPU against its fp64 oracle, within the oracle's bound
(oracle/attn_oracle.py) with the weights' bf16 rounding (2^-8) where there is one, plus half a
step of the output's type."""

import numpy as np
import pytest
import torch

from gated_delta_rule_kla_amd import kla
from oracle.attn_oracle import attend

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a GPU")]

DEV = torch.device("cuda:0")
HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}
BF, F32 = torch.bfloat16, torch.float32


def f64(t):
    return t.detach().cpu().to(torch.float64).numpy()


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def inputs(dtype, B, Hq, Hkv, Tq, Tk, D, seed=0):
    gen = torch.Generator().manual_seed(seed)
    return [torch.randn(B, h, t, D, generator=gen).to(dtype).to(DEV) for h, t in ((Hq, Tq), (Hkv, Tk), (Hkv, Tk))]


def check(o, lse, q, k, v, scale, dtype, cu_q=None, cu_k=None, heads=None, rows=None):
    q, k, v, o, lse = (f64(t) for t in (q, k, v, o, lse))
    B, Hq, Tq, D = q.shape
    G = Hq // k.shape[1]
    spans = [(b, 0, Tq, 0, k.shape[2]) for b in range(B)]
    if cu_q is not None:
        cu_k = cu_q if cu_k is None else cu_k
        spans = [(0, *x) for x in zip(cu_q, cu_q[1:], cu_k, cu_k[1:])]
    for b, a, z, ka, kz in spans:
        for h in range(Hq) if heads is None else heads:
            at = np.arange(a, z) if rows is None else a + np.asarray(rows)
            mask = np.arange(ka, kz)[None] - ka <= (at - a)[:, None] + (kz - ka) - (z - a)
            want, wl, bound, bl = attend(q[b, h, at], k[b, h // G, ka:kz], v[b, h // G, ka:kz], scale, mask,
                                         2.0 ** -8 if dtype == BF else 2.0 ** -23)
            off = np.abs(o[b, h, at] - want) - (bound + HALF[dtype] * (np.abs(want) + bound))
            assert np.isfinite(o[b, h, at]).all(), (b, a, h)
            assert (off <= 0).all(), (b, a, h, float(off.max()))
            none = ~mask.any(1)
            assert (lse[b, h, at][none] == -np.inf).all() and not o[b, h, at][none].any()
            some = ~none
            assert (np.abs(lse[b, h, at][some] - wl[some]) <= (bl + 2.0 ** -23 * np.abs(wl))[some]).all(), (b, a, h)


DTYPES = [BF, F32]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("B,Hq,Hkv,Tq,Tk", [
    (1, 1, 1, 1, 1), (2, 3, 3, 5, 5), (1, 4, 2, 31, 31), (1, 2, 1, 64, 64), (1, 5, 1, 65, 65), (3, 2, 2, 127, 127),
    (1, 8, 2, 200, 200), (1, 1, 1, 513, 513), (2, 2, 1, 1, 300), (1, 2, 2, 100, 133), (1, 2, 1, 33, 1000),
    (1, 2, 2, 300, 100), (1, 1, 1, 70, 1), (1, 2, 1, 5, 0)])
def test_dense(dtype, D, B, Hq, Hkv, Tq, Tk):
    q, k, v = inputs(dtype, B, Hq, Hkv, Tq, Tk, D, Tq + Tk)
    o, lse = kla.attn_fwd(q, k, v)
    check(o, lse, q, k, v, D ** -0.5, dtype)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("D,Hq,Hkv", [(128, 4, 1), (64, 3, 3)])
def test_packed(dtype, D, Hq, Hkv):
    cu = [0, 0, 1, 65, 65, 193, 450, 451, 700, 700]
    q, k, v = inputs(dtype, 1, Hq, Hkv, 700, 700, D, 1)
    o, lse = kla.attn_fwd(q, k, v, cu_seqlens=i32(cu))
    check(o, lse, q, k, v, D ** -0.5, dtype, cu)


@pytest.mark.parametrize("dtype", DTYPES)
def test_packed_with_other_keys(dtype):
    """Continued prompts, a sequence without keys, one with fewer keys than queries, one without
    queries."""
    cu, ck = [0, 40, 50, 120, 120, 250], [0, 300, 300, 310, 340, 470]
    q, k, v = inputs(dtype, 1, 4, 2, 250, 470, 128, 2)
    o, lse = kla.attn_fwd(q, k, v, 0.11, i32(cu), torch.tensor(cu, dtype=torch.int32), i32(ck),
                          torch.tensor(ck, dtype=torch.int32))
    check(o, lse, q, k, v, 0.11, dtype, cu, ck)


@pytest.mark.parametrize("dtype", DTYPES)
def test_many_short_sequences(dtype):
    cu = np.concatenate([[0], np.cumsum(np.random.default_rng(0).integers(0, 30, 300))]).tolist()
    q, k, v = inputs(dtype, 1, 2, 1, cu[-1], cu[-1], 64, 3)
    o, lse = kla.attn_fwd(q, k, v, cu_seqlens=i32(cu))
    check(o, lse, q, k, v, 0.125, dtype, cu)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("Hq,T", [(16, 4096), (40, 2000)])
def test_large(dtype, Hq, T):
    q, k, v = inputs(dtype, 1, Hq, Hq // 8, T, T, 128, 4)
    o, lse = kla.attn_fwd(q, k, v)
    check(o, lse, q, k, v, 128 ** -0.5, dtype, heads=[0, Hq // 2, Hq - 1], rows=[0, 1, 63, 64, 1000, T - 130, T - 1])


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("B,Hq,T,cu", [
    (1, 8, 1000, None), (1, 16, 900, None), (1, 16, 2000, None), (1, 16, 3000, None), (2, 32, 2100, None),
    (1, 8, 1000, [0, 1, 1, 34, 600, 1000]), (1, 4, 2500, [0, 1200, 1201, 2500]), (1, 16, 3000, [0, 700, 701, 3000])])
def test_tilings(D, B, Hq, T, cu):
    """32, 64, 64 and 128 queries with the keys in groups, 256 queries; packed: 64 queries with
    the keys in groups twice, 128 queries."""
    q, k, v = inputs(BF, B, Hq, 2, T, T, D, 10)
    o, lse = kla.attn_fwd(q, k, v, cu_seqlens=None if cu is None else i32(cu))
    rows = [0, 1, 127, 128, 255, 256, T - 1] if cu is None else None
    check(o, lse, q, k, v, D ** -0.5, BF, cu, heads=[1, Hq - 1], rows=rows)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("scale", [4.0, -0.3, 0.0, 1e-3])
def test_scales(dtype, scale):
    """Scores far apart, reversed, and all alike."""
    q, k, v = inputs(dtype, 1, 2, 2, 150, 150, 64, 5)
    o, lse = kla.attn_fwd(q, k, v, scale)
    check(o, lse, q, k, v, scale, dtype)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("scale", [0.0, 0.125])
def test_a_query_that_is_not_finite(dtype, scale):
    q, k, v = inputs(dtype, 1, 2, 1, 150, 150, 64, 8)
    q[0, 0, 70, 3], q[0, 1, 149, 9] = float("nan"), float("inf")
    o, lse = kla.attn_fwd(q, k, v, scale)
    q[0, 0, 70], q[0, 1, 149] = 0.0, 0.0
    for h, t in ((0, 70), (1, 149)):
        assert o[0, h, t].isnan().all() and lse[0, h, t].isnan()
        o[0, h, t], lse[0, h, t] = kla.attn_fwd(q, k, v, scale)[0][0, h, t], kla.attn_fwd(q, k, v, scale)[1][0, h, t]
    check(o, lse, q, k, v, scale, dtype)


@pytest.mark.parametrize("dtype", DTYPES)
def test_growing_scores(dtype):
    """Every later key beats the ones before, so the running maximum moves in every tile."""
    q, k, v = inputs(dtype, 1, 1, 1, 400, 400, 64, 6)
    q.fill_(1.0)
    k.copy_((torch.arange(400, device=DEV)[None, None, :, None] * 0.05).expand_as(k))
    for scale in (0.125, -0.125):
        o, lse = kla.attn_fwd(q, k, v, scale)
        check(o, lse, q, k, v, scale, dtype)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_what_is_not_seen_does_not_matter(dtype, bad):
    q, k, v = inputs(dtype, 1, 4, 2, 700, 700, 128, 7)
    cu = [0, 300, 700]
    clean = kla.attn_fwd(q, k, v, cu_seqlens=i32(cu))
    for t in (100, 299, 300, 350, 699):
        for which in (1, 2):
            x = [q, k.clone(), v.clone()]
            x[which][0, 1, t, 5] = bad
            o, lse = kla.attn_fwd(*x, cu_seqlens=i32(cu))
            end = 300 if t < 300 else 700
            assert torch.equal(o[0, :2], clean[0][0, :2])
            if which == 2:
                assert not torch.isfinite(o[0, 2:, t:end, 5]).any()
                o[0, 2:, t:end, 5] = clean[0][0, 2:, t:end, 5]
            else:
                o[0, 2:, t:end], lse[0, 2:, t:end] = clean[0][0, 2:, t:end], clean[1][0, 2:, t:end]
            check(o, lse, q, k, v, 128 ** -0.5, dtype, cu, heads=[2, 3])


def test_continued_equals_whole():
    q, k, v = inputs(BF, 1, 4, 2, 500, 500, 64, 8)
    whole, lse = kla.attn_fwd(q, k, v)
    part, lp = kla.attn_fwd(q[:, :, 320:].contiguous(), k, v)
    # tiles of queries begin elsewhere, tiles of keys do not: the same sums
    assert torch.equal(part, whole[:, :, 320:]) and torch.equal(lp, lse[:, :, 320:])


@pytest.mark.parametrize("dtype", DTYPES)
def test_repeats_streams_and_graphs(dtype):
    q, k, v = inputs(dtype, 1, 8, 2, 900, 900, 128, 9)
    o, lse = kla.attn_fwd(q, k, v)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        o2, lse2 = kla.attn_fwd(q, k, v)
    side.synchronize()
    assert torch.equal(o, o2) and torch.equal(lse, lse2)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o3, lse3 = kla.attn_fwd(q, k, v)
    for _ in range(3):
        q.mul_(-0.7)
        graph.replay()
        torch.cuda.synchronize()
        o4, lse4 = kla.attn_fwd(q, k, v)
        torch.cuda.synchronize()
        assert torch.equal(o3, o4) and torch.equal(lse3, lse4)


def test_refusals():
    q, k, v = inputs(BF, 1, 4, 2, 10, 10, 64)
    with pytest.raises(kla.KlaError):
        kla.attn_fwd(q[:, :3].contiguous(), k, v)
    with pytest.raises(ValueError):
        kla.attn_fwd(q, k, v[:, :, :9].contiguous())
    with pytest.raises(TypeError):
        kla.attn_fwd(q, k.float(), v)
    with pytest.raises(ValueError):
        kla.attn_fwd(q.transpose(1, 2).contiguous().transpose(1, 2), k, v)
    with pytest.raises(kla.KlaError):
        kla.attn_fwd(q[..., :32].contiguous(), k[..., :32].contiguous(), v[..., :32].contiguous())
    with pytest.raises(kla.KlaError):
        kla.attn_fwd(q, k, v, float("nan"))
    with pytest.raises(kla.KlaError):
        kla.attn_fwd(q, k, v, cu_seqlens=i32([0, 4, 9]))
    with pytest.raises(ValueError):
        kla.attn_fwd(q, k, v, cu_seqlens_k=i32([0, 10]))
