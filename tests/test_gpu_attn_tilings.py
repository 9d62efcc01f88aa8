"""Attention over prompts: what is hard for a kernel, on every tiling that it has.

The tiling goes by the workgroups W that tiles of 128 queries make: 32 queries and four key groups
(W <= 64), 64 queries and two key groups (W <= 128; dense batches up to 256), 128 queries and two
key groups (dense, W <= 512), 256 queries (W > 512, long sequences), 128 queries (the rest).  Each
case below is of one of them, with heads sampled so that the oracle stays cheap.  Tolerances as in
test_gpu_attn.py."""

import numpy as np
import pytest
import torch

from gated_delta_rule_kla_amd import kla
from test_gpu_attn import BF, DEV, F32, check, f64, i32, inputs

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a GPU")]

# dtype, D, B, Hq, Hkv, Tq, and sampled queries (None: all)
DENSE = {
    "32 queries, four groups": (BF, 128, 1, 6, 3, 200, None),
    "64 queries, two groups": (BF, 128, 2, 30, 15, 180, None),
    "64 queries, two groups, D 64": (BF, 64, 1, 70, 35, 150, None),
    "128 queries, two groups": (BF, 128, 1, 150, 75, 250, None),
    "128 queries, two groups, D 64": (BF, 64, 3, 60, 30, 190, None),
    "256 queries": (BF, 128, 1, 64, 32, 2049, [0, 1, 31, 32, 255, 256, 700, 1023, 1024, 1500, 1999, 2047, 2048]),
    "256 queries, D 64": (BF, 64, 2, 32, 16, 2100, [0, 33, 255, 256, 900, 1001, 1900, 2099]),
    "128 queries": (BF, 128, 1, 300, 150, 130, None),
    "128 queries, D 64": (BF, 64, 1, 520, 260, 100, None),
    "fp32": (F32, 128, 1, 20, 10, 200, None),
    "fp32, D 64": (F32, 64, 1, 20, 10, 333, None),
}


def dense(name, more_keys=0, seed=0):
    dtype, D, B, Hq, Hkv, Tq, rows = DENSE[name]
    q, k, v = inputs(dtype, B, Hq, Hkv, Tq, Tq + more_keys, D, seed)
    return dtype, D, [0, Hq // 2 + 1, Hq - 1], rows, q, k, v


@pytest.mark.parametrize("more_keys", [1, 77, -1, -70])
@pytest.mark.parametrize("name", DENSE)
def test_other_numbers_of_keys(name, more_keys):
    """Continued prompts, and queries that see no key."""
    dtype, D, heads, rows, q, k, v = dense(name, more_keys, 1)
    o, lse = kla.attn_fwd(q, k, v)
    if rows is not None and more_keys < 0:
        rows = sorted({*rows, *range(-more_keys), -more_keys})
    check(o, lse, q, k, v, D ** -0.5, dtype, heads=heads, rows=rows)


def test_many_keys_of_few_queries():
    """128 queries and two key groups, where the keys are at least twice the queries."""
    q, k, v = inputs(BF, 1, 160, 20, 90, 1000, 128, 2)
    o, lse = kla.attn_fwd(q, k, v)
    check(o, lse, q, k, v, 128 ** -0.5, BF, heads=[0, 81, 159])


@pytest.mark.parametrize("scale", [4.0, -0.3, 0.0, 1e-3])
@pytest.mark.parametrize("name", DENSE)
def test_scales(name, scale):
    dtype, D, heads, rows, q, k, v = dense(name, 3, 3)
    o, lse = kla.attn_fwd(q, k, v, scale)
    check(o, lse, q, k, v, scale, dtype, heads=heads, rows=rows)


@pytest.mark.parametrize("scale", [0.125, -0.125])
@pytest.mark.parametrize("name", DENSE)
def test_growing_scores(name, scale):
    """The running maximum moves in every tile, or never."""
    dtype, D, heads, rows, q, k, v = dense(name, 0, 4)
    q.fill_(1.0)
    k.copy_((torch.arange(k.shape[2], device=DEV)[None, None, :, None] * (12.0 / k.shape[2])).expand_as(k))
    o, lse = kla.attn_fwd(q, k, v, scale)
    check(o, lse, q, k, v, scale, dtype, heads=heads, rows=rows)


@pytest.mark.parametrize("at", [0.45, 0.999])
@pytest.mark.parametrize("which,bad", [("k", float("nan")), ("k", float("inf")), ("v", float("nan")),
                                       ("v", -float("inf"))])
@pytest.mark.parametrize("name", DENSE)
def test_keys_and_values_that_are_not_finite(name, which, bad, at):
    """One bad channel of one key or value: other heads keep every bit, earlier queries are right
    (the bad key shares their tiles), later ones are not finite where they have to be."""
    dtype, D, heads, rows, q, k, v = dense(name, 5, 5)
    B, Hq, Tq, _ = q.shape
    G, t = Hq // k.shape[1], int(at * k.shape[2])
    first = max(0, t - 5)  # the first query that sees key t
    clean = kla.attn_fwd(q, k, v)
    x = {"q": q, "k": k.clone(), "v": v.clone()}
    head = heads[1]
    x[which][B - 1, head // G, t, 5] = bad
    o, lse = kla.attn_fwd(x["q"], x["k"], x["v"])
    same = torch.ones(B, Hq, dtype=torch.bool, device=DEV)
    same[B - 1, head // G * G:head // G * G + G] = False
    assert torch.equal(o[same], clean[0][same]) and torch.equal(lse[same], clean[1][same])
    late = o[B - 1, head, first:]
    assert late.shape[0] > 0
    if which == "v":
        assert not torch.isfinite(late[:, 5]).any()
        o[B - 1, :, first:, 5] = clean[0][B - 1, :, first:, 5]
        check(o, lse, q, k, v, D ** -0.5, dtype, heads=[head], rows=rows)
    else:
        # a score of minus infinity has no weight, any other one that is not finite makes NaN
        none = q[B - 1, head, first:, 5] < 0 if bad == float("inf") else torch.zeros(Tq - first, dtype=torch.bool, device=DEV)
        assert late[~none].isnan().all()
        sane = o.clone(), lse.clone()
        for i in (0, 1):
            sane[i][B - 1, :, first:] = clean[i][B - 1, :, first:]
        check(*sane, q, k, v, D ** -0.5, dtype, heads=[head], rows=rows)
        if none.any():
            # those queries, as if the key were not there
            keep = [i for i in range(k.shape[2]) if i != t]
            pick = (none.nonzero()[:4, 0] + first).tolist()
            for i in pick:
                n = i + 6  # the keys that query i sees
                cut = [j for j in keep if j < n]
                one = kla.attn_fwd(*(z.contiguous() for z in (q[B - 1:, head:head + 1, i:i + 1],
                                                              k[B - 1:, head // G:head // G + 1, cut],
                                                              v[B - 1:, head // G:head // G + 1, cut])))[0]
                got, want = f64(o[B - 1, head, i]), f64(one[0, 0, 0])
                # each is an average of values up to `top`: twice a score's error of (D + 2) 2^-24 of
                # its products' magnitudes (below 16 here: 2^-12 in all), in bf16 the weights' and the
                # output's rounding besides (2^-8 each)
                top = np.abs(f64(v[B - 1, head // G, :n])).max()
                assert (np.abs(got - want) <= 2 * (2.0 ** -12 + (2 * 2.0 ** -8 if dtype == BF else 0)) * top).all()


@pytest.mark.parametrize("scale", [0.0, 0.125])
@pytest.mark.parametrize("name", DENSE)
def test_queries_that_are_not_finite(name, scale):
    dtype, D, heads, rows, q, k, v = dense(name, 0, 6)
    head, Tq = heads[1], q.shape[2]
    clean = kla.attn_fwd(q, k, v, scale)
    x = q.clone()
    x[0, head, Tq // 2, 3], x[0, head, Tq - 1, 9] = float("nan"), -float("inf")
    o, lse = kla.attn_fwd(x, k, v, scale)
    for t in (Tq // 2, Tq - 1):
        assert o[0, head, t].isnan().all() and lse[0, head, t].isnan()
        o[0, head, t], lse[0, head, t] = clean[0][0, head, t], clean[1][0, head, t]
    assert torch.equal(o, clean[0]) and torch.equal(lse, clean[1])


# Packed: B = 1, Hq, Hkv, offsets of the queries and of the keys
PACKED = {
    "32 queries, four groups": (BF, 128, 6, 2, [0, 0, 40, 50, 120, 120, 250], [0, 3, 300, 300, 310, 340, 470]),
    "64 queries, two groups": (BF, 128, 14, 2, [0, 0, 40, 50, 120, 120, 250], [0, 3, 300, 300, 310, 340, 470]),
    "64 queries, two groups, D 64": (BF, 64, 15, 5, [0, 300, 301, 301, 500], [0, 290, 290, 350, 800]),
    "128 queries": (BF, 128, 40, 8, [0, 0, 40, 50, 120, 120, 250], [0, 3, 300, 300, 310, 340, 470]),
    "128 queries, D 64": (BF, 64, 60, 4, [0, 300, 301, 301, 500], [0, 290, 290, 350, 800]),
    "256 queries": (BF, 128, 64, 4, [0, 2300, 4200], [0, 2400, 4100]),
    "256 queries, D 64": (BF, 64, 64, 8, [0, 1, 6200, 6203], [0, 0, 6100, 6400]),
    "fp32": (F32, 128, 8, 2, [0, 0, 40, 50, 120, 120, 250], [0, 3, 300, 300, 310, 340, 470]),
}


@pytest.mark.parametrize("name", PACKED)
@pytest.mark.parametrize("scale", [0.11, -0.11])
def test_packed(name, scale):
    """Continued prompts, sequences without keys or queries, fewer keys than queries."""
    dtype, D, Hq, Hkv, cu, ck = PACKED[name]
    q, k, v = inputs(dtype, 1, Hq, Hkv, cu[-1], ck[-1], D, 7)
    o, lse = kla.attn_fwd(q, k, v, scale, i32(cu), torch.tensor(cu, dtype=torch.int32), i32(ck),
                          torch.tensor(ck, dtype=torch.int32))
    if cu[-1] < 1000:
        check(o, lse, q, k, v, scale, dtype, cu, ck, heads=[0, Hq // 2, Hq - 1])
        return
    # long sequences one by one, at sampled queries
    for a, z, ka, kz in zip(cu, cu[1:], ck, ck[1:]):
        rows = [i for i in (0, 1, 99, 100, 101, 255, 256, 1200, z - a - 1) if i < z - a]
        part = (t.contiguous() for t in (o[:, :, a:z], lse[:, :, a:z], q[:, :, a:z], k[:, :, ka:kz], v[:, :, ka:kz]))
        check(*part, scale, dtype, heads=[0, Hq // 2, Hq - 1], rows=rows)


@pytest.mark.parametrize("name", PACKED)
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_packed_values_that_are_not_finite(name, bad):
    """The last value of a sequence: its last query alone sees it, and no other sequence."""
    dtype, D, Hq, Hkv, cu, ck = PACKED[name]
    q, k, v = inputs(dtype, 1, Hq, Hkv, cu[-1], ck[-1], D, 8)
    args = 0.11, i32(cu), torch.tensor(cu, dtype=torch.int32), i32(ck), torch.tensor(ck, dtype=torch.int32)
    clean = kla.attn_fwd(q, k, v, *args)
    for n in range(len(cu) - 1):
        if cu[n] == cu[n + 1] or ck[n] == ck[n + 1]:
            continue
        x = v.clone()
        x[0, 0, ck[n + 1] - 1] = bad
        o, lse = kla.attn_fwd(q, k, x, *args)
        last, G = cu[n + 1] - 1, Hq // Hkv
        assert not torch.isfinite(o[0, :G, last]).any()
        assert torch.isfinite(o).sum() == o.numel() - G * D and torch.equal(lse[:, G:], clean[1][:, G:])
        o[0, :G, last] = clean[0][0, :G, last]
        assert torch.equal(o[:, G:], clean[0][:, G:])
        a, z = cu[n], cu[n + 1]
        rows = None if z - a < 1000 else list(range(z - a - 140, z - a, 7)) + [z - a - 2, z - a - 1]
        part = (t.contiguous() for t in (o[:, :, a:z], lse[:, :, a:z], q[:, :, a:z], k[:, :, ck[n]:ck[n + 1]],
                                         v[:, :, ck[n]:ck[n + 1]]))
        check(*part, 0.11, dtype, heads=[0, G - 1], rows=rows)
        # every other sequence keeps its bits
        o[:, :, a:z], lse[:, :, a:z] = clean[0][:, :, a:z], clean[1][:, :, a:z]
        assert torch.equal(o, clean[0]) and torch.equal(lse, clean[1])


@pytest.mark.parametrize("name", PACKED)
def test_other_lengths_on_the_device(name):
    """Results go by the device's offsets, as where a captured call is replayed with other lengths;
    queries behind the last sequence stay as they were."""
    dtype, D, Hq, Hkv, host, host_k = PACKED[name]
    Tq, Tk, N = host[-1], host_k[-1], len(host) - 1
    cu = [0] * (N - 1) + [Tq // 3, Tq - 37]
    ck = [0] * (N - 1) + [Tk // 2, Tk - 50]
    q, k, v = inputs(dtype, 1, Hq, Hkv, Tq, Tk, D, 9)
    o, lse = torch.full_like(q, 7.0), torch.full((1, Hq, Tq), 7.0, device=DEV)
    kla.attn_fwd(q, k, v, 0.11, i32(cu), torch.tensor(host, dtype=torch.int32), i32(ck),
                 torch.tensor(host_k, dtype=torch.int32), out=o, lse=lse)
    assert (o[:, :, cu[-1]:] == 7).all() and (lse[:, :, cu[-1]:] == 7).all()
    for a, z, ka, kz in zip(cu, cu[1:], ck, ck[1:]):
        if z > a:
            part = (t.contiguous() for t in (o[:, :, a:z], lse[:, :, a:z], q[:, :, a:z], k[:, :, ka:kz], v[:, :, ka:kz]))
            check(*part, 0.11, dtype, heads=[0, Hq - 1], rows=sorted({*range(0, z - a, 1 + (z - a) // 40), z - a - 1}))
