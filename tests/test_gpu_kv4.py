"""The 4-bit cache and the attention of single tokens over it, on the GPU, against fp64 oracles.

What is stored and read back has to equal the format's definition; attention is held to the
oracle's bound (oracle/attn_oracle.py) with the weights' bf16 rounding (2^-8, bf16 queries) or
three bf16 terms (2^-24, fp32), plus half a step of the output's type."""

import numpy as np
import pytest
import torch

from gated_delta_rule_kla_amd import kla
from oracle.attn_oracle import attend, quantise, values

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a GPU")]

DEV = torch.device("cuda:0")
HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}
BF, F32 = torch.bfloat16, torch.float32


def f64(t):
    return t.detach().cpu().to(torch.float64).numpy()


def pages(lens, page, seed=0, spare=2):
    """A block table of shuffled pages; unused entries are -1."""
    need = [-(-n // page) for n in lens]
    M, P = max(max(need), 1), sum(need) + spare
    order = np.random.default_rng(seed).permutation(P)
    table, at = np.full((len(lens), M), -1, np.int32), 0
    for n, k in enumerate(need):
        table[n, :k] = order[at:at + k]
        at += k
    return torch.tensor(table, device=DEV), P


def packed(lens):
    host = torch.tensor(np.concatenate([[0], np.cumsum(lens)]), dtype=torch.int32)
    return host.to(DEV), host


def make_kv(lens, Hkv, D, dtype, seed=0):
    gen = torch.Generator().manual_seed(seed)
    T = int(sum(lens))
    k = torch.randn(1, Hkv, T, D, generator=gen) * torch.exp(2 * torch.randn(1, Hkv, T, 1, generator=gen))
    v = torch.randn(1, Hkv, T, D, generator=gen)
    return k.to(dtype).to(DEV), v.to(dtype).to(DEV)


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("D,page,Hkv", [(128, 16, 1), (64, 48, 3), (128, 64, 4)])
def test_store_and_read(dtype, D, page, Hkv):
    start, lens = [0, 5, 17, 0, 100], [33, 1, 64, 0, 7]
    table, P = pages([a + b for a, b in zip(start, lens)], page)
    codes, scales = kla.kv4_cache(P, Hkv, page, D, DEV)
    codes.fill_(0xA5)
    scales.fill_(0x77)
    k, v = make_kv(lens, Hkv, D, dtype)
    cu, host = packed(lens)
    kla.kv4_append(k, v, codes, scales, table, i32(start), cu, host)
    got = kla.kv4_read(codes, scales, table, i32(start), cu, dtype, host)
    touched = torch.zeros(P, page, dtype=torch.bool)
    tb = table.cpu()
    for x, y, j in ((k, got[0], 0), (v, got[1], 1)):
        want_c, want_s = quantise(f64(x)[0])
        np.testing.assert_array_equal(f64(y)[0], values(want_c, want_s))
        for n in range(len(lens)):
            for i in range(lens[n]):
                pos, t = start[n] + i, int(host[n]) + i
                p, at = int(tb[n, pos // page]), pos % page
                touched[p, at] = True
                c = codes[p, j, :, at].cpu().numpy()
                np.testing.assert_array_equal(scales[p, j, :, at].cpu().numpy(), want_s[:, t])
                nib = np.stack([c & 15, c >> 4], -1).reshape(Hkv, D)
                np.testing.assert_array_equal(np.where(nib == 8, 0, nib), np.where(want_c[:, t] == 8, 0, want_c[:, t]))
    rest = ~touched
    assert (codes.cpu().permute(0, 3, 1, 2, 4)[rest] == 0xA5).all()
    assert (scales.cpu().permute(0, 3, 1, 2, 4)[rest] == 0x77).all()


@pytest.mark.parametrize("dtype,D,Hkv,T", [(BF, 128, 4, 50000), (BF, 128, 4, 132000), (BF, 64, 8, 51000),
                                           (F32, 128, 4, 26000), (F32, 64, 4, 50000)])
def test_many_tokens(dtype, D, Hkv, T):
    """Larger workgroups, and rows that go past the caches: the same as sequence by sequence,
    and the oracle's values at sampled tokens."""
    lens, page = [3, T // 3, 1, T - T // 3 - T // 8 - 11, T // 8 + 7], 64
    start = [0, 70, 5, 1, 64]
    table, P = pages([a + b for a, b in zip(start, lens)], page)
    whole, parts = kla.kv4_cache(P, Hkv, page, D, DEV), kla.kv4_cache(P, Hkv, page, D, DEV)
    k, v = make_kv(lens, Hkv, D, dtype)
    cu, host = packed(lens)
    kla.kv4_append(k, v, *whole, table, i32(start), cu, host)
    out = [torch.full((Hkv * T + 1, D), 7.0, dtype=dtype, device=DEV) for _ in range(2)]
    view = tuple(t[:-1].view(1, Hkv, T, D) for t in out)
    kla.kv4_read(*whole, table, i32(start), cu, dtype, host, out=view)
    for n, (a, z) in enumerate(zip(host[:-1].tolist(), host[1:].tolist())):
        for b in range(a, z, 4000):  # small calls
            e = min(b + 4000, z)
            at, c, h = i32([start[n] + b - a]), i32([0, e - b]), torch.tensor([0, e - b], dtype=torch.int32)
            kla.kv4_append(k[:, :, b:e].contiguous(), v[:, :, b:e].contiguous(), *parts, table[n:n + 1], at, c, h)
            one = kla.kv4_read(*parts, table[n:n + 1], at, c, dtype, h)
            assert torch.equal(one[0], view[0][:, :, b:e]) and torch.equal(one[1], view[1][:, :, b:e])
    assert torch.equal(whole[0], parts[0]) and torch.equal(whole[1], parts[1])
    some = torch.cat([host[1:].long() - 1, torch.arange(0, T, T // 50)])
    for x, y in ((k, view[0]), (v, view[1])):
        np.testing.assert_array_equal(f64(y[:, :, some.to(DEV)]), values(*quantise(f64(x[:, :, some.to(DEV)]))))
    assert (out[0][-1] == 7).all() and (out[1][-1] == 7).all()


def test_dense_batch_and_padding():
    """One new token for each of four sequences; the second is padding (negative start), the
    third has no page there, the fourth's page is outside the cache."""
    k, v = torch.randn(4, 2, 1, 64, device=DEV), torch.randn(4, 2, 1, 64, device=DEV)
    codes, scales = kla.kv4_cache(6, 2, 16, 64, DEV)
    table = i32([[1, 2], [3, 4], [5, -1], [0, 6]])
    kla.kv4_append(k, v, codes, scales, table, i32([17, -1, 16, 20]))
    touched = [int(i) for i in codes.flatten(1).any(1).nonzero()]
    assert touched == [2] and int(codes[2].any(-1).sum()) == 4  # one place, two heads, K and V
    cu, host = packed([1, 1, 1, 1])
    kk, vv = kla.kv4_read(codes, scales, table, i32([17, -1, 16, 20]), cu, F32, host)
    np.testing.assert_array_equal(f64(kk)[0, :, 0], values(*quantise(f64(k)[0, :, 0])))
    assert not kk[:, :, 1:].any() and not vv[:, :, 1:].any()
    far = i32([32, 2 ** 31 - 1, 0, 0])
    before = codes.clone()
    kla.kv4_append(k, v, codes, scales, i32([[1, 2], [3, 4], [-1, -1], [6, 7]]), far)
    assert torch.equal(before, codes)


def test_values_that_are_not_finite_or_tiny():
    x = torch.zeros(1, 1, 6, 64)
    x[0, 0, 0, 3], x[0, 0, 1, 40], x[0, 0, 2, 63] = float("nan"), float("inf"), -float("inf")
    x[0, 0, 3] = 2.0 ** -130
    x[0, 0, 4] = torch.finfo(F32).max
    x[0, 0, 5, :32] = 2.0 ** -126 * torch.arange(32)
    table, P = pages([6], 16)
    codes, scales = kla.kv4_cache(P, 1, 16, 64, DEV)
    cu, host = packed([6])
    for dtype in (F32, BF):
        k = x.to(dtype).to(DEV)
        kla.kv4_append(k, torch.zeros_like(k), codes, scales, table, i32([0]), cu, host)
        y = kla.kv4_read(codes, scales, table, i32([0]), cu, dtype, host)[0][0, 0].cpu()
        # NaN in the blocks that hold an infinity or a NaN and nowhere else; fp32's largest number
        # is one of them in bf16, whose largest lies 2^119 below it: it rounds to infinity
        odd = ~torch.isfinite(x.to(dtype)[0, 0]).unflatten(-1, (-1, 32)).all(-1)
        assert odd.sum() == (3 if dtype == F32 else 5)
        assert torch.equal(torch.isnan(y), odd.repeat_interleave(32, -1))
        assert not y[3].any()
        if dtype == F32:
            np.testing.assert_array_equal(f64(y[4:]), values(*quantise(f64(k)[0, 0, 4:])))


def fill(lens, Hkv, D, page, seed=0, dtype=BF):
    """A cache of random tokens, and its values per sequence in fp64."""
    table, P = pages(lens, page, seed)
    codes, scales = kla.kv4_cache(P, Hkv, page, D, DEV)
    scales.fill_(255)  # what no token has written is NaN
    k, v = make_kv(lens, Hkv, D, dtype, seed)
    cu, host = packed(lens)
    if host[-1]:
        kla.kv4_append(k, v, codes, scales, table, i32([0] * len(lens)), cu, host)
    kq, vq = (values(*quantise(f64(x)[0])) for x in (k, v))
    b = host.tolist()
    return codes, scales, table, [(kq[:, a:z], vq[:, a:z]) for a, z in zip(b, b[1:])]


def check(o, q, kv, scale, dtype, what=""):
    q, o = f64(q), f64(o)
    N, Hq, D = q.shape
    for n in range(N):
        k, v = kv[n]
        G = Hq // k.shape[0]
        for h in range(k.shape[0]):
            rows = slice(h * G, (h + 1) * G)
            want, _, bound, _ = attend(q[n, rows], k[h], v[h], scale, np.ones((G, k.shape[1]), bool),
                                       2.0 ** -8 if dtype == BF else 2.0 ** -23)
            off = np.abs(o[n, rows] - want) - (bound + HALF[dtype] * (np.abs(want) + bound))
            assert np.isfinite(o[n, rows]).all(), (what, n, h)
            assert (off <= 0).all(), (what, n, h, float(off.max()))


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("Hq,Hkv,D,page", [(1, 1, 128, 16), (4, 4, 64, 64), (16, 2, 128, 64), (5, 1, 64, 48),
                                           (20, 1, 128, 32), (33, 1, 64, 16)])
def test_decode(dtype, Hq, Hkv, D, page):
    lens = [1, 0, 15, 16, 17, 31, 33, 64, 127, 129, 300]
    codes, scales, table, kv = fill(lens, Hkv, D, page)
    q = torch.randn(len(lens), Hq, D, device=DEV).to(dtype)
    o = kla.attn_kv4_decode_step(q, codes, scales, table, i32(lens))
    check(o, q, kv, D ** -0.5, dtype)
    assert not o[1].any()


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("lens", [[5000], [9000, 700, 0, 4100]])
def test_decode_in_several_runs(dtype, lens):
    codes, scales, table, kv = fill(lens, 2, 128, 64)
    q = torch.randn(len(lens), 8, 128, device=DEV).to(dtype)
    assert kla.attn_kv4_decode_workspace_bytes(len(lens), 8, 2, 128, max(lens), dtype) > 0
    o = kla.attn_kv4_decode_step(q, codes, scales, table, i32(lens), scale=0.2, max_len=max(lens))
    check(o, q, kv, 0.2, dtype)
    for _ in range(3):
        assert torch.equal(o, kla.attn_kv4_decode_step(q, codes, scales, table, i32(lens), scale=0.2, max_len=max(lens)))


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("D,Hkv", [(128, 1), (64, 4)])
def test_decode_of_a_large_cache(dtype, D, Hkv):
    """A bound on the lengths that stands for a cache past what the device keeps: its codes are
    read past the caches, and most runs are empty."""
    lens = [1, 33, 700, 0, 2000, 1664, 1665, 3400]
    codes, scales, table, kv = fill(lens, Hkv, D, 64)
    q = torch.randn(len(lens), 4, D, device=DEV).to(dtype)
    check(kla.attn_kv4_decode_step(q, codes, scales, table, i32(lens), max_len=200000), q, kv, D ** -0.5, dtype)


def test_many_short_sequences():
    lens = [int(n) for n in np.random.default_rng(0).integers(0, 90, 700)]
    codes, scales, table, kv = fill(lens, 2, 64, 16)
    q = torch.randn(700, 6, 64, device=DEV).to(BF)
    check(kla.attn_kv4_decode_step(q, codes, scales, table, i32(lens)), q, kv, 0.125, BF)


def test_large_scores():
    """One key dominates; and scores far apart, where most weights vanish."""
    codes, scales, table, kv = fill([400, 400], 1, 64, 16)
    q = 50 * torch.randn(2, 4, 64, device=DEV)
    for dtype in (BF, F32):
        qq = q.to(dtype)
        check(kla.attn_kv4_decode_step(qq, codes, scales, table, i32([400, 400])), qq, kv, 0.125, dtype)


def test_lengths_beyond_the_table_or_the_bound():
    codes, scales, table, kv = fill([100, 60], 1, 64, 16)
    q = torch.randn(2, 2, 64, device=DEV).to(BF)
    whole = kla.attn_kv4_decode_step(q, codes, scales, table, i32([100, 60]), max_len=50)
    check(whole, q, [(k[:, :50], v[:, :50]) for k, v in kv], 0.125, BF, "bound")
    got = kla.attn_kv4_decode_step(q, codes, scales, table[:, :2].contiguous(), i32([2 ** 31 - 1, -5]),
                                   max_len=100000)
    check(got[:1], q[:1], [(kv[0][0][:, :32], kv[0][1][:, :32])], 0.125, BF, "table")
    assert not got[1].any()


def test_missing_pages_are_left_out():
    codes, scales, table, kv = fill([100], 1, 64, 16)
    q = torch.randn(1, 2, 64, device=DEV).to(BF)
    t = table.clone()
    t[0, 1], t[0, 4] = -7, codes.shape[0]
    keep = np.r_[0:16, 32:64, 80:100]
    check(kla.attn_kv4_decode_step(q, codes, scales, t, i32([100])), q,
          [(kv[0][0][:, keep], kv[0][1][:, keep])], 0.125, BF)
    t.fill_(-1)
    assert not kla.attn_kv4_decode_step(q, codes, scales, t, i32([100])).any()


def test_shared_pages():
    """Two sequences with the same first pages, as after a common prompt."""
    codes, scales, table, kv = fill([80, 40], 1, 64, 16)
    t = table.clone()
    t[1, :3], t[1, 3:] = table[0, :3], -1
    q = torch.randn(2, 2, 64, device=DEV).to(BF)
    check(kla.attn_kv4_decode_step(q, codes, scales, t, i32([80, 45])), q,
          [kv[0], (kv[0][0][:, :45], kv[0][1][:, :45])], 0.125, BF)


def test_steps_in_a_graph_on_another_stream():
    """Append and attend, captured once; lengths and tokens advance between replays."""
    lens = [70, 3000]
    codes, scales, table, kv = fill([n + 8 for n in lens], 2, 128, 64)
    eager = codes.clone(), scales.clone()
    q, k, v = torch.zeros(2, 8, 128, device=DEV, dtype=BF), *(torch.zeros(2, 2, 1, 128, device=DEV, dtype=BF) for _ in "kv")
    start, now = i32(lens), i32([n + 1 for n in lens])

    def step(codes, scales):
        kla.kv4_append(k, v, codes, scales, table, start)
        return kla.attn_kv4_decode_step(q, codes, scales, table, now, max_len=3008)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        o = step(codes, scales)
    for _ in range(4):
        for x in (q, k, v):
            x.normal_()
        graph.replay()
        torch.cuda.synchronize()
        want = step(*eager)
        torch.cuda.synchronize()
        assert torch.equal(o, want) and torch.equal(codes, eager[0]) and torch.equal(scales, eager[1])
        start += 1
        now += 1


def test_parts_of_a_batch():
    """Slices of the block table, the lengths and the starts, which are aligned to 4 bytes only."""
    lens = [40, 17, 33]
    codes, scales, table, kv = fill(lens, 1, 64, 16)
    assert table.shape[1] == 3
    q = torch.randn(3, 4, 64, device=DEV).to(BF)
    whole = kla.attn_kv4_decode_step(q, codes, scales, table, i32(lens))
    part = kla.attn_kv4_decode_step(q[1:], codes, scales, table[1:], i32([0] + lens)[2:])
    assert torch.equal(part, whole[1:])
    k, v = make_kv([2, 2], 1, 64, BF, 5)
    cu, host = packed([2, 2])
    one, two = (codes.clone(), scales.clone()), (codes.clone(), scales.clone())
    kla.kv4_append(k, v, *one, table[1:], i32([9, 17, 33])[1:], cu, host)
    kla.kv4_append(k, v, *two, table[1:].clone(), i32([17, 33]), cu, host)
    assert torch.equal(one[0], two[0]) and torch.equal(one[1], two[1]) and not torch.equal(one[0], codes)


def test_refusals():
    codes, scales = kla.kv4_cache(4, 2, 16, 64, DEV)
    q, k = torch.zeros(1, 4, 64, device=DEV), torch.zeros(1, 2, 1, 64, device=DEV)
    table, one = i32([[0, 1]]), i32([1])
    with pytest.raises(TypeError):
        kla.attn_kv4_decode_step(q, codes.int(), scales, table, one)
    with pytest.raises(ValueError):
        kla.attn_kv4_decode_step(q, codes, scales[..., :1], table, one)
    with pytest.raises(ValueError):
        kla.attn_kv4_decode_step(q[..., :32].contiguous(), codes, scales, table, one)
    with pytest.raises(TypeError):
        kla.attn_kv4_decode_step(q, codes, scales, table.long(), one)
    with pytest.raises(kla.KlaError):
        kla.attn_kv4_decode_step(q[:, :3].contiguous(), codes, scales, table, one)
    with pytest.raises(kla.KlaError):
        kla.attn_kv4_decode_step(q, codes, scales, table, one, max_len=2 ** 32 + 1)
    with pytest.raises(ValueError):
        kla.kv4_append(k[:, :1].contiguous(), k, codes, scales, table, one)
    with pytest.raises(ValueError):
        kla.kv4_append(k, k, codes, scales, table, i32([1, 2]))
    with pytest.raises(ValueError):
        kla.kv4_append(k.cpu(), k, codes, scales, table, one)
    with pytest.raises(kla.KlaError):
        kla.kv4_append(k, k, codes[:, :, :, :8].contiguous(), scales[:, :, :, :8].contiguous(), table, one)
