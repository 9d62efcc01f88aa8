"""Attention of new tokens over the 4-bit cache, and the weights they give, on the GPU against
fp64 oracles, within their bounds (the weights' bf16 rounding 2^-8 for bf16 queries, three bf16
terms, 2^-24, for fp32; half a step of the output's type)."""

import numpy as np
import pytest
import torch

from gated_delta_rule_kla_amd import kla
from oracle.attn_oracle import attend, quantise, values
from oracle.kv4_oracle import weigh
from test_gpu_kv4 import BF, DEV, F32, HALF, f64, i32, make_kv, packed, pages

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a GPU")]

DTYPES = [BF, F32]


class Cache:
    """A cache of lens tokens a sequence, and the values it holds [Hkv, tokens, D] per sequence."""

    def __init__(self, lens, Hkv, D, page=64, seed=0, room=None):
        self.lens, self.Hkv, self.D, self.page = lens, Hkv, D, page
        self.table, P = pages([max(n, 1) for n in lens] if room is None else room, page, seed)
        self.codes, self.scales = kla.kv4_cache(P, Hkv, page, D, DEV)
        self.codes.fill_(0x6B)
        self.scales.fill_(0xFF)  # what was not stored reads as NaN
        cu, host = packed(lens)
        k, v = make_kv(lens, Hkv, D, BF, seed)
        kla.kv4_append(k, v, self.codes, self.scales, self.table, i32([0] * len(lens)), cu, host)
        self.k, self.v = ([y[:, a:z] for a, z in zip(host, host[1:])] for y in (values(*quantise(f64(x)[0])) for x in (k, v)))

    def args(self):
        return self.codes, self.scales, self.table, i32(self.lens)


def queries(Hq, T, D, dtype, seed=1, B=1):
    gen = torch.Generator().manual_seed(seed)
    return torch.randn(B, Hq, T, D, generator=gen).to(dtype).to(DEV)


def seen(m, n, length=None, max_len=None):
    length = n if length is None else length
    mask = np.arange(n)[None, :] <= np.arange(m)[:, None] + (length - m)
    return mask & (np.arange(n)[None, :] < (n if max_len is None else max_len))


def check_rows(got, want, bound, dtype):
    far = np.abs(got - want) - (bound + HALF[dtype] * (np.abs(want) + bound) + 1e-30)
    assert not np.isnan(far).any() and far.max(initial=-1) <= 0, far.max()


def check(cache, new, q, o, lse, scale=None, max_len=None, skip=()):
    D, G = cache.D, q.shape[1] // cache.Hkv
    scale = D ** -0.5 if scale is None else scale
    dense = q.shape[0] > 1
    at = np.concatenate([[0], np.cumsum(new)])
    for n, m in enumerate(new):
        if n in skip:
            continue
        rows = (n, slice(0, m)) if dense else (0, slice(at[n], at[n] + m))
        for h in range(q.shape[1]):
            mask = seen(m, cache.lens[n], max_len=max_len)
            w, l, eo, el = attend(f64(q[rows[0], h, rows[1]]), cache.k[n][h // G], cache.v[n][h // G], scale, mask,
                                  HALF[q.dtype])
            check_rows(f64(o[rows[0], h, rows[1]]), w, eo, q.dtype)
            got = f64(lse[rows[0], h, rows[1]])
            some = np.isfinite(l)
            np.testing.assert_array_equal(got[~some], l[~some])
            assert (np.abs(got[some] - l[some]) <= el[some] + 2 ** -23 * np.abs(l[some])).all()


def check_weights(cache, new, q, lse, before, after, scale=None, max_len=None):
    D, G = cache.D, q.shape[1] // cache.Hkv
    scale = D ** -0.5 if scale is None else scale
    dense = q.shape[0] > 1
    at = np.concatenate([[0], np.cumsum(new)])
    before, after = f64(before), f64(after)
    for n, m in enumerate(new):
        rows = (n, slice(0, m)) if dense else (0, slice(at[n], at[n] + m))
        L = cache.lens[n]
        np.testing.assert_array_equal(after[n, :, L:], before[n, :, L:])
        for hk in range(cache.Hkv):
            want, err = before[n, hk, :L].copy(), np.zeros(L)
            for h in range(hk * G, hk * G + G):
                w, e = weigh(f64(q[rows[0], h, rows[1]]), cache.k[n][hk], f64(lse[rows[0], h, rows[1]]), scale,
                             seen(m, L, max_len=max_len))
                want, err = want + w, err + e
            check_rows(after[n, hk, :L], want, err + (G + 2) * 2.0 ** -24 * np.abs(want), F32)


def run(cache, new, Hq, dtype, dense=False, **kw):
    q = queries(Hq, new[0] if dense else sum(new), cache.D, dtype, B=len(new) if dense else 1)
    cu, host = (None, None) if dense else packed(new)
    o, lse = kla.attn_kv4_chunk_fwd(q, *cache.args(), cu, cu_seqlens_host=host, **kw)
    check(cache, new, q, o, lse, kw.get("scale"), kw.get("max_len"))
    w = torch.rand(len(new), cache.Hkv, cache.table.shape[1] * cache.page + 5, device=DEV)
    before = w.clone()
    kla.attn_kv4_weigh(q, lse, *cache.args(), w, cu, cu_seqlens_host=host, **kw)
    check_weights(cache, new, q, lse, before, w, kw.get("scale"), kw.get("max_len"))
    return q, o, lse


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("D,page,Hkv,G", [(128, 64, 2, 4), (64, 16, 3, 5), (128, 48, 1, 16), (64, 128, 4, 1)])
def test_few_new_tokens(dtype, D, page, Hkv, G):
    """Rows of one 32-row tile and a little more, keys over several runs."""
    new = [1, 5, 0, 3, 8, 1, 2]
    lens = [1, 5, 10, 3, 2100, 700, 64]
    run(Cache(lens, Hkv, D, page), new, Hkv * G, dtype)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("D,Hkv,G", [(128, 2, 4), (64, 1, 8), (128, 1, 3)])
def test_chunks(dtype, D, Hkv, G):
    """128- and 256-row tiles, ragged, at the start of a prompt and behind earlier tokens."""
    for new, lens in (([70, 1, 129, 33], [70, 1000, 300, 95]), ([300, 257], [300, 1300])):
        run(Cache(lens, Hkv, D, seed=D), new, Hkv * G, dtype)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("T,L", [(1, 3000), (1, 1), (7, 500), (200, 333)])
def test_dense(dtype, T, L):
    run(Cache([L, L, L], 2, 128, 32), [T] * 3, 8, dtype, dense=True)


@pytest.mark.parametrize("dtype", DTYPES)
def test_more_queries_than_keys(dtype):
    """The first queries see nothing: o = 0, lse = -inf, and they give no weight."""
    q, o, lse = run(Cache([10, 0, 100], 2, 64), [40, 20, 130], 4, dtype)
    assert not o[:, :, :30].any() and (lse[:, :, :30] == -float("inf")).all()
    assert not o[:, :, 40:60].any() and (lse[:, :, 40:60] == -float("inf")).all()


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("scale", [0.0, -0.3, 1e-3, 40.0])
def test_scales(dtype, scale):
    run(Cache([200, 90], 1, 64), [60, 3], 4, dtype, scale=scale)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("new", [[2, 3], [150, 90]])
def test_a_bound_below_the_lengths(dtype, new):
    run(Cache([700, 400], 2, 64), new, 4, dtype, max_len=250)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("new", [[1], [6], [200]])
def test_the_bound_only_cuts_the_work(dtype, new):
    """The block table's room and a tight bound: other runs, the same result within rounding."""
    cache = Cache([900], 1, 128, room=[20000])
    run(cache, new, 4, dtype)
    run(cache, new, 4, dtype, max_len=900)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("new", [4, 100, 600])
def test_values_that_are_not_finite(dtype, new):
    """NaN in keys and values of the newest tokens reaches the queries that see them and no others;
    a page that is not there is left out."""
    L, hole = 700, 2
    cache = Cache([L, L], 1, 64, 64, seed=5)
    at = L - max(new // 2, 1)
    page, pos = int(cache.table[0, at // 64]), at % 64
    cache.scales[page, 1, 0, pos, 1] = 255
    page2, pos2 = int(cache.table[1, (L - 1) // 64]), (L - 1) % 64
    cache.scales[page2, 0, 0, pos2, 0] = 255
    cache.table[:, hole] = torch.tensor([-1, 1 << 30], dtype=torch.int32)
    q = queries(4, 2 * new, 64, dtype)
    cu, host = packed([new, new])
    o, lse = kla.attn_kv4_chunk_fwd(q, *cache.args(), cu, cu_seqlens_host=host)
    w = kla.kv4_weights(cache.table, 1, 64)
    kla.attn_kv4_weigh(q, lse, *cache.args(), w, cu, cu_seqlens_host=host)
    assert not w[:, :, hole * 64:hole * 64 + 64].any()
    keep = np.r_[0:hole * 64, hole * 64 + 64:L]
    for n in range(2):
        first_bad = (at if n == 0 else L - 1) - (L - new)  # the first query that sees the NaN
        for h in range(4):
            mask = seen(new, L)[:, keep]
            want, l, eo, el = attend(f64(q[0, h, n * new:n * new + new]), cache.k[n][0][keep], cache.v[n][0][keep],
                                     64 ** -0.5, mask, HALF[dtype])
            got = f64(o[0, h, n * new:n * new + new])
            check_rows(got[:first_bad], want[:first_bad], eo[:first_bad], dtype)
            bad = np.isnan(got[first_bad:])
            if n == 0:
                assert bad[:, 32:].all() and not bad[:, :32].any()
            else:
                assert bad.all() and np.isnan(f64(lse[0, h, n * new + first_bad:n * new + new])).all()
    # a token whose key is NaN gets nothing from queries that do not see it, and their keys all
    total = f64(w[0, 0]).sum()
    assert abs(total - 4 * new) < 1e-3 * new


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("new", [[3, 3, 3], [100, 100, 100], [700, 10, 10]])
def test_offsets_of_the_device_decide(dtype, new):
    """Other lengths than the host's, also longer ones, and a padded batch: its rows keep theirs."""
    T = sum(new) + 7
    host = torch.tensor([0, new[0], new[0] + new[1], T], dtype=torch.int32)
    real = [3, 3, max(T - 40, 4), T - 1]  # an empty one, a long one, rows before and behind
    cu = torch.tensor(real, dtype=torch.int32, device=DEV)
    m = [b - a for a, b in zip(real, real[1:])]
    cache = Cache([50, max(m[1], 60), m[2] + 500], 2, 64, 32)
    q = queries(4, T, 64, dtype)
    q[:, :, :3], q[:, :, T - 1:] = float("nan"), float("nan")
    out, lse = torch.full_like(q, 7.0), torch.full((1, 4, T), 7.0, device=DEV)
    kla.attn_kv4_chunk_fwd(q, *cache.args(), cu, cu_seqlens_host=host, out=out, lse=lse)
    for x in (out, lse):
        assert (x[:, :, :3] == 7).all() and (x[:, :, T - 1:] == 7).all()
    part = slice(3, T - 1)
    check(cache, m, q[:, :, part], out[:, :, part], lse[:, :, part])
    w = kla.kv4_weights(cache.table, 2, 32)
    before = w.clone()
    kla.attn_kv4_weigh(q, lse, *cache.args(), w, cu, cu_seqlens_host=host)
    check_weights(cache, m, q[:, :, part], lse[:, :, part], before, w)


@pytest.mark.parametrize("dtype", DTYPES)
def test_one_token_as_the_decode_step(dtype):
    """Both read the same cache; each is within its bound of the oracle, so of the other."""
    lens = [5000, 17, 1, 2048]
    cache = Cache(lens, 2, 128)
    q = queries(8, 1, 128, dtype, B=4)
    o, _ = kla.attn_kv4_chunk_fwd(q, *cache.args())
    step = kla.attn_kv4_decode_step(q[:, :, 0].contiguous(), *cache.args())
    for n, L in enumerate(lens):
        for h in range(8):
            # |o - step| <= |o - want| + |step - want|, and each of those is at most the oracle's
            # bound (scores of loud keys are off by (D + 2) U32 of their magnitudes, which in fp32 is
            # more than the outputs' rounding) and half a step
            want, _, eo, _ = attend(f64(q[n, h]), cache.k[n][h // 4], cache.v[n][h // 4], 128 ** -0.5, seen(1, L), HALF[dtype])
            far = np.abs(f64(o[n, h]) - f64(step[n, h])[None])
            assert (far <= 2 * (eo + HALF[dtype] * (np.abs(want) + eo))).all()


@pytest.mark.parametrize("new", [[5, 5], [200, 90]])
def test_captured_and_replayed_on_another_stream(new):
    cache = Cache([900, 1500], 2, 128)
    args = cache.args()
    cu, host = packed(new)
    T = sum(new)
    q = queries(8, T, 128, BF)
    w = kla.kv4_weights(cache.table, 2, 64)

    def call():
        o, lse = kla.attn_kv4_chunk_fwd(q, *args, cu, cu_seqlens_host=host, max_len=1500)
        kla.attn_kv4_weigh(q, lse, *args, w, cu, cu_seqlens_host=host, max_len=1500)
        return o, lse

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        call()
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        got = call()
    for i in range(3):
        q.copy_(queries(8, T, 128, BF, 30 + i))
        args[3].copy_(i32([900 - 100 * i, 1500 - i]))
        cu.copy_(i32([0, new[0] - i, T]))
        w.fill_(i)
        graph.replay()
        torch.cuda.synchronize()
        have, after = [t.clone() for t in got], w.clone()
        w.fill_(i)
        for a, b in zip(have, call()):
            assert torch.equal(a, b)
        assert torch.equal(after, w)


def test_a_long_cache():
    """Offsets past 32 bits: pages far into a cache of 4.6 GB of codes, against a small cache of the same."""
    lens, D, Hkv, page = [5000], 128, 4, 64
    small = Cache(lens, Hkv, D, page)
    P = 140000
    codes, scales = kla.kv4_cache(P, Hkv, page, D, DEV)
    assert codes.numel() > 2 ** 32
    far = P - 1 - torch.arange(small.table.shape[1], device=DEV, dtype=torch.int32)[None]
    codes[far[0].long()] = small.codes[small.table[0].long()]
    scales[far[0].long()] = small.scales[small.table[0].long()]
    for T in (2, 300):
        q = queries(8, T, D, BF)
        cu, host = packed([T])
        a = kla.attn_kv4_chunk_fwd(q, *small.args(), cu, cu_seqlens_host=host)
        b = kla.attn_kv4_chunk_fwd(q, codes, scales, far, i32(lens), cu, cu_seqlens_host=host)
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
        w = [kla.kv4_weights(far, Hkv, page) for _ in "ab"]
        kla.attn_kv4_weigh(q, a[1], *small.args(), w[0], cu, cu_seqlens_host=host)
        kla.attn_kv4_weigh(q, a[1], codes, scales, far, i32(lens), w[1], cu, cu_seqlens_host=host)
        assert torch.equal(*w)
    w = torch.rand(1, Hkv, far.shape[1] * page, device=DEV)
    got = []
    for c, s, t in ((small.codes, small.scales, small.table), (codes, scales, far)):
        x = w.clone()
        n, kept = kla.kv4_evict(c, s, t, i32(lens), x, 1000, 10)
        got.append((x, kept, *kla.kv4_read(c, s, t, i32([0]), *packed([1000])[:1], BF, packed([1000])[1])))
    assert all(torch.equal(a, b) for a, b in zip(*got))
