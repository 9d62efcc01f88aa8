"""A stack that serves long prompts in a bounded cache: linear attention, and softmax attention
over a 4-bit cache whose tokens are weighed and cut to a budget.  Prompts come in two chunks, then
single tokens over what the cut left; each mixer against its own fp64 oracle at the inputs it was
given."""

import numpy as np
import pytest
import torch

from gated_delta_rule_kla_amd import inputs, kla
from oracle.attn_oracle import U32, attend, quantise, values
from oracle.kv4_oracle import evict, weigh
from oracle.la_oracle import la_decode_step, la_forward

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a GPU")]

DEV = torch.device("cuda:0")
BF = torch.bfloat16
f = inputs.to_f64


def near(got, ref, tol=2e-2):
    """The framework's criterion for bf16: of the largest value."""
    got = f(got)
    assert np.isfinite(got).all()
    assert np.abs(got - ref).max() <= tol * np.abs(ref).max()


@pytest.mark.parametrize("D,page", [(64, 16), (128, 64)])
def test_chunks_eviction_and_tokens(D, page):
    gen = torch.Generator().manual_seed(D)
    Hq, Hkv, M, N = 4, 2, 320 // page, 3
    budget, recent = 64, 8

    def rnd(*shape, std=1.0):
        return (torch.randn(*shape, generator=gen) * std).to(BF).to(DEV)

    table = torch.randperm(N * M, generator=gen).to(torch.int32).reshape(N, M).to(DEV)
    codes, scales = kla.kv4_cache(N * M, Hkv, page, D, DEV)
    weights = kla.kv4_weights(table, Hkv, page)
    want_w, err_w = np.zeros(weights.shape), np.zeros(weights.shape)
    hist = [[[np.zeros((0, D))] * Hkv, [np.zeros((0, D))] * Hkv] for _ in range(N)]  # cached K, V by key head
    S, rS = torch.zeros(N, Hq, D, D, device=DEV), np.zeros((N, Hq, D, D))
    now = torch.zeros(N, dtype=torch.int32, device=DEV)

    def remember(ak, av, spans):
        for i, (b, sl) in enumerate(spans):
            for j, p in ((0, ak), (1, av)):
                new = values(*quantise(f(p)[b, :, sl]))
                hist[i][j] = [np.concatenate([hist[i][j][h], new[h]]) for h in range(Hkv)]

    def expect(aq, ao, lse, spans):
        for i, (b, sl) in enumerate(spans):
            m = sl.stop - sl.start
            for h in range(Hq):
                k, v = (hist[i][j][h // 2] for j in (0, 1))
                mask = np.tril(np.ones((m, len(k)), bool), len(k) - m)
                want, wl, _, _ = attend(f(aq)[b, h, sl], k, v, D ** -0.5, mask, 0)
                near(ao[b, h, sl], want)
                assert np.abs(f(lse)[b, h, sl] - wl).max() <= 1e-3
                w, e = weigh(f(aq)[b, h, sl], k, f(lse)[b, h, sl], D ** -0.5, mask)
                want_w[i, h // 2, :len(k)] += w
                err_w[i, h // 2, :len(k)] += e + 2 * U32 * want_w[i, h // 2, :len(k)]

    for lens in ([70, 1, 200], [19, 5, 33]):
        T = sum(lens)
        host = torch.tensor(np.concatenate([[0], np.cumsum(lens)]), dtype=torch.int32)
        cu, b = host.to(DEV), host.tolist()
        spans = [(0, slice(x, y)) for x, y in zip(b, b[1:])]
        q, k, v = rnd(1, Hq, T, D, std=D ** -0.5), rnd(1, Hq, T, D, std=D ** -0.5), rnd(1, Hq, T, D)
        g = -0.1 * torch.nn.functional.softplus(rnd(1, Hq, T))
        y, S = kla.la_chunk_fwd(q, k, v, g, S, cu, cu_seqlens_host=host, final_state=S)
        ry, rS, *_ = la_forward(f(q), f(k), f(v), f(g), rS, b)
        near(y, ry)
        near(S, rS, 1e-4)
        ak, av = rnd(1, Hkv, T, D), rnd(1, Hkv, T, D)
        kla.kv4_append(ak, av, codes, scales, table, now, cu, host)
        now += (cu[1:] - cu[:-1]).to(torch.int32)
        remember(ak, av, spans)
        ao, lse = kla.attn_kv4_chunk_fwd(y, codes, scales, table, now, cu, max_len=320, cu_seqlens_host=host)
        kla.attn_kv4_weigh(y, lse, codes, scales, table, now, weights, cu, max_len=320, cu_seqlens_host=host)
        expect(y, ao, lse, spans)
        assert (np.abs(f(weights) - want_w) <= err_w + 4 * U32 * want_w).all()

    lens = now.tolist()
    before = f(weights)
    now, kept = kla.kv4_evict(codes, scales, table, now, weights, budget, recent)
    assert now.tolist() == [min(n, budget) for n in lens]
    want_w[:], err_w[:] = f(weights), 0
    for i in range(N):
        for h in range(Hkv):
            stay = evict(before[i, h, :lens[i]], lens[i], budget, recent)
            np.testing.assert_array_equal(kept[i, h].cpu().numpy()[:len(stay)], stay)
            np.testing.assert_array_equal(want_w[i, h, :len(stay)], before[i, h, stay])
            for j in (0, 1):
                hist[i][j][h] = hist[i][j][h][stay]

    spans = [(i, slice(0, 1)) for i in range(N)]
    for _ in range(3):
        q, k, v = rnd(N, Hq, D, std=D ** -0.5), rnd(N, Hq, D, std=D ** -0.5), rnd(N, Hq, D)
        g = -0.1 * torch.nn.functional.softplus(rnd(N, Hq))
        y = kla.la_decode_step(q, k, v, g, S)
        ry, rS = la_decode_step(f(q), f(k), f(v), f(g), rS)
        near(y, ry)
        ak, av = rnd(N, Hkv, 1, D), rnd(N, Hkv, 1, D)
        kla.kv4_append(ak, av, codes, scales, table, now)
        now = now + 1
        remember(ak, av, spans)
        aq = y[:, :, None].contiguous()
        ao, lse = kla.attn_kv4_chunk_fwd(aq, codes, scales, table, now, max_len=320)
        kla.attn_kv4_weigh(aq, lse, codes, scales, table, now, weights, max_len=320)
        expect(aq, ao, lse, spans)
        near(kla.attn_kv4_decode_step(y, codes, scales, table, now), f(ao[:, :, 0]), 2 ** -6)
    assert (np.abs(f(weights) - want_w) <= err_w + 4 * U32 * want_w).all()
