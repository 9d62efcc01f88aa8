"""The operators together, as a stack serves a prompt: a delta-rule mixer, a gated recurrence and
softmax attention over a 4-bit cache in turn, a packed batch of prompts, one of them continued
after its cached tokens, then single tokens; against the same stack in fp64.

Every mixer takes the layer's rounded input, so that each is held to its own oracle at the
inputs it was given; nothing accumulates over layers."""

import numpy as np
import pytest
import torch

from gated_delta_rule_kla_amd import inputs, kla
from oracle import kla_decode_step, kla_forward
from oracle.attn_oracle import attend, quantise, values
from oracle.glr_oracle import glr_forward

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a GPU")]

DEV = torch.device("cuda:0")
BF = torch.bfloat16
f = inputs.to_f64


def near(got, ref, tol=2e-2):
    """The framework's criterion for bf16: of the largest value."""
    got = f(got)
    assert np.isfinite(got).all()
    assert np.abs(got - ref).max() <= tol * np.abs(ref).max()


def heads(x, n):  # [1, n D, T, ...] of a layer's rows into heads, rounded as the layer would
    T = x.shape[2]
    return x.to(BF).reshape(1, T, n, -1).transpose(1, 2).contiguous()


@pytest.mark.parametrize("D", [64, 128])
def test_prompts_a_continuation_and_tokens(D):
    gen = torch.Generator().manual_seed(D)
    lens, Hq, Hkv, page = [70, 1, 200], 4, 2, 16
    N, T = len(lens), sum(lens)
    host = torch.tensor(np.concatenate([[0], np.cumsum(lens)]), dtype=torch.int32)
    cu, b = host.to(DEV), host.tolist()

    def rnd(*shape, std=1.0):
        return (torch.randn(*shape, generator=gen) * std).to(BF).to(DEV)

    # a delta-rule layer
    q, k, v = rnd(1, Hq, T, D, std=D ** -0.5), rnd(1, Hq, T, D, std=D ** -0.5), rnd(1, Hq, T, D)
    g, eta = (-torch.nn.functional.softplus(rnd(1, Hq, T))), torch.sigmoid(rnd(1, Hq, T))
    o, S = kla.chunk_fwd(q, k, v, g, eta, 1e-6, cu_seqlens=cu, cu_seqlens_host=host)
    ro, rS = kla_forward(f(q), f(k), f(v), f(g), f(eta), 1e-6, np.zeros((N, Hq, D, D)), cu_seqlens=b)
    near(o, ro)

    # its output through a gated recurrence, one head of the whole width
    x = o.transpose(1, 2).reshape(1, 1, T, Hq * D).contiguous()
    gate = -torch.nn.functional.softplus(rnd(1, 1, T, Hq * D))
    y, h = kla.glr_chunk_fwd(x, gate, None, cu, cu_seqlens_host=host)
    ry, rh, *_ = glr_forward(f(x), f(gate), None, b)
    near(y, ry)

    # attention over the prompts, whose keys go to the cache
    table, codes, scales = torch.arange(N * 16, dtype=torch.int32, device=DEV).flip(0).reshape(N, 16), *kla.kv4_cache(
        N * 16, Hkv, page, D, DEV)
    ak, av = rnd(1, Hkv, T, D), rnd(1, Hkv, T, D)
    aq = y.reshape(1, T, Hq, D).transpose(1, 2).contiguous()
    ao, lse = kla.attn_fwd(aq, ak, av, cu_seqlens=cu, cu_seqlens_host=host)
    zero = torch.zeros(N, dtype=torch.int32, device=DEV)
    kla.kv4_append(ak, av, codes, scales, table, zero, cu, host)
    for n in range(N):
        for hh in range(Hq):
            sl = slice(b[n], b[n + 1])
            mask = np.tril(np.ones((lens[n], lens[n]), bool))
            want, *_ = attend(f(aq)[0, hh, sl], f(ak)[0, hh // 2, sl], f(av)[0, hh // 2, sl], D ** -0.5, mask, 0)
            near(ao[0, hh, sl], want)

    # the last sequence goes on with 19 more tokens, attending to what its cache holds
    more, n = 19, 2
    nk, nv, nq = rnd(1, Hkv, more, D), rnd(1, Hkv, more, D), rnd(1, Hq, more, D)
    at = torch.tensor([lens[n]], dtype=torch.int32, device=DEV)
    kla.kv4_append(nk, nv, codes, scales, table[n:], at)
    both = torch.tensor([0, lens[n] + more], dtype=torch.int32)
    ck, cv = kla.kv4_read(codes, scales, table[n:], at * 0, both.to(DEV), BF, both)
    co, _ = kla.attn_fwd(nq, ck, cv)
    kept = [values(*quantise(np.concatenate([f(p)[0, :, b[n]:], f(s)[0]], 1))) for p, s in ((ak, nk), (av, nv))]
    np.testing.assert_array_equal(f(ck)[0], kept[0])
    np.testing.assert_array_equal(f(cv)[0], kept[1])
    for hh in range(Hq):
        mask = np.tril(np.ones((more, lens[n] + more), bool), lens[n])
        want, *_ = attend(f(nq)[0, hh], kept[0][hh // 2], kept[1][hh // 2], D ** -0.5, mask, 0)
        near(co[0, hh], want)
    lens[n] += more

    # three tokens for every sequence through the same three layers
    hist = [[np.concatenate([values(*quantise(f(p)[0, :, b[i]:b[i + 1]])), ], 1) for p in (ak, av)] for i in range(N)]
    hist[2] = list(kept)
    now = torch.tensor(lens, dtype=torch.int32, device=DEV)
    rS = f(S)
    rh = f(h)
    for _ in range(3):
        tq, tk, tv = rnd(N, Hq, D, std=D ** -0.5), rnd(N, Hq, D, std=D ** -0.5), rnd(N, Hq, D)
        tg, te = -torch.nn.functional.softplus(rnd(N, Hq)), torch.sigmoid(rnd(N, Hq))
        o = kla.decode_step(tq, tk, tv, tg, te, 1e-6, S)
        ro, rS = kla_decode_step(f(tq), f(tk), f(tv), f(tg), f(te), 1e-6, rS)
        near(o, ro)
        gate = -torch.nn.functional.softplus(rnd(N, 1, Hq * D))
        x = o.reshape(N, 1, Hq * D)
        y = kla.glr_decode_step(x, gate, h)
        rh = np.exp(f(gate)) * rh + f(x)
        near(y, rh)
        ak, av = rnd(N, Hkv, 1, D), rnd(N, Hkv, 1, D)
        kla.kv4_append(ak, av, codes, scales, table, now)
        now += 1
        aq = y.reshape(N, Hq, D)
        ao = kla.attn_kv4_decode_step(aq, codes, scales, table, now)
        for i in range(N):
            for j, p in ((0, ak), (1, av)):
                hist[i][j] = np.concatenate([hist[i][j], values(*quantise(f(p)[i]))], 1)
            for hh in range(Hq):
                kk, vv = hist[i][0][hh // 2], hist[i][1][hh // 2]
                want, *_ = attend(f(aq)[i, hh:hh + 1], kk, vv, D ** -0.5, np.ones((1, len(kk)), bool), 0)
                near(ao[i, hh:hh + 1], want)
