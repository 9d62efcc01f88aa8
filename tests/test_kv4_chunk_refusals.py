"""What the calls of new tokens over the 4-bit cache and of its eviction refuse (on the host,
before any HIP call), and the eviction oracle's pins."""

import ctypes
import os

import numpy as np
import pytest

from gated_delta_rule_kla_amd import kla
from oracle.attn_oracle import attend
from oracle.kv4_oracle import evict, weigh

needs_lib = pytest.mark.skipif(not os.path.exists(kla.lib_path()), reason="libkla.so not built")

FAKE = 0x7F0000000000  # never dereferenced
OK, NULL, SHAPE, DTYPE, UNSUPPORTED, SEQLENS, WORKSPACE, ALIGN, PARAM = 0, -1, -2, -3, -4, -5, -7, -8, -11


def ints(*x):
    return ctypes.cast((ctypes.c_int32 * len(x))(*x), ctypes.c_void_p)


def chunk(q=FAKE, codes=FAKE, scale=0.1, cu=None, host=None, N=2, B=2, Hq=8, Hkv=4, T=10, D=64, P=8, page=16, M=4,
          max_len=64, dtype=0, ws=None, wsb=0):
    return kla.lib().kla_attn_kv4_chunk_fwd(q, codes, FAKE, FAKE, FAKE, scale, FAKE, None, cu, host, N, B, Hq, Hkv, T,
                                            D, P, page, M, max_len, dtype, ws, wsb, None)


def weights(q=FAKE, codes=FAKE, scale=0.1, cu=None, host=None, N=2, B=2, Hq=8, Hkv=4, T=10, D=64, P=8, page=16, M=4,
            max_len=64, dtype=0, W=64):
    return kla.lib().kla_attn_kv4_weigh(q, FAKE, codes, FAKE, FAKE, FAKE, scale, FAKE, cu, host, N, B, Hq, Hkv, T, D,
                                        P, page, M, max_len, W, dtype, None)


@needs_lib
@pytest.mark.parametrize("call", [chunk, weights])
def test_refusals_of_new_tokens(call):
    assert call(dtype=2) == DTYPE
    for bad in (dict(Hq=0), dict(Hq=6), dict(Hkv=0), dict(T=-1), dict(N=3), dict(P=0), dict(M=0), dict(max_len=-1),
                dict(max_len=2 ** 31 - 1), dict(T=2 ** 31 - 1), dict(N=-1, B=-1), dict(T=2 ** 30, Hq=16, B=1, N=1),
                dict(N=2 ** 24, B=2 ** 24, T=1)):
        assert call(**bad) == SHAPE, bad
    for bad in (dict(D=32), dict(D=256), dict(page=24), dict(page=1 << 21)):
        assert call(**bad) == UNSUPPORTED, bad
    for scale in (float("nan"), float("inf"), 3e38):
        assert call(scale=scale) == PARAM
    assert call(q=None) == NULL and call(codes=None) == NULL
    assert call(q=FAKE + 2) == ALIGN and call(codes=FAKE + 4) == ALIGN
    assert call(cu=FAKE, N=1, B=1) == NULL and call(host=ints(0, 10), N=1, B=1) == NULL
    assert call(cu=FAKE, host=ints(0, 7, 5, 10), N=3, B=1) == SEQLENS
    assert call(cu=FAKE, host=ints(0, 4, 5, 10), N=3, B=2) == SHAPE
    assert call(N=0, B=0) == OK and call(T=0) == OK


@needs_lib
def test_workspaces_and_room():
    L = kla.lib()
    need = L.kla_attn_kv4_chunk_workspace_bytes(None, None, 2, 2, 8, 4, 1, 128, 100000, 0)
    assert need > 0 and chunk(T=1, D=128, max_len=100000) == WORKSPACE
    assert chunk(T=1, D=128, max_len=100000, ws=FAKE, wsb=need - 1) == WORKSPACE
    assert L.kla_attn_kv4_chunk_workspace_bytes(None, None, 3, 2, 8, 4, 1, 128, 100000, 0) == 0
    assert weights(W=63) == SHAPE


@needs_lib
def test_refusals_of_eviction():
    def cut(codes=FAKE, new=FAKE, budget=10, recent=2, N=2, Hkv=4, D=64, P=8, page=16, M=4, W=64, ws=FAKE, wsb=1 << 40):
        return kla.lib().kla_kv4_evict(codes, FAKE, FAKE, FAKE, FAKE, new, FAKE, budget, recent, N, Hkv, D, P, page, M,
                                       W, ws, wsb, None)

    for bad in (dict(budget=0), dict(budget=-5), dict(recent=-1), dict(recent=11), dict(budget=2 ** 31 - 1)):
        assert cut(**bad) == PARAM, bad
    for bad in (dict(W=63), dict(N=-1), dict(Hkv=0), dict(P=0), dict(N=2 ** 24), dict(N=2 ** 20, budget=2 ** 20)):
        assert cut(**bad) == SHAPE, bad
    assert cut(D=96) == UNSUPPORTED and cut(page=8) == UNSUPPORTED
    assert cut(codes=None) == NULL and cut(new=None) == NULL
    assert cut(codes=FAKE + 8) == ALIGN and cut(new=FAKE + 2) == ALIGN
    assert cut(ws=None) == WORKSPACE and cut(wsb=100) == WORKSPACE
    assert cut(N=0) == OK
    assert kla.lib().kla_kv4_evict_workspace_bytes(2, 4, 64, 0, 16, 4) == 0
    assert kla.lib().kla_kv4_evict_workspace_bytes(2, 4, 64, 10, 16, 4) >= 2 * 4 * 10 * 96


def test_weights_sum_to_the_queries():
    r = np.random.default_rng(0)
    q, k, v = r.normal(size=(5, 8)), r.normal(size=(12, 8)), r.normal(size=(12, 3))
    mask = np.tril(np.ones((5, 12), bool), 7)
    _, lse, _, _ = attend(q, k, v, 0.3, mask, 0.0)
    w, _ = weigh(q, k, lse, 0.3, mask)
    assert abs(w.sum() - 5) < 1e-12
    lse[0] = -np.inf
    assert abs(weigh(q, k, lse, 0.3, mask)[0].sum() - 4) < 1e-12


def test_eviction_keeps_order_and_the_earlier_of_equals():
    w = np.array([1.0, 5, 1, np.nan, 0, 1, -2, 9])
    assert evict(w, 8, 8, 2).tolist() == list(range(8))
    assert evict(w, 8, 4, 1).tolist() == [0, 1, 3, 7]
    assert evict(w, 8, 5, 1).tolist() == [0, 1, 2, 3, 7]
    assert evict(w, 8, 3, 3).tolist() == [5, 6, 7]
