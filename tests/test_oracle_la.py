"""The linear attention oracle's pins, and the refusals of its entry points (CPU)."""

import ctypes
import os

import numpy as np
import pytest

from gated_delta_rule_kla_amd import kla
from oracle.la_oracle import la_backward, la_decode_step, la_forward

needs_lib = pytest.mark.skipif(not os.path.exists(kla.lib_path()), reason="libkla.so not built")


def make(B=1, H=2, T=11, dk=4, dv=3, N=None, seed=0):
    r = np.random.default_rng(seed)
    N = B if N is None else N
    return (r.normal(size=(B, H, T, dk)), r.normal(size=(B, H, T, dk)), r.normal(size=(B, H, T, dv)),
            -r.random((B, H, T)), r.normal(size=(B, H, T, dv)), r.normal(size=(N, H, dk, dv)), r.normal(size=(N, H, dk, dv)))


def test_without_decay_it_is_a_masked_product():
    q, k, v, g, _, _, _ = make(T=20)
    o, S, _, _ = la_forward(q, k, v, 0 * g)
    np.testing.assert_allclose(o, np.tril(q @ k.swapaxes(2, 3)) @ v, rtol=1e-12, atol=1e-12)
    np.testing.assert_allclose(S, k.swapaxes(2, 3) @ v, rtol=1e-12, atol=1e-12)


def test_a_decay_of_nothing_forgets():
    q, k, v, g, _, s0, _ = make(T=9)
    g[:, :, 4] = -np.inf
    o, S, _, _ = la_forward(q, k, v, g, s0)
    cut = [x[:, :, 4:] for x in (q, k, v, g)]
    o2, S2, _, _ = la_forward(*cut)
    np.testing.assert_allclose(o[:, :, 4:], o2)
    np.testing.assert_allclose(S, S2)


def test_packed_is_each_sequence_and_a_continued_one():
    q, k, v, g, do, s0, df = make(T=10, N=3)
    o, S, _, _ = la_forward(q, k, v, g, s0, [0, 4, 4, 10])
    for n, (a, z) in enumerate([(0, 4), (4, 4), (4, 10)]):
        o2, S2, _, _ = la_forward(q[:, :, a:z], k[:, :, a:z], v[:, :, a:z], g[:, :, a:z], s0[n:n + 1])
        np.testing.assert_allclose(o[:, :, a:z], o2)
        np.testing.assert_allclose(S[n:n + 1], S2)
    o1, S1, _, _ = la_forward(*(x[:, :, :6] for x in (q, k, v, g)), s0[:1])
    o2, S2, _, _ = la_forward(*(x[:, :, 6:] for x in (q, k, v, g)), S1)
    o, S, _, _ = la_forward(q, k, v, g, s0[:1])
    np.testing.assert_allclose(np.concatenate([o1, o2], 2), o)
    np.testing.assert_allclose(S2, S)


@pytest.mark.parametrize("fixed", [False, True])
def test_gradients_are_differences(fixed):
    q, k, v, g, do, s0, df = make(B=2, T=6)
    if fixed:
        g = -np.array([0.3, 0.7])
    want, _ = la_backward(q, k, v, g, do, s0, df)

    def loss():
        o, S, _, _ = la_forward(q, k, v, g, s0)
        return (o * do).sum() + (S * df).sum()

    for x, d in zip((q, k, v, g, s0), want):
        flat, r = x.reshape(-1), np.random.default_rng(1)
        for i in r.choice(flat.size, min(flat.size, 12), replace=False):
            keep, h = flat[i], 1e-5
            flat[i] = keep + h
            up = loss()
            flat[i] = keep - h
            down = loss()
            flat[i] = keep
            assert abs((up - down) / (2 * h) - d.reshape(-1)[i]) < 1e-6


def test_steps_are_the_prompt():
    q, k, v, g, _, s0, _ = make(T=7)
    o, S, _, _ = la_forward(q, k, v, g, s0)
    state = s0
    for t in range(7):
        y, state = la_decode_step(q[:, :, t], k[:, :, t], v[:, :, t], g[:, :, t], state)
        np.testing.assert_allclose(y, o[:, :, t])
    np.testing.assert_allclose(state, S)


FAKE = 0x7F0000000000  # never dereferenced
OK, NULL, SHAPE, DTYPE, UNSUPPORTED, SEQLENS, WORKSPACE, ALIGN, PARAM = 0, -1, -2, -3, -4, -5, -7, -8, -11


def fwd(q=FAKE, g=FAKE, decay=None, s0=None, cu=None, host=None, N=2, B=2, H=4, T=10, dk=64, dv=64, dtype=0, ws=None,
        wsb=0):
    return kla.lib().kla_la_chunk_fwd(q, FAKE, FAKE, g, decay, s0, FAKE, None, cu, host, N, B, H, T, dk, dv, dtype, ws,
                                      wsb, None)


def bwd(q=FAKE, g=FAKE, decay=None, s0=None, cu=None, host=None, N=2, B=2, H=4, T=10, dk=64, dv=64, dtype=0, ws=FAKE,
        wsb=0, dg=FAKE):
    return kla.lib().kla_la_chunk_bwd(q, FAKE, FAKE, g, decay, s0, FAKE, None, FAKE, FAKE, FAKE, dg, None, cu, host, N,
                                      B, H, T, dk, dv, dtype, ws, wsb, None)


def ints(*x):
    return ctypes.cast((ctypes.c_int32 * len(x))(*x), ctypes.c_void_p)


@needs_lib
@pytest.mark.parametrize("call", [fwd, bwd])
def test_refusals(call):
    assert call(dtype=2) == DTYPE
    for bad in (dict(H=0), dict(T=-1), dict(dk=0), dict(dv=-16), dict(N=3), dict(T=2 ** 31 - 10), dict(B=-1, N=-1),
                dict(B=2 ** 16, N=2 ** 16, H=2 ** 16), dict(B=2 ** 12, N=2 ** 12, H=2 ** 14, T=1)):
        assert call(**bad) == SHAPE, bad
    for bad in (dict(dk=8), dict(dk=272), dict(dv=40), dict(dv=512)):
        assert call(**bad) == UNSUPPORTED, bad
    assert call(q=None) == NULL and call(g=None) == NULL
    assert call(decay=FAKE) == PARAM
    assert call(q=FAKE + 2) == ALIGN and call(s0=FAKE + 4) == ALIGN and call(g=None, decay=FAKE + 2) == ALIGN
    assert call(cu=FAKE, N=1, B=1) == NULL and call(host=ints(0, 10), N=1, B=1) == NULL
    for c in ((0, 6, 5, 10), (1, 4, 4, 10), (0, 4, 4, 11)):
        assert call(cu=FAKE, host=ints(*c), N=3, B=1) == SEQLENS
    assert call(cu=FAKE + 2, host=ints(0, 4, 4, 10), N=3, B=1) == ALIGN
    assert call(cu=FAKE, host=ints(0, 4, 4, 10), N=3, B=2) == SHAPE


@needs_lib
def test_workspaces():
    L = kla.lib()
    assert bwd(wsb=16) == WORKSPACE and bwd(ws=None, wsb=1 << 40) == WORKSPACE
    need = L.kla_la_chunk_bwd_workspace_bytes(None, None, 2, 2, 4, 100, 64, 64, 0)
    assert need >= 2 * (2 * 2 * 4 * 64 * 64 * 2)  # two states of each of two chunks
    assert L.kla_la_chunk_bwd_workspace_bytes(None, None, 3, 2, 4, 100, 64, 64, 0) == 0
    assert L.kla_la_chunk_workspace_bytes(None, None, 2, 2, 4, 100, 64, 60, 0) == 0
    assert bwd(g=None, decay=FAKE, dg=None, T=0, ws=None) == NULL


@needs_lib
def test_step_refusals():
    def step(q=FAKE, g=FAKE, decay=None, N=2, H=4, dk=64, dv=64, dtype=0):
        return kla.lib().kla_la_decode_step(q, FAKE, FAKE, g, decay, FAKE, FAKE, N, H, dk, dv, dtype, None)

    assert step(dtype=-1) == DTYPE and step(N=-1) == SHAPE and step(H=0) == SHAPE
    assert step(dk=24) == UNSUPPORTED and step(dv=264) == UNSUPPORTED
    assert step(N=2 ** 30, H=2 ** 20) == SHAPE and step(N=2 ** 20, H=2 ** 8) == SHAPE
    assert step(q=None) == NULL and step(g=None) == NULL and step(decay=FAKE) == PARAM
    assert step(q=FAKE + 8) == ALIGN and step(N=0) == OK
