"""The gated linear recurrence's oracle, pinned without its own formulas: closed forms, the
split of a sequence, packed against separate sequences, and central differences for the
gradients; and the arguments that kla_glr_* refuse (on the host, before any HIP call)."""

import os

import numpy as np
import pytest

from gated_delta_rule_kla_amd import kla
from oracle.glr_oracle import glr_backward, glr_forward

RNG = np.random.default_rng


def make(B=2, H=3, T=9, d=4, seed=0):
    r = RNG(seed)
    return r.normal(size=(B, H, T, d)), -np.logaddexp(0, r.normal(size=(B, H, T, d))), r.normal(size=(B, H, d))


def test_without_decay_it_sums():
    x, g, h0 = make()
    o, hf, *_ = glr_forward(x, np.zeros_like(g), h0)
    want = np.cumsum(x, 2) + h0[:, :, None]
    np.testing.assert_allclose(o, want, rtol=0, atol=1e-13)
    np.testing.assert_array_equal(hf, o[:, :, -1])


def test_without_input_it_decays():
    x, g, h0 = make()
    o, *_ = glr_forward(np.zeros_like(x), g, h0)
    np.testing.assert_allclose(o, np.exp(np.cumsum(g, 2)) * h0[:, :, None], rtol=1e-13)


def test_a_closed_gate_forgets():
    x, g, h0 = make()
    g[:, :, 4] = -np.inf
    o, *_ = glr_forward(x, g, h0)
    np.testing.assert_array_equal(o[:, :, 4], x[:, :, 4])
    rest, *_ = glr_forward(x[:, :, 5:], g[:, :, 5:], x[:, :, 4])
    np.testing.assert_array_equal(o[:, :, 5:], rest)


def test_a_sequence_can_be_split_and_packed():
    x, g, h0 = make(B=1, T=11)
    whole, hf, *_ = glr_forward(x, g, h0)
    first, h1, *_ = glr_forward(x[:, :, :4], g[:, :, :4], h0)
    second, h2, *_ = glr_forward(x[:, :, 4:], g[:, :, 4:], h1)
    np.testing.assert_array_equal(np.concatenate([first, second], 2), whole)
    np.testing.assert_array_equal(h2, hf)
    cu = [0, 4, 4, 11]  # an empty sequence keeps its state
    o, hp, *_ = glr_forward(x, g, np.concatenate([h0, h0 + 1, h1]), cu)
    np.testing.assert_array_equal(o, whole)
    np.testing.assert_array_equal(hp[1], (h0 + 1)[0])


def test_gradients_against_differences():
    x, g, h0 = make(B=1, H=2, T=7, d=3, seed=3)
    cu = [0, 3, 3, 7]
    h0 = RNG(5).normal(size=(3, 2, 3))
    do, df = RNG(6).normal(size=x.shape), RNG(7).normal(size=h0.shape)

    def loss(x, g, h0):
        o, hf, *_ = glr_forward(x, g, h0, cu)
        return (o * do).sum() + (hf * df).sum()

    dx, dg, d0, *_ = glr_backward(g, glr_forward(x, g, h0, cu)[0], do, h0, df, cu)
    for k, grad in enumerate((dx, dg, d0)):
        for i in np.ndindex(*grad.shape):
            two = []
            for s in (1e-6, -1e-6):
                args = [x.copy(), g.copy(), h0.copy()]
                args[k][i] += s
                two.append(loss(*args))
            assert abs((two[0] - two[1]) / 2e-6 - grad[i]) < 1e-8


def test_the_bound_covers_fp32_composed_another_way():
    """Pairs of tokens composed first, in fp32: within the bound, which is not wildly wide."""
    x, g, h0 = (t.astype(np.float32) for t in make(B=1, H=1, T=512, d=8, seed=9))
    o, hf, bound, _ = glr_forward(x.astype(np.float64), g.astype(np.float64), h0.astype(np.float64))
    a, h = np.exp(g), h0
    got = np.empty_like(x)
    for t in range(0, 512, 2):
        A, C = a[:, :, t] * a[:, :, t + 1], a[:, :, t + 1] * x[:, :, t] + x[:, :, t + 1]
        got[:, :, t] = a[:, :, t] * h + x[:, :, t]
        h = A * h + C
        got[:, :, t + 1] = h
    err = np.abs(got - o)
    assert (err <= bound).all()
    assert bound.max() < 3e-5 * np.abs(o).max()


# ---- refusals --------------------------------------------------------------------------------

pytestmark = pytest.mark.skipif(not os.path.exists(kla.lib_path()), reason="libkla.so not built")

FAKE = 0x7F0000000000  # never dereferenced


def call(fn, **kw):
    import ctypes
    a = dict(N=2, B=2, H=4, T=100, d=64, dtype=0, cu=None, cuh=None, ws=None, wsb=0, p=FAKE, s=FAKE, N_=None)
    a.update(kw)
    cuh = None if a["cuh"] is None else (ctypes.c_int32 * len(a["cuh"]))(*a["cuh"])
    cuh_p = None if cuh is None else ctypes.addressof(cuh)
    tail = (a["cu"], cuh_p, a["N"], a["B"], a["H"], a["T"], a["d"], a["dtype"], a["ws"], a["wsb"], None)
    if fn == "fwd":
        return kla.lib().kla_glr_chunk_fwd(a["p"], FAKE, a["s"], FAKE, a["s"], *tail)
    if fn == "bwd":
        return kla.lib().kla_glr_chunk_bwd(a["p"], FAKE, a["s"], FAKE, a["s"], FAKE, FAKE, a["s"], *tail)
    return kla.lib().kla_glr_decode_step(a["p"], FAKE, a["s"], FAKE, a["N"], a["H"], a["d"], a["dtype"], None)


@pytest.mark.parametrize("fn", ["fwd", "bwd"])
@pytest.mark.parametrize("kw,status", [
    (dict(dtype=2), -3), (dict(dtype=-1), -3), (dict(B=-1), -2), (dict(H=0), -2), (dict(T=-1), -2), (dict(d=0), -2),
    (dict(d=(1 << 24) + 1), -2), (dict(N=3), -2), (dict(N=-1), -2), (dict(T=0x7fffffff), -2),
    (dict(H=1 << 20, B=1 << 12, N=1 << 12), -2), (dict(H=64, B=1 << 20, N=1 << 20, T=1), -2),
    (dict(H=1, B=1 << 24, N=1 << 24, T=1, d=1 << 10), -2), (dict(p=None), -1), (dict(p=FAKE + 8), -8), (dict(s=FAKE + 4), -8),
    (dict(cuh=[0, 100], N=1, B=1), -1), (dict(cu=FAKE, N=1, B=1), -1), (dict(cu=FAKE, cuh=[0, 50, 100], B=2), -2),
    (dict(cu=FAKE, cuh=[0, 50, 99], B=1), -5), (dict(cu=FAKE, cuh=[1, 50, 100], B=1), -5),
    (dict(cu=FAKE, cuh=[0, 101, 100], B=1), -5), (dict(cu=FAKE + 2, cuh=[0, 50, 100], B=1), -8),
    (dict(B=1, N=1, H=1, d=64, T=100000), -7), (dict(B=1, N=1, H=1, d=64, T=100000, ws=FAKE, wsb=16), -7),
    (dict(B=0, N=0), 0), (dict(B=0, N=0, T=100000), 0), (dict(cu=FAKE, cuh=[0], N=0, B=1, T=0), 0),
])
def test_refusals(fn, kw, status):
    assert call(fn, **kw) == status


@pytest.mark.parametrize("kw,status", [(dict(dtype=9), -3), (dict(N=-1), -2), (dict(H=0), -2), (dict(d=0), -2),
                                       (dict(p=None), -1), (dict(s=FAKE + 4), -8), (dict(N=0), 0),
                                       (dict(N=1 << 30, H=1, d=1 << 20), -2), (dict(N=1 << 30, H=1, d=33), -2),
                                       (dict(N=(1 << 30) + 1, H=1, d=5), -2)])
def test_step_refusals(kw, status):
    assert call("step", **kw) == status


def test_workspace_only_where_segments_are_used():
    assert kla.glr_chunk_workspace_bytes(4, 16, 4096, 128) == 0
    assert kla.glr_chunk_workspace_bytes(1, 1, 100, 64) == 0
    assert kla.glr_chunk_workspace_bytes(1, 1, 65536, 64) > 0
    assert kla.glr_chunk_workspace_bytes(1, 1, 65536, 0) == 0


def test_python_refuses_before_the_library():
    import torch
    x = torch.zeros(1, 1, 4, 8)
    with pytest.raises(ValueError):
        kla.glr_chunk_fwd(x, x)
    with pytest.raises(ValueError):
        kla.glr_decode_step(x[0], x[0], x[0])
    with pytest.raises(ValueError):
        kla.glr_chunk_bwd(x, x, x)
