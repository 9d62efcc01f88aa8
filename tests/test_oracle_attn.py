"""The attention oracle and the 4-bit format's, pinned without their own formulas, and the
arguments that kla_kv4_* and kla_attn_kv4_decode_step refuse (on the host, before any HIP call)."""

import ctypes
import math
import os

import numpy as np
import pytest

from gated_delta_rule_kla_amd import kla
from oracle.attn_oracle import E2M1, attend, quantise, values

RNG = np.random.default_rng


def test_equal_keys_average_the_values():
    q, v = RNG(0).normal(size=(3, 8)), RNG(1).normal(size=(5, 8))
    mask = np.array([[1, 1, 1, 1, 1], [1, 0, 0, 1, 0], [0, 0, 0, 0, 0]], bool)
    o, lse, *_ = attend(q, np.ones((5, 8)), v, 0.3, mask, 0)
    np.testing.assert_allclose(o[0], v.mean(0), rtol=1e-13)
    np.testing.assert_allclose(o[1], v[[0, 3]].mean(0), rtol=1e-13)
    assert not o[2].any() and lse[2] == -np.inf
    np.testing.assert_allclose(lse[1], 0.3 * q[1].sum() + math.log(2), rtol=1e-13)


def test_a_far_key_wins_and_shifts_do_not_matter():
    q, k, v = RNG(0).normal(size=(2, 4)), RNG(1).normal(size=(6, 4)), RNG(2).normal(size=(6, 4))
    far = k.copy()
    far[3] = 1e4 * q[0] / (q[0] @ q[0])
    o, *_ = attend(q[:1], far, v, 1.0, np.ones((1, 6), bool), 0)
    np.testing.assert_array_equal(o[0], v[3])
    a, la, *_ = attend(q, k, v, 1.0, np.ones((2, 6), bool), 0)
    b, lb, *_ = attend(q, k + 100.0, v, 1.0, np.ones((2, 6), bool), 0)
    np.testing.assert_allclose(a, b, rtol=1e-9, atol=1e-11)
    np.testing.assert_allclose(lb - la, 100.0 * q.sum(1), rtol=1e-9)


def test_a_run_of_keys_joins_another():
    q, k, v = RNG(0).normal(size=(2, 4)), RNG(1).normal(size=(9, 4)), RNG(2).normal(size=(9, 4))
    one = np.ones((2, 9), bool)
    o, lse, *_ = attend(q, k, v, 0.5, one, 0)
    parts = [attend(q, k[s], v[s], 0.5, one[:, s], 0)[:2] for s in (slice(0, 4), slice(4, 9))]
    w = [np.exp(p[1] - lse)[:, None] for p in parts]
    np.testing.assert_allclose(w[0] * parts[0][0] + w[1] * parts[1][0], o, rtol=1e-12)


def test_the_bound_covers_fp32():
    q, k, v = (RNG(i).normal(size=(64, 64)).astype(np.float32) for i in range(3))
    o, lse, eo, el = attend(*(t.astype(np.float64) for t in (q, k, v)), 0.125, np.ones((64, 64), bool), 0)
    s = (q @ k.T) * np.float32(0.125)
    p = np.exp(s - s.max(1, keepdims=True))
    got = (p @ v) / p.sum(1, keepdims=True)
    assert (np.abs(got - o) <= eo).all() and eo.max() < 3e-4
    assert (np.abs(s.max(1) + np.log(p.sum(1)) - lse) <= el).all()


def test_every_code_stands_for_itself():
    x = np.concatenate([E2M1, -E2M1, E2M1, -E2M1])
    for e in (-126, -20, 0, 31):
        codes, scales = quantise(x * 2.0 ** e)
        assert scales[0] == e + 127
        np.testing.assert_array_equal(values(codes, scales), x * 2.0 ** e)


def test_rounding_of_values_between():
    x = np.zeros(32)
    x[0] = 4.0
    mids = [0.25, 0.75, 1.25, 1.75, 2.5, 3.5]
    x[1:7], x[7:13] = mids, np.negative(mids)
    x[13], x[14], x[15] = 0.2500001, 0.2499999, 5.0
    got = values(*quantise(x))
    np.testing.assert_array_equal(got[1:7], [0, 1, 1, 2, 2, 4])
    np.testing.assert_array_equal(got[7:13], [0, -1, -1, -2, -2, -4])
    np.testing.assert_array_equal(got[13:16], [0.5, 0.0, 4.0])
    x[0] = 7.9
    assert values(*quantise(x))[0] == 6.0
    assert (quantise(np.zeros(32))[1] == 1).all()


# ---- refusals --------------------------------------------------------------------------------

FAKE = 0x7F0000000000  # never dereferenced
built = pytest.mark.skipif(not os.path.exists(kla.lib_path()), reason="libkla.so not built")


def move(fn, **kw):
    a = dict(k=FAKE, codes=FAKE, scales=FAKE, table=FAKE, start=FAKE, cu=None, cuh=None, N=2, B=2, Hkv=4, T=10, D=128,
             P=8, page=16, M=2, dtype=0)
    a.update(kw)
    cuh = None if a["cuh"] is None else (ctypes.c_int32 * len(a["cuh"]))(*a["cuh"])
    return getattr(kla.lib(), fn)(a["k"], FAKE, a["codes"], a["scales"], a["table"], a["start"], a["cu"],
                                  None if cuh is None else ctypes.addressof(cuh), a["N"], a["B"], a["Hkv"], a["T"],
                                  a["D"], a["P"], a["page"], a["M"], a["dtype"], None)


@built
@pytest.mark.parametrize("fn", ["kla_kv4_append", "kla_kv4_read"])
@pytest.mark.parametrize("kw,status", [
    (dict(dtype=5), -3), (dict(B=-1, N=-1), -2), (dict(Hkv=0), -2), (dict(T=-1), -2), (dict(P=0), -2),
    (dict(page=0), -2), (dict(M=0), -2), (dict(N=3), -2), (dict(D=96), -4), (dict(page=24), -4),
    (dict(page=1 << 21), -4), (dict(T=0x7fffffff), -2), (dict(T=1 << 28, Hkv=4), -2),
    (dict(T=(1 << 28) - 1, Hkv=4), -2), (dict(k=None), -1),
    (dict(codes=None), -1), (dict(start=None), -1), (dict(table=FAKE + 2), -8), (dict(scales=FAKE + 8), -8),
    (dict(start=FAKE + 1), -8),
    (dict(cu=FAKE, cuh=[0, 4, 9], B=1), -5), (dict(cu=FAKE, cuh=[0, 11, 10], B=1), -5), (dict(cu=FAKE, B=1), -1),
    (dict(cuh=[0, 4, 10]), -1), (dict(T=0, k=None), 0), (dict(B=0, N=0), 0),
])
def test_move_refusals(fn, kw, status):
    assert move(fn, **kw) == status


def decode(**kw):
    a = dict(q=FAKE, codes=FAKE, lens=FAKE, scale=0.1, N=2, Hq=8, Hkv=4, D=128, P=8, page=16, M=4, ml=64, dtype=0,
             ws=None, wsb=0)
    a.update(kw)
    return kla.lib().kla_attn_kv4_decode_step(a["q"], a["codes"], FAKE, FAKE, a["lens"], a["scale"], FAKE, a["N"],
                                              a["Hq"], a["Hkv"], a["D"], a["P"], a["page"], a["M"], a["ml"],
                                              a["dtype"], a["ws"], a["wsb"], None)


@built
@pytest.mark.parametrize("kw,status", [
    (dict(dtype=5), -3), (dict(N=-1), -2), (dict(Hq=7), -2), (dict(Hq=0), -2), (dict(ml=-1), -2),
    (dict(ml=0x7fffffff), -2), (dict(D=32), -4), (dict(page=8), -4), (dict(scale=float("nan")), -11),
    (dict(scale=float("inf")), -11), (dict(q=None), -1), (dict(lens=None), -1), (dict(q=FAKE + 2), -8), (dict(lens=FAKE + 2), -8),
    (dict(ml=100000, M=10000), -7), (dict(ml=100000, M=10000, ws=FAKE, wsb=100), -7),
    (dict(N=1 << 20, Hq=1 << 14, Hkv=1 << 13), -2), (dict(N=1 << 20, Hq=16, Hkv=16), -2), (dict(N=0, q=None), 0),
])
def test_decode_refusals(kw, status):
    assert decode(**kw) == status


@built
def test_decode_workspace():
    assert kla.attn_kv4_decode_workspace_bytes(256, 16, 4, 128, 4096) == 0
    one = kla.attn_kv4_decode_workspace_bytes(1, 16, 2, 128, 131072)
    assert one > 0 and one % (16 * 130 * 4) == 0
    assert kla.attn_kv4_decode_workspace_bytes(1, 15, 2, 128, 131072) == 0


def attn(**kw):
    a = dict(q=FAKE, k=FAKE, lse=FAKE, scale=0.1, cu=None, cuh=None, ck=None, ckh=None, N=2, B=2, Hq=8, Hkv=4, Tq=10,
             Tk=10, D=128, dtype=0)
    a.update(kw)
    host = [None if x is None else (ctypes.c_int32 * len(x))(*x) for x in (a["cuh"], a["ckh"])]
    at = [None if x is None else ctypes.addressof(x) for x in host]
    return kla.lib().kla_attn_fwd(a["q"], a["k"], FAKE, a["scale"], FAKE, a["lse"], a["cu"], at[0], a["ck"], at[1],
                                  a["N"], a["B"], a["Hq"], a["Hkv"], a["Tq"], a["Tk"], a["D"], a["dtype"], None)


@built
@pytest.mark.parametrize("kw,status", [
    (dict(dtype=2), -3), (dict(B=-1, N=-1), -2), (dict(Hq=6), -2), (dict(Hkv=0), -2), (dict(Tq=-1), -2),
    (dict(Tk=-1), -2), (dict(Tk=0x7fffffff), -2), (dict(N=3), -2), (dict(D=0), -2), (dict(D=80), -4),
    (dict(B=1 << 20, N=1 << 20, Hq=1 << 12), -2), (dict(B=1 << 15, N=1 << 15, Hq=1 << 15, Tq=1 << 20), -2),
    (dict(B=1 << 18, N=1 << 18, Hq=32), -2), (dict(scale=float("nan")), -11), (dict(q=None), -1), (dict(k=None), -1),
    (dict(q=FAKE + 8), -8), (dict(lse=FAKE + 4), -8), (dict(cu=FAKE, cuh=[0, 4, 10]), -2), (dict(cu=FAKE, cuh=[0, 4, 9], B=1), -5),
    (dict(cu=FAKE, cuh=[0, 4, 10], B=1, Tk=11), -2), (dict(cu=FAKE, cuh=[0, 4, 10], ck=FAKE, B=1), -1),
    (dict(cu=FAKE, cuh=[0, 4, 10], ck=FAKE, ckh=[0, 4, 11], B=1), -5), (dict(ck=FAKE, ckh=[0, 4, 10]), -1),
    (dict(cu=FAKE, cuh=[0, 4, 10], ck=FAKE + 2, ckh=[0, 4, 10], B=1), -8), (dict(Tq=0, q=None), 0),
    (dict(B=0, N=0), 0),
])
def test_attn_refusals(kw, status):
    assert attn(**kw) == status
