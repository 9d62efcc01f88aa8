"""The gated linear recurrence on the GPU against its fp64 oracle.

Tolerance: the oracle's own bound on fp32 arithmetic (oracle/glr_oracle.py), plus half a step of
the output's type."""

import numpy as np
import pytest
import torch

from gated_delta_rule_kla_amd import kla
from oracle.glr_oracle import glr_backward, glr_forward

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a GPU")]

DEV = torch.device("cuda:0")
HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}
BF, F32 = torch.bfloat16, torch.float32


def f64(t):
    return None if t is None else t.detach().cpu().to(torch.float64).numpy()


def near(got, ref, bound, dtype, what):
    got = f64(got)
    off = np.abs(got - ref) - (bound + HALF[dtype] * (np.abs(ref) + bound) + 1e-37)
    assert np.isfinite(got).all(), what
    assert got.shape == ref.shape and (off <= 0).all(), (what, float(off.max()))


def inputs(dtype, B, H, T, d, cu=None, seed=0, slow=1.0):
    gen = torch.Generator().manual_seed(seed)
    x = torch.randn(B, H, T, d, generator=gen).to(dtype)
    g = (-slow * torch.nn.functional.softplus(torch.randn(B, H, T, d, generator=gen))).to(dtype)
    N = B if cu is None else len(cu) - 1
    return x, g, torch.randn(N, H, d, generator=gen), torch.randn(B, H, T, d, generator=gen).to(dtype), \
        torch.randn(N, H, d, generator=gen)


def cu_of(cu):
    return (None, None) if cu is None else (torch.tensor(cu, dtype=torch.int32, device=DEV),
                                            torch.tensor(cu, dtype=torch.int32))


def check(dtype, B, H, T, d, cu=None, seed=0, slow=0.3, states=True):
    x, g, h0, do, df = inputs(dtype, B, H, T, d, cu, seed, slow)
    if not states:
        h0 = df = None
    dev, host = cu_of(cu)
    put = lambda t: None if t is None else t.to(DEV)  # noqa: E731
    o, hf = kla.glr_chunk_fwd(put(x), put(g), put(h0), dev, cu_seqlens_host=host)
    want, wf, eo, ef = glr_forward(f64(x), f64(g), f64(h0), cu)
    near(o, want, eo, dtype, "o")
    near(hf, wf, ef, F32, "final state")
    dx, dg, d0 = kla.glr_chunk_bwd(put(g), o, put(do), put(h0), put(df), dev, cu_seqlens_host=host)
    rx, rg, r0, ex, eg, e0 = glr_backward(f64(g), f64(o), f64(do), f64(h0), f64(df), cu)
    near(dx, rx, ex, dtype, "dx")
    near(dg, rg, eg, dtype, "dg")
    near(d0, r0, e0, F32, "dh0")


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("B,H,T,d", [
    (1, 1, 1, 1), (1, 1, 1, 128), (2, 3, 5, 8), (1, 2, 63, 16), (3, 1, 64, 36), (1, 1, 257, 100), (2, 2, 300, 7),
    (1, 1, 1000, 2560), (2, 5, 513, 128), (1, 16, 300, 250)])
def test_dense(dtype, B, H, T, d):
    check(dtype, B, H, T, d, seed=T + d)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("d", [64, 20, 3])
def test_packed(dtype, d):
    check(dtype, 1, 2, 700, d, cu=[0, 0, 1, 130, 130, 131, 387, 700, 700], seed=d)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("d,cu", [(16, None), (5, None), (64, [0, 1500, 1500, 1501, 5200])])
def test_long_with_few_channels(dtype, d, cu):
    """Cut into segments."""
    assert kla.glr_chunk_workspace_bytes(1, 1, 5200, d, dtype,
                                         None if cu is None else torch.tensor(cu, dtype=torch.int32)) > 0
    check(dtype, 1, 1, 5200, d, cu, seed=d, slow=0.02)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("B,H,T,cu,lines", [(4, 64, 600, None, 1), (2, 64, 1100, None, 2),
                                            (1, 64, 3500, [0, 0, 700, 701, 1000, 1020, 1600, 1620, 2900, 2990, 3500], 1)])
def test_whole_lines(dtype, B, H, T, cu, lines):
    """Many heads of one or two 128-byte lines; packed, the longest sequences start first."""
    check(dtype, B, H, T, lines * (64 if dtype == BF else 32), cu, seed=T, slow=0.05)


def test_order_of_other_lengths():
    """The launch's order is the host's lengths'; a replayed graph may hold others."""
    x, g, h0, *_ = (t.to(DEV) for t in inputs(BF, 1, 64, 3000, 64, [0, 1, 2], seed=11))
    h0 = h0[:1].expand(10, 64, 64).contiguous()
    host = torch.arange(0, 3001, 300, dtype=torch.int32)
    cu = torch.tensor([0, 10, 900, 901, 1500, 1500, 1600, 2000, 2900, 2950, 3000], dtype=torch.int32)
    want = kla.glr_chunk_fwd(x, g, h0, cu.to(DEV), cu_seqlens_host=cu)
    got = kla.glr_chunk_fwd(x, g, h0, cu.to(DEV), cu_seqlens_host=host)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


@pytest.mark.parametrize("T", [4, 3000])
def test_without_states(T):
    check(F32, 1, 1, T, 16, states=False)


def test_many_sequences():
    cu = [0]
    for n in range(400):
        cu.append(cu[-1] + n % 7)
    check(BF, 1, 1, cu[-1], 24, cu=cu, seed=2)


def test_closed_gates():
    x, g, h0, do, df = inputs(F32, 1, 2, 200, 8)
    g[:, :, [0, 17, 18, 140, 199]] = -float("inf")
    o, hf = kla.glr_chunk_fwd(x.to(DEV), g.to(DEV), h0.to(DEV))
    want, wf, eo, ef = glr_forward(f64(x), f64(g), f64(h0))
    near(o, want, np.nan_to_num(eo), F32, "o")
    dx, dg, d0 = kla.glr_chunk_bwd(g.to(DEV), o, do.to(DEV), h0.to(DEV), df.to(DEV))
    assert torch.equal(d0, torch.zeros_like(d0))
    assert torch.equal(dg[:, :, [0, 17, 18, 140, 199]], torch.zeros_like(dg[:, :, :5]))


@pytest.mark.parametrize("T", [200, 3000])
def test_nan_stays_in_its_channel_and_sequence(T):
    x, g, h0, *_ = inputs(BF, 2, 1, T, 16)
    clean, _ = kla.glr_chunk_fwd(x.to(DEV), g.to(DEV), h0.to(DEV))
    x[0, 0, 50, 3] = float("nan")
    o, hf = kla.glr_chunk_fwd(x.to(DEV), g.to(DEV), h0.to(DEV))
    bad = torch.isnan(o)
    assert bad[0, 0, 50:, 3].all() and int(bad.sum()) == T - 50
    assert torch.equal(o[~bad], clean[~bad])


@pytest.mark.parametrize("T,d", [(300, 128), (5000, 32)])
def test_state_in_place_repeats_bit_for_bit(T, d):
    x, g, h0, do, df = (t.to(DEV) for t in inputs(BF, 1, 1, T, d))
    o, hf = kla.glr_chunk_fwd(x, g, h0)
    state = h0.clone()
    for _ in range(3):
        state.copy_(h0)
        o2, same = kla.glr_chunk_fwd(x, g, state, final_state=state)
        assert same is state and torch.equal(state, hf) and torch.equal(o, o2)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("N,H,d", [(1, 1, 1), (3, 5, 7), (2, 16, 128), (300, 3, 60)])
def test_step(dtype, N, H, d):
    x, g, h0, *_ = inputs(dtype, 1, N, H, d)
    x, g, h0 = x[0], g[0], torch.randn(N, H, d)
    state = h0.to(DEV)
    o = kla.glr_decode_step(x.to(DEV), g.to(DEV), state)
    want = np.exp(f64(g)) * f64(h0) + f64(x)
    bound = 8 * 2.0 ** -24 * (np.abs(f64(h0)) * (1 + np.abs(f64(g))) + np.abs(f64(x)))
    near(state, want, bound, F32, "state")
    near(o, want, bound, dtype, "o")


def test_prompt_then_steps():
    x, g, h0, *_ = inputs(F32, 2, 3, 40, 24)
    want, wf, eo, ef = glr_forward(f64(x), f64(g), f64(h0))
    x, g = x.to(DEV), g.to(DEV)
    o, state = kla.glr_chunk_fwd(x[:, :, :30].contiguous(), g[:, :, :30].contiguous(), h0.to(DEV))
    near(o, want[:, :, :30], eo[:, :, :30], F32, "prompt")
    for t in range(30, 40):
        near(kla.glr_decode_step(x[:, :, t].contiguous(), g[:, :, t].contiguous(), state), want[:, :, t], eo[:, :, t],
             F32, f"step {t}")


def test_gradients_against_differences():
    """Along random directions, of a loss of all outputs, in fp32 on the GPU's own forward."""
    x, g, h0, do, df = (t.to(DEV) for t in inputs(F32, 1, 2, 130, 8, seed=4))
    o, _ = kla.glr_chunk_fwd(x, g, h0)
    grads = kla.glr_chunk_bwd(g, o, do, h0, df)
    s = 2.0 ** -6
    for k in range(3):
        u = torch.randn_like((x, g, h0)[k])
        two = []
        for sign in (1, -1):
            a = [x, g, h0]
            a[k] = a[k] + sign * s * u
            oo, hh = kla.glr_chunk_fwd(*a)
            two.append(float((oo.double() * do).sum() + (hh.double() * df).sum()))
        slope = (two[0] - two[1]) / (2 * s)
        along = float((grads[k].double() * u).sum())
        # the difference's own error: s^2/6 of the third derivative (zero for x and h0, which
        # enter linearly; up to a few units for g), and 2^-24 of the summed magnitudes over 2 s
        size = float((o.double() * do).abs().sum())
        assert abs(slope - along) <= size * 2.0 ** -20 / (2 * s) + (s * s * size if k == 1 else 0), (k, slope, along)


def test_another_stream_and_a_graph():
    x, g, h0, do, df = (t.to(DEV) for t in inputs(BF, 1, 1, 3000, 64))
    o, hf = kla.glr_chunk_fwd(x, g, h0)
    want = kla.glr_chunk_bwd(g, o, do, h0, df)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        o2, hf2 = kla.glr_chunk_fwd(x, g, h0)
        got = kla.glr_chunk_bwd(g, o2, do, h0, df)
    side.synchronize()
    assert torch.equal(o, o2) and torch.equal(hf, hf2) and all(torch.equal(a, b) for a, b in zip(want, got))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o3, hf3 = kla.glr_chunk_fwd(x, g, h0)
        g3 = kla.glr_chunk_bwd(g, o3, do, h0, df)
    for k in range(3):
        x.mul_(0.5)
        graph.replay()
        torch.cuda.synchronize()
        o4, hf4 = kla.glr_chunk_fwd(x, g, h0)
        g4 = kla.glr_chunk_bwd(g, o4, do, h0, df)
        torch.cuda.synchronize()
        assert torch.equal(o3, o4) and torch.equal(hf3, hf4) and all(torch.equal(a, b) for a, b in zip(g3, g4))


def test_refusals():
    x = torch.zeros(2, 3, 4, 8, device=DEV)
    with pytest.raises(ValueError):
        kla.glr_chunk_fwd(x.transpose(1, 2), x.transpose(1, 2))
    with pytest.raises(TypeError):
        kla.glr_chunk_fwd(x, x.bfloat16())
    with pytest.raises(TypeError):
        kla.glr_chunk_fwd(x.half(), x.half())
    with pytest.raises(ValueError):
        kla.glr_chunk_fwd(x, x, torch.zeros(2, 3, 9, device=DEV))
    with pytest.raises(ValueError):
        kla.glr_chunk_fwd(x[0], x[0])
    with pytest.raises(kla.KlaError):
        kla.glr_chunk_fwd(x, x, cu_seqlens=torch.tensor([0, 2, 4], dtype=torch.int32, device=DEV))
    with pytest.raises(ValueError):
        kla.glr_decode_step(x[0], x[0], torch.zeros(3, 4, 9, device=DEV))
