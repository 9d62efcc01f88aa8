"""Linear attention with a decay per head on the GPU, against the fp64 oracle within its bounds
(oracle/la_oracle.py): a rounding to the element type of scores and states, fp32 sums, and half a
step of the output's type."""

import numpy as np
import pytest
import torch

from gated_delta_rule_kla_amd import kla
from oracle.la_oracle import la_backward, la_decode_step, la_forward

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a GPU")]

DEV = torch.device("cuda:0")
BF, F32 = torch.bfloat16, torch.float32
HALF = {BF: 2.0 ** -8, F32: 2.0 ** -24}  # half a step
U = {BF: 2.0 ** -8, F32: 0.0}            # of the factors that are rounded
DTYPES = [BF, F32]


def f64(t):
    return None if t is None else t.detach().cpu().to(torch.float64).numpy()


def packed(lens):
    host = torch.tensor(np.concatenate([[0], np.cumsum(lens)]), dtype=torch.int32)
    return host.to(DEV), host


def make(B, H, T, dk, dv, N, dtype, fixed=False, rate=0.1, seed=0):
    gen = torch.Generator().manual_seed(seed)
    q, k = (torch.randn(B, H, T, dk, generator=gen) * dk ** -0.25 for _ in "qk")
    v, do = (torch.randn(B, H, T, dv, generator=gen) for _ in "vo")
    if fixed:
        g = -rate * torch.rand(H, generator=gen)
    else:
        g = (-rate * torch.nn.functional.softplus(torch.randn(B, H, T, generator=gen))).to(dtype)
    s0, df = (torch.randn(N, H, dk, dv, generator=gen) for _ in "sd")
    return [x.to(dtype).to(DEV) for x in (q, k, v)] + [g.to(DEV), do.to(dtype).to(DEV), s0.to(DEV), df.to(DEV)]


def near(got, want, bound, dtype):
    got = f64(got)
    far = np.abs(got - want) - (bound + HALF[dtype] * (np.abs(want) + bound) + 1e-30)
    assert not np.isnan(far).any() and far.max(initial=-1.0) <= 0, (far.max(), np.abs(got - want).max())


def check(q, k, v, g, do, s0, df, cu=None, host=None, seqs=None):
    """Forward and backward against the oracle."""
    dtype = q.dtype
    u = U[dtype]
    o, S = kla.la_chunk_fwd(q, k, v, g, s0, cu, cu_seqlens_host=host)
    grads = kla.la_chunk_bwd(q, k, v, g, do, s0, df, cu, cu_seqlens_host=host)
    cu_np = None if host is None else host.numpy()
    wo, ws, eo, es = la_forward(f64(q), f64(k), f64(v), f64(g), f64(s0), cu_np, u)
    near(o, wo, eo, dtype)
    near(S, ws, es, F32)
    want, err = la_backward(f64(q), f64(k), f64(v), f64(g), f64(do), f64(s0), f64(df), cu_np, u)
    for x, w, e, t in zip(grads, want, err, (dtype, dtype, dtype, F32 if g.dim() == 1 else dtype, F32)):
        near(x, w, e, t)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("dk,dv", [(16, 16), (128, 128), (48, 80), (64, 256), (256, 64), (256, 256), (112, 144)])
def test_dense(dtype, dk, dv):
    check(*make(2, 2, 150, dk, dv, 2, dtype, seed=dk + dv))


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("fixed", [False, True])
def test_packed(dtype, fixed):
    lens = [1, 64, 0, 65, 63, 2, 128, 31, 33, 0, 200]
    cu, host = packed(lens)
    check(*make(1, 3, sum(lens), 64, 96, len(lens), dtype, fixed), cu, host)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("T", [1, 2, 31, 32, 33, 64, 65, 193])
def test_lengths_without_states(dtype, T):
    q, k, v, g, do, _, _ = make(1, 5, T, 32, 48, 1, dtype, seed=T)
    check(q, k, v, g, do, None, None)


@pytest.mark.parametrize("dtype", DTYPES)
def test_tokens_that_forget(dtype):
    """Decays of nothing, of a rounding's size and of all that came before, in the middle of
    chunks: what comes behind them is as exact as elsewhere."""
    q, k, v, g, do, s0, df = make(1, 2, 260, 64, 64, 1, dtype, rate=0.01, seed=3)
    g[0, 0, 7::9] = -float("inf")
    g[0, 1, 5::40] = -1000.0
    g[0, 1, 20::40] = -60.0
    g[0, :, 100:130] = 0.0
    check(q, k, v, g, do, s0, df)
    _, S = kla.la_chunk_fwd(q, k, v, g, s0)
    _, want, _, bound = la_forward(f64(q), f64(k), f64(v), f64(g), f64(s0), None, U[dtype])
    assert np.abs(f64(S) - want).max() <= 2e-5 * np.abs(want).max()


@pytest.mark.parametrize("dtype", DTYPES)
def test_values_that_are_not_finite_stay_in_their_sequence(dtype):
    lens = [70, 30, 100]
    cu, host = packed(lens)
    q, k, v, g, do, s0, df = make(1, 2, 200, 32, 32, 3, dtype, seed=4)
    o, S = kla.la_chunk_fwd(q, k, v, g, s0, cu, cu_seqlens_host=host)
    grads = kla.la_chunk_bwd(q, k, v, g, do, s0, df, cu, cu_seqlens_host=host)
    for x in (q, k, v, g, do):
        x[:, :, 70:100] = float("nan")
    s0[1] = float("inf")
    o2, S2 = kla.la_chunk_fwd(q, k, v, g, s0, cu, cu_seqlens_host=host)
    grads2 = kla.la_chunk_bwd(q, k, v, g, do, s0, df, cu, cu_seqlens_host=host)
    keep = list(range(70)) + list(range(100, 200))
    for a, b in zip((o, *grads[:4]), (o2, *grads2[:4])):
        assert torch.equal(a[:, :, keep], b[:, :, keep])
    for a, b in ((S, S2), (grads[4], grads2[4])):
        assert torch.equal(a[[0, 2]], b[[0, 2]])
    assert o2[:, :, 70:100].isnan().all()


@pytest.mark.parametrize("dtype", DTYPES)
def test_offsets_of_the_device_decide(dtype):
    """Other lengths than the host's, also longer ones, and a batch whose rows go on behind the
    last sequence: those stay as they were."""
    T = 300
    host = torch.tensor([0, 100, 200, T], dtype=torch.int32)
    real = [10, 15, 15, 290]
    cu = torch.tensor(real, dtype=torch.int32, device=DEV)
    q, k, v, g, do, s0, df = make(1, 2, T, 32, 48, 3, dtype, seed=5)
    for x in (q, k, v, do):
        x[:, :, :10], x[:, :, 290:] = float("nan"), float("nan")
    out = torch.full_like(v, 7.0)
    o, S = kla.la_chunk_fwd(q, k, v, g, s0, cu, cu_seqlens_host=host, out=out)
    assert (o[:, :, :10] == 7).all() and (o[:, :, 290:] == 7).all()
    grads = kla.la_chunk_bwd(q, k, v, g, do, s0, df, cu, cu_seqlens_host=host)
    cut = [x[:, :, 10:290].contiguous() for x in (q, k, v, g, do)]
    cu2, host2 = packed([5, 0, 275])
    o2, S2 = kla.la_chunk_fwd(*cut[:4], s0, cu2, cu_seqlens_host=host2)
    grads2 = kla.la_chunk_bwd(*cut, s0, df, cu2, cu_seqlens_host=host2)
    assert torch.equal(o[:, :, 10:290], o2) and torch.equal(S, S2)
    for a, b in zip(grads[:4], grads2[:4]):
        assert torch.equal(a[:, :, 10:290], b)
    assert torch.equal(grads[4], grads2[4])


def test_final_state_over_the_initial_one():
    q, k, v, g, _, s0, _ = make(2, 3, 130, 64, 64, 2, BF, seed=6)
    o, S = kla.la_chunk_fwd(q, k, v, g, s0)
    keep = s0.clone()
    o2, S2 = kla.la_chunk_fwd(q, k, v, g, keep, final_state=keep)
    assert S2 is keep and torch.equal(S, S2) and torch.equal(o, o2)


def test_nothing_to_do():
    q, k, v, g, do, s0, df = make(2, 2, 0, 32, 32, 2, BF)
    o, S = kla.la_chunk_fwd(q, k, v, g, s0)
    assert o.shape == (2, 2, 0, 32) and torch.equal(S, s0)
    grads = kla.la_chunk_bwd(q, k, v, g, do, s0, df)
    assert torch.equal(grads[4], df)
    fixed = torch.tensor([-0.1, -0.2], device=DEV)
    assert not kla.la_chunk_bwd(q, k, v, fixed, do, s0, df)[3].any()
    q, k, v, g, do, s0, df = make(0, 2, 5, 32, 32, 0, BF)
    assert kla.la_chunk_fwd(q, k, v, g, s0)[1].shape == (0, 2, 32, 32)
    assert not kla.la_chunk_bwd(q, k, v, fixed, do, s0, df)[3].any()


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("N,H,dk,dv,fixed", [(1, 1, 16, 16, False), (3, 2, 128, 128, False), (5, 3, 48, 80, True),
                                              (200, 4, 256, 144, False), (300, 2, 64, 256, True), (2, 2, 256, 16, True)])
def test_step(dtype, N, H, dk, dv, fixed):
    gen = torch.Generator().manual_seed(N)
    q, k = (torch.randn(N, H, dk, generator=gen).to(dtype).to(DEV) for _ in "qk")
    v = torch.randn(N, H, dv, generator=gen).to(dtype).to(DEV)
    g = -torch.rand(*((H,) if fixed else (N, H)), generator=gen)
    g.view(-1)[0] = -float("inf")
    g = g.to(F32 if fixed else dtype).to(DEV)
    S = torch.randn(N, H, dk, dv, generator=gen).to(DEV)
    wo, ws = la_decode_step(f64(q), f64(k), f64(v), f64(g), f64(S))
    mag = la_decode_step(*(np.abs(f64(x)) for x in (q, k, v)), f64(g), np.abs(f64(S)))
    o = kla.la_decode_step(q, k, v, g, S)
    near(S, ws, 8 * 2.0 ** -24 * mag[1], F32)
    near(o, wo, (dk + 8) * 2.0 ** -24 * mag[0], dtype)


@pytest.mark.parametrize("dtype", DTYPES)
def test_steps_continue_a_prompt(dtype):
    q, k, v, g, _, s0, _ = make(2, 3, 100, 64, 64, 2, dtype, seed=8)
    _, S = kla.la_chunk_fwd(q, k, v, g, s0)
    part = [x[:, :, :90].contiguous() for x in (q, k, v, g)]
    _, state = kla.la_chunk_fwd(*part, s0)
    wo, _, eo, es = la_forward(*(f64(x) for x in (q, k, v, g, s0)), None, U[dtype])
    for t in range(90, 100):
        o = kla.la_decode_step(*(x[:, :, t].contiguous() for x in (q, k, v, g)), state)
        near(o, wo[:, :, t], eo[:, :, t], dtype)
    near(state, f64(S), 2 * es, F32)


@pytest.mark.parametrize("dtype", DTYPES)
def test_captured_and_replayed_on_another_stream(dtype):
    """Forward, backward and a step in one graph, replayed with other inputs and other lengths,
    with eager calls between."""
    host = torch.tensor([0, 90, 200], dtype=torch.int32)
    cu = host.to(DEV)
    x = make(1, 2, 200, 64, 64, 2, dtype, seed=9)
    one = [t[:, :, 0].contiguous() for t in x[:4]]
    state = torch.zeros(1, 2, 64, 64, device=DEV)

    def run():
        a = kla.la_chunk_fwd(*x[:4], x[5], cu, cu_seqlens_host=host)
        b = kla.la_chunk_bwd(*x[:5], x[5], x[6], cu, cu_seqlens_host=host)
        return (*a, *b, kla.la_decode_step(*one, state))

    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        run()
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        got = run()
    for i in range(3):
        for t, s in zip(x, make(1, 2, 200, 64, 64, 2, dtype, seed=20 + i)):
            t.copy_(s)
        cu.copy_(torch.tensor([0, [90, 1, 0][i], [200, 200, 150][i]], dtype=torch.int32))
        for t in got[:6]:
            t.zero_()
        state.fill_(i)
        graph.replay()
        torch.cuda.synchronize()
        have = [t.clone() for t in got]
        after = state.clone()
        state.fill_(i)
        for a, b in zip(have, run()):
            if a.shape[-1] == 200 or a.dim() == 4 and a.shape[2] == 200:
                a, b = a[:, :, :int(cu[-1])], b[:, :, :int(cu[-1])]
            assert torch.equal(a, b)
        assert torch.equal(state, after)


def test_the_same_bits_again():
    lens = [500, 3, 200, 900]
    cu, host = packed(lens)
    x = make(1, 4, sum(lens), 128, 128, 4, BF, seed=10)
    first = [*kla.la_chunk_fwd(*x[:4], x[5], cu, cu_seqlens_host=host), *kla.la_chunk_bwd(*x[:5], x[5], x[6], cu, cu_seqlens_host=host)]
    for _ in range(3):
        again = [*kla.la_chunk_fwd(*x[:4], x[5], cu, cu_seqlens_host=host), *kla.la_chunk_bwd(*x[:5], x[5], x[6], cu, cu_seqlens_host=host)]
        assert all(torch.equal(a, b) for a, b in zip(first, again))


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("fixed", [False, True])
def test_few_long_sequences(dtype, fixed):
    """Sequences in segments that are scanned side by side, beside shorter ones and an empty one."""
    lens = [2500, 0, 3, 1100, 700]
    cu, host = packed(lens)
    check(*make(1, 1, sum(lens), 64, 48, len(lens), dtype, fixed, rate=0.02, seed=11), cu, host)


@pytest.mark.parametrize("dtype", DTYPES)
def test_segments_over_the_initial_state(dtype):
    q, k, v, g, _, s0, _ = make(1, 2, 4100, 32, 32, 1, dtype, rate=0.001, seed=12)
    o, S = kla.la_chunk_fwd(q, k, v, g, s0)
    for _ in range(3):
        keep = s0.clone()
        o2, S2 = kla.la_chunk_fwd(q, k, v, g, keep, final_state=keep)
        assert torch.equal(S, S2) and torch.equal(o, o2)
    wo, ws, eo, es = la_forward(f64(q), f64(k), f64(v), f64(g), f64(s0), None, U[dtype])
    near(o, wo, eo, dtype)
    near(S, ws, es, F32)


@pytest.mark.parametrize("dtype", DTYPES)
def test_segments_of_other_lengths_on_the_device(dtype):
    """A call cut for even sequences, replayed with one that is longer than any of them."""
    T = 4000
    host = torch.tensor([0, 2000, T], dtype=torch.int32)
    q, k, v, g, do, s0, df = make(1, 1, T, 32, 32, 2, dtype, rate=0.02, seed=13)
    for real in ([0, 100, 3900], [0, 3990, 4000]):
        cu = torch.tensor(real, dtype=torch.int32, device=DEV)
        o, S = kla.la_chunk_fwd(q, k, v, g, s0, cu, cu_seqlens_host=host)
        grads = kla.la_chunk_bwd(q, k, v, g, do, s0, df, cu, cu_seqlens_host=host)
        n = real[-1]
        cut = [f64(x[:, :, :n]) for x in (q, k, v, g)]
        wo, ws, eo, es = la_forward(*cut, f64(s0), real, U[dtype])
        near(o[:, :, :n], wo, eo, dtype)
        near(S, ws, es, F32)
        want, err = la_backward(*cut, f64(do[:, :, :n]), f64(s0), f64(df), real, U[dtype])
        for i in range(4):
            near(grads[i][:, :, :n], want[i], err[i], dtype)
        near(grads[4], want[4], err[4], F32)
