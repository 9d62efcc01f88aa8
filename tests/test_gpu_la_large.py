"""Linear attention where there are enough workgroups for slices of 64 columns, and over batches
of many sequences, on the GPU against the fp64 oracle within its bounds."""

import pytest
import torch

from gated_delta_rule_kla_amd import kla
from oracle.la_oracle import la_forward
from test_gpu_la import BF, DEV, F32, U, check, f64, make, near, packed

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a GPU")]


@pytest.mark.parametrize("dk,dv", [(64, 48), (64, 256), (128, 80), (128, 112), (96, 256)])
def test_wide_slices(dk, dv):
    """256 workgroups and more of 64 columns, the last slice of 16 to 64."""
    H = 256 // -(-dv // 64) + 1
    q, k, v, g, _, s0, _ = make(1, H, 140, dk, dv, 1, BF, seed=dk + dv)
    o, S = kla.la_chunk_fwd(q, k, v, g, s0)
    wo, ws, eo, es = la_forward(f64(q), f64(k), f64(v), f64(g), f64(s0), None, U[BF])
    near(o, wo, eo, BF)
    near(S, ws, es, F32)


@pytest.mark.parametrize("fixed", [False, True])
def test_wide_slices_in_segments(fixed):
    """A long sequence, whose segments make the workgroups."""
    q, k, v, g, _, s0, _ = make(1, 8, 8200, 64, 128, 1, BF, fixed=fixed, rate=0.01, seed=6)
    o, S = kla.la_chunk_fwd(q, k, v, g, s0)
    wo, ws, eo, es = la_forward(f64(q), f64(k), f64(v), f64(g), f64(s0), None, U[BF])
    near(o, wo, eo, BF)
    near(S, ws, es, F32)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_many_short_sequences(dtype):
    lens = [n % 5 + (70 if n % 50 == 7 else 0) for n in range(300)]
    cu, host = packed(lens)
    check(*make(1, 2, sum(lens), 32, 48, len(lens), dtype, seed=7), cu, host)


@pytest.mark.parametrize("big", [1e-20, 1e25])
def test_states_far_from_one(big):
    """The backward's states are kept with a power of two of their own: values of any size, and
    parts of a state that are smaller than others by 2^20."""
    q, k, v, g, do, s0, df = make(1, 2, 200, 64, 96, 1, BF, rate=0.05, seed=8)
    v, s0 = v * big, s0 * big
    v[..., :32] *= 2.0 ** -20
    s0[..., :32] *= 2.0 ** -20
    check(q, k, v, g, do, s0, df)


def test_infinite_parts_of_a_state():
    """Channels of a state that are infinite leave the gradients of the others' keys alone."""
    q, k, v, g, do, s0, df = make(1, 1, 130, 64, 64, 1, BF, seed=9)
    clean = kla.la_chunk_bwd(q, k, v, g, do, s0, df)
    s0[0, 0, 5, 7] = float("inf")
    got = kla.la_chunk_bwd(q, k, v, g, do, s0, df)
    rest = [i for i in range(64) if i != 5]
    assert not got[0][..., 5].isfinite().all()
    assert torch.equal(got[0][..., rest], clean[0][..., rest])
    for i in (1, 2, 4):
        assert torch.equal(got[i], clean[i])
