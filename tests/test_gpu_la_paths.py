"""Linear attention's instantiations that few shapes reach, on the GPU against the fp64 oracle, and
the 24 bits of its final state."""

import numpy as np
import pytest
import torch

from gated_delta_rule_kla_amd import kla
from test_gpu_la import BF, DEV, check, f64, make

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a GPU")]


@pytest.mark.parametrize("dk,dv,fixed,rate", [(80, 48, False, 0.02), (16, 48, True, 0.02), (32, 64, False, 0.002)])
def test_backward_of_wide_slices_in_segments(dk, dv, fixed, rate):
    """Slices of 64 columns in the pass over the segments' ends, in both directions: bf16, dk up to
    128, dv over 32, and 256 workgroups and more."""
    H, T = 32, 2100
    slices32, slices64, chunks = -(-dv // 32), -(-dv // 64), -(-T // 64)
    segments = min(512 // (H * slices32), chunks // 8)
    assert H * slices32 <= 128 and chunks >= 32 and segments > 1 and 2 * H * segments * slices64 >= 256
    # more than the gradients' fixed buffers: the segments' states are there
    states = segments * H * dk * dv * 4
    assert kla.la_chunk_workspace_bytes(1, H, T, dk, dv) >= states
    check(*make(1, H, T, dk, dv, 1, BF, fixed, rate=rate, seed=dk + dv))


@pytest.mark.parametrize("T", [2, 17, 64, 130, 200])
@pytest.mark.parametrize("place", [0, 1])
def test_the_final_state_has_24_bits(T, place):
    """One token writes and the others only decay: a state is one product, and what its bf16
    factors, the decay and fp32 make of it is known.  Relative to the state: the decay's exponent
    (at most 1 in base two) rounded, 2^-24, and the hardware's exponential, 2^-23, once for the
    token's chunk and once for each of three chunks behind it; the value times its decay, 2^-24,
    in three bf16 terms, 2^-24; three additions and a product for each chunk, 2^-24 each.  In all
    less than 2^-20; two terms would be off by up to 2^-16."""
    H, dk, dv = 3, 64, 96
    gen = torch.Generator().manual_seed(T)
    q, k = (torch.randn(1, H, T, dk, generator=gen).to(BF).to(DEV) for _ in "qk")
    v = torch.zeros(1, H, T, dv)
    v[:, :, place] = torch.randn(1, H, dv, generator=gen)
    v = v.to(BF).to(DEV)
    g = -0.69 * torch.rand(1, H, T, generator=gen).to(DEV) / T
    g = g.to(BF)
    _, S = kla.la_chunk_fwd(q, k, v, g)
    decay = np.exp(f64(g)[0, :, place + 1:].sum(1))
    want = decay[:, None, None] * f64(k)[0, :, place, :, None] * f64(v)[0, :, place, None, :]
    assert decay.min() > 0.5 and (np.abs(f64(S)[0] - want) <= 2.0 ** -20 * np.abs(want) + 1e-30).all()
