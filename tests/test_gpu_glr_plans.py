"""The gated linear recurrence in every way a call can run: 64-byte slices, 32-byte slices
(narrow), whole lines, segments, and tiles for short sequences; against the oracle, with states,
several heads and batch rows, and closed gates.
Tolerances as in test_gpu_glr.py."""

import pytest
import torch

from gated_delta_rule_kla_amd import kla
from oracle.glr_oracle import glr_backward, glr_forward
from test_gpu_glr import BF, DEV, F32, check, cu_of, f64, inputs, near

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a GPU")]

DTYPES = [BF, F32]

# B, H, T, d, cu.  64-byte slices are W = N H ceil(d / 32) (bf16; 16 in fp32): W >= 256, or up to
# 2,048 tokens, run whole; else 32-byte slices where W >= 128 or up to 3,584 tokens; else segments.
NARROW = [(2, 3, 3000, 64, None), (1, 5, 2049, 40, None), (3, 2, 3584, 16, None),
          (1, 3, 5000, 72, [0, 0, 7, 2500, 2501, 2501, 5000])]
NARROW_LONG = {BF: (1, 4, 4100, 1024, None), F32: (1, 4, 4100, 512, None)}
SEGMENTS = [(2, 3, 3700, 40, None), (3, 2, 5200, 5, None), (1, 2, 4096, 6, None), (2, 2, 3585, 64, None),
            (1, 3, 9000, 24, [0, 1, 1, 4000, 8500, 8600, 9000]), (1, 2, 6000, 3, [0, 5000, 5000, 5513, 6000])]


def segmented(B, H, T, d, cu, dtype):
    return kla.glr_chunk_workspace_bytes(B, H, T, d, dtype,
                                         None if cu is None else torch.tensor(cu, dtype=torch.int32)) > 0


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("B,H,T,d,cu", NARROW)
def test_narrow(dtype, B, H, T, d, cu):
    assert not segmented(B, H, T, d, cu, dtype)
    check(dtype, B, H, T, d, cu, seed=T + d, slow=0.02)


@pytest.mark.parametrize("dtype", DTYPES)
def test_narrow_and_long(dtype):
    B, H, T, d, cu = NARROW_LONG[dtype]
    assert not segmented(B, H, T, d, cu, dtype)
    check(dtype, B, H, T, d, cu, seed=1, slow=0.02)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("B,H,T,d,cu", SEGMENTS)
def test_segments(dtype, B, H, T, d, cu):
    assert segmented(B, H, T, d, cu, dtype)
    check(dtype, B, H, T, d, cu, seed=T + d, slow=0.02)


PLANS = {"short": (2, 3, 60, 16, None), "four waves": (2, 3, 200, 16, None), "wide": (2, 3, 600, 40, None),
         "narrow": (2, 3, 2500, 64, None), "lines": (4, 64, 700, 64, None), "segments": (2, 3, 3700, 40, None),
         "segments, elements": (1, 2, 4000, 5, None), "packed segments": (1, 3, 9000, 24, [0, 1, 1, 4000, 8500, 8600, 9000])}


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("plan", PLANS)
def test_closed_gates(dtype, plan):
    """exp(-inf) = 0 forgets whatever was before, in tiles, between tiles and segments."""
    B, H, T, d, cu = PLANS[plan]
    x, g, h0, do, df = inputs(dtype, B, H, T, d, cu, seed=3, slow=0.02)
    for t in (0, 17, 18, 64, 511, 512, 513, 1023, 1024, 2048, T // 2, T - 1):
        if t < T:
            g[:, :, t, ::2] = -float("inf")
    dev, host = cu_of(cu)
    put = lambda t: t.to(DEV)  # noqa: E731
    o, hf = kla.glr_chunk_fwd(put(x), put(g), put(h0), dev, cu_seqlens_host=host)
    want, wf, eo, ef = glr_forward(f64(x), f64(g), f64(h0), cu)
    near(o, want, eo, dtype, "o")
    near(hf, wf, ef, F32, "final state")
    dx, dg, d0 = kla.glr_chunk_bwd(put(g), o, put(do), put(h0), put(df), dev, cu_seqlens_host=host)
    rx, rg, r0, ex, eg, e0 = glr_backward(f64(g), f64(o), f64(do), f64(h0), f64(df), cu)
    near(dx, rx, ex, dtype, "dx")
    near(dg, rg, eg, dtype, "dg")
    near(d0, r0, e0, F32, "dh0")
    shut = torch.isinf(g).to(DEV)
    assert not dg[shut].any()


@pytest.mark.parametrize("dtype,d", [(BF, 600000), (BF, 540001), (F32, 270002)])
def test_rows_of_more_than_a_mebibyte(dtype, d):
    """Whose offsets within a tile would pass 32 bits: they go 8 bytes or one element at a time."""
    check(dtype, 1, 1, 9, d, seed=d, slow=0.3)
    check(dtype, 1, 2, 5, d, cu=[0, 0, 2, 5], seed=d, slow=0.3)
