"""The smallest and largest scales of attention: a subnormal one weighs all keys alike, and one
near the limit leaves the largest score alone, also where masked keys stand beside it."""

import pytest
import torch

from gated_delta_rule_kla_amd import kla
from test_gpu_attn import BF, DEV, F32, check, f64, inputs
from test_gpu_kv4 import check as check_decode
from test_gpu_kv4 import fill, i32

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a GPU")]


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("scale", [1e-45, -1e-40])
def test_subnormal(dtype, scale):
    q, k, v = inputs(dtype, 1, 4, 2, 200, 233, 64, 1)
    o, lse = kla.attn_fwd(q, k, v, scale)
    check(o, lse, q, k, v, scale, dtype)
    codes, scales, table, kv = fill([70, 1, 0], 2, 64, 16)
    q = torch.randn(3, 4, 64, device=DEV).to(dtype)
    check_decode(kla.attn_kv4_decode_step(q, codes, scales, table, i32([70, 1, 0]), scale=scale), q, kv, scale, dtype)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("sign", [1, -1])
def test_large(dtype, sign):
    """Scores 128 apart, up to 19,072: each query's best key has all the weight there is, the next
    one e^-128 of it, which is zero in fp32.

    The best weight itself is exp of a score's rounding error, w, near 1; o = (w v) / w.  In bf16 w
    is rounded before it meets v (2^-8), and o is (2^-8).  In fp32 w and v are three bf16 terms each
    (2^-24 each), of whose products six are summed (6 2^-24), and the sum is divided by a reciprocal
    (2 2^-24) and rounded (2^-24): 16 2^-24 covers that."""
    scale = sign * 2.0 ** 127
    q, k, v = inputs(dtype, 1, 2, 1, 150, 150, 64, 2)
    q.zero_(), k.zero_()
    q[..., 0] = 2.0 ** -60
    k[0, 0, :, 0] = torch.randperm(150, generator=torch.Generator().manual_seed(0)).to(DEV) * 2.0 ** -60 * sign
    o, lse = kla.attn_fwd(q, k, v, scale)
    best = torch.cummax(k[0, 0, :, 0].float() * sign, 0).indices
    tol = 2 * 2.0 ** -8 if dtype == BF else 2.0 ** -20
    for h in (0, 1):
        assert (abs(f64(o[0, h]) - f64(v[0, 0, best])) <= tol * abs(f64(v[0, 0, best]))).all()
    want = f64(k[0, 0, best, 0]) * 2.0 ** -60 * scale
    assert (abs(f64(lse[0, 0]) - want) <= 2.0 ** -20 * abs(want)).all()
