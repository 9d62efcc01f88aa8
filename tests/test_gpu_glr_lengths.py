"""The gated linear recurrence with offsets on the device that are not the host's: results are the
device's, in every way a call can run, and rows of no sequence stay as they were.  Tolerances as in
test_gpu_glr.py."""

import pytest
import torch

from gated_delta_rule_kla_amd import kla
from oracle.glr_oracle import glr_backward, glr_forward
from test_gpu_glr import BF, DEV, F32, f64, inputs, near

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a GPU")]

DTYPES = [BF, F32]


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


# Offsets on the device that are not the host's, as where a captured call is replayed with other
# lengths: host, device, heads, channels
OTHER = {"short": ([0, 60, 120, 180], [0, 0, 3, 180], 2, 16),
         "four waves": ([0, 200, 400, 600], [0, 590, 591, 600], 2, 16),
         "wide": ([0, 1000, 2000], [0, 1, 2000], 2, 40),
         "narrow": ([0, 2500, 5000], [0, 4900, 5000], 3, 64),
         "segments": ([0, 4000, 8000], [0, 500, 8000], 3, 40),
         "segments, the other way": ([0, 4000, 8000], [0, 7990, 8000], 1, 16),
         "segments, elements": ([0, 5000, 5001, 9000], [0, 0, 8900, 9000], 2, 5),
         "segments, shorter": ([0, 8000, 8100, 8200], [0, 2700, 5400, 8200], 2, 24)}


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("plan", OTHER)
def test_other_lengths_on_the_device(dtype, plan):
    host, cu, H, d = OTHER[plan]
    T = cu[-1]
    x, g, h0, do, df = (t.to(DEV) for t in inputs(dtype, 1, H, T, d, cu, seed=4, slow=0.02))
    dev, host = i32(cu), torch.tensor(host, dtype=torch.int32)
    o = torch.full_like(x, float("nan"))
    hf = torch.full_like(h0, float("nan"))
    kla.glr_chunk_fwd(x, g, h0, dev, cu_seqlens_host=host, out=o, final_state=hf)
    want, wf, eo, ef = glr_forward(f64(x), f64(g), f64(h0), cu)
    near(o, want, eo, dtype, "o")
    near(hf, wf, ef, F32, "final state")
    # the gradients' buffers are allocated by the call: memory of their sizes full of NaN is there first
    spoil = [torch.full_like(x, float("nan")) for _ in range(2)] + [torch.full_like(h0, float("nan"))]
    del spoil
    dx, dg, d0 = kla.glr_chunk_bwd(g, o, do, h0, df, dev, cu_seqlens_host=host)
    rx, rg, r0, ex, eg, e0 = glr_backward(f64(g), f64(o), f64(do), f64(h0), f64(df), cu)
    near(dx, rx, ex, dtype, "dx")
    near(dg, rg, eg, dtype, "dg")
    near(d0, r0, e0, F32, "dh0")


@pytest.mark.parametrize("plan", OTHER)
def test_rows_behind_the_last_sequence(plan):
    """A padded batch: the device's last offset lies before the end of the rows, which stay as
    they were from there on."""
    host, cu, H, d = OTHER[plan]
    T, end = host[-1], host[-1] - 37
    cu = [min(c, end) for c in cu]
    x, g, h0, *_ = (t.to(DEV) for t in inputs(BF, 1, H, T, d, cu, seed=5, slow=0.02))
    o = torch.full_like(x, 7.0)
    o, hf = kla.glr_chunk_fwd(x, g, h0, i32(cu), cu_seqlens_host=torch.tensor(host, dtype=torch.int32), out=o)
    want, wf, eo, ef = glr_forward(f64(x[:, :, :end]), f64(g[:, :, :end]), f64(h0), cu)
    near(o[:, :, :end], want, eo, BF, "o")
    near(hf, wf, ef, F32, "final state")
    assert (o[:, :, end:] == 7).all()


@pytest.mark.parametrize("dtype", DTYPES)
def test_a_replayed_graph_with_other_lengths(dtype):
    host, H, d = [0, 4000, 8000], 2, 16
    x, g, h0, *_ = (t.to(DEV) for t in inputs(dtype, 1, H, 8000, d, host, seed=6, slow=0.02))
    dev, mirror = i32(host), torch.tensor(host, dtype=torch.int32)
    o, hf = torch.empty_like(x), torch.empty_like(h0)
    kla.glr_chunk_fwd(x, g, h0, dev, cu_seqlens_host=mirror, out=o, final_state=hf)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        kla.glr_chunk_fwd(x, g, h0, dev, cu_seqlens_host=mirror, out=o, final_state=hf)
    for cut in (4000, 100, 7999, 0):
        dev[1] = cut
        o.fill_(float("nan"))
        hf.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        want, wf, eo, ef = glr_forward(f64(x), f64(g), f64(h0), [0, cut, 8000])
        near(o, want, eo, dtype, ("o", cut))
        near(hf, wf, ef, F32, ("final state", cut))
