"""New tokens over the 4-bit cache where their number lies between the plans: some tens to some
hundreds of rows of a sequence, against the fp64 oracles within their bounds."""

import pytest
import torch

from test_gpu_kv4 import BF, F32
from test_gpu_kv4_chunk import Cache, run

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a GPU")]


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("new", [9, 17, 33, 65, 97, 130])
@pytest.mark.parametrize("D,Hkv,G", [(128, 2, 4), (64, 3, 3)])
def test_rows_between(dtype, new, D, Hkv, G):
    """Every sequence with as many new tokens, among them one with all of its tokens new, and
    one where they end inside a tile of keys."""
    run(Cache([new, new + 1, 700, 1029], Hkv, D, 16, seed=new), [new] * 4, Hkv * G, dtype)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("top", [60, 200])
def test_uneven(dtype, top):
    """Sequences with far more rows than the mean, by which the call is planned, and with none."""
    new = [1, 0, top, 2, 3 * top // 2, 5]
    run(Cache([900, 5, 2 * top, 300, 1500, 64], 2, 128), new, 8, dtype)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("T", [20, 40, 90])
def test_dense(dtype, T):
    run(Cache([400, T, 650], 2, 64, 32), [T] * 3, 8, dtype, dense=True)
