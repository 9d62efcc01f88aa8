"""The 4-bit cache and padded batches, whose offsets on the device end before the rows do."""

import numpy as np
import pytest
import torch

from gated_delta_rule_kla_amd import kla
from oracle.attn_oracle import quantise, values
from test_gpu_kv4 import BF, DEV, F32, f64, make_kv

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a GPU")]

DTYPES = [BF, F32]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("N", [4, 1100])
def test_tokens_of_no_sequence(dtype, N):
    """A padded batch: the device's offsets end before the rows (and begin behind their first
    ones).  Tokens in front of the first sequence and behind the last have no place: the pages
    that the table leads them to keep what they hold, and their rows are not written."""
    lens = [3] * N
    M, page = 2, 16
    table = torch.arange(N * M, dtype=torch.int32, device=DEV).reshape(N, M)
    T = 3 * N + 29
    host = torch.tensor([3 * n for n in range(N)] + [T], dtype=torch.int32)
    cu = torch.tensor([2] + [3 * n for n in range(1, N)] + [3 * N], dtype=torch.int32, device=DEV)
    start = torch.full((N,), 5, dtype=torch.int32, device=DEV)
    k, v = make_kv([T], 2, 64, dtype, 1)
    codes, scales = kla.kv4_cache(N * M, 2, page, 64, DEV)
    codes.fill_(0xA5)
    scales.fill_(0x77)
    kla.kv4_append(k, v, codes, scales, table, start, cu, host)
    touched = torch.zeros(N * M, page, dtype=torch.bool)
    touched[torch.arange(N) * M, 5] = True
    for i in (1, 2):
        touched[torch.arange(1, N) * M, 5 + i] = True
    rest = ~touched
    assert (codes.cpu().permute(0, 3, 1, 2, 4)[rest] == 0xA5).all()
    assert (scales.cpu().permute(0, 3, 1, 2, 4)[rest] == 0x77).all()
    out = tuple(torch.full_like(k, 7.0) for _ in "kv")
    kla.kv4_read(codes, scales, table, start, cu, dtype, host, out=out)
    for x, y in ((k, out[0]), (v, out[1])):
        assert (y[:, :, :2] == 7).all() and (y[:, :, 3 * N:] == 7).all()
        np.testing.assert_array_equal(f64(y[:, :, 2:3 * N]), values(*quantise(f64(x[:, :, 2:3 * N]))))


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("dense", [False, True])
def test_a_negative_start_is_padding(dtype, dense):
    """For all tokens of the sequence, also those that would come to lie at position 0 and up."""
    start = torch.tensor([3, -1, -5, -2 ** 31], dtype=torch.int32, device=DEV)
    table = torch.arange(8, dtype=torch.int32, device=DEV).reshape(4, 2)
    k, v = make_kv([24], 2, 64, dtype, 2)
    codes, scales = kla.kv4_cache(8, 2, 16, 64, DEV)
    host = torch.tensor([0, 6, 12, 18, 24], dtype=torch.int32)
    if dense:
        rows = [t.view(2, 4, 6, 64).transpose(0, 1).contiguous() for t in (k[0], v[0])]
        kla.kv4_append(*rows, codes, scales, table, start)
    else:
        kla.kv4_append(k, v, codes, scales, table, start, host.to(DEV), host)
    assert codes[0, :, :, 3:9].any(-1).all()
    codes[0, :, :, 3:9], scales[0, :, :, 3:9] = 0, 0
    assert not codes.any() and not scales.any()
    codes.fill_(0x22)  # ones, times 2^0
    scales.fill_(127)
    y = kla.kv4_read(codes, scales, table, start, host.to(DEV), dtype, host)
    for t in y:
        assert (t[:, :, :6] == 1).all() and not t[:, :, 6:].any()
