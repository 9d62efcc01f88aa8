"""The 4-bit cache where it is rarely used: many sequences, scales that other programs write, NaN
among the tokens that are read."""

import numpy as np
import pytest
import torch

from gated_delta_rule_kla_amd import kla
from oracle.attn_oracle import quantise, values
from test_gpu_kv4 import BF, DEV, F32, check, f64, fill, i32, make_kv, packed, pages

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a GPU")]

DTYPES = [BF, F32]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("N", [1022, 1023, 1024, 1500])
def test_many_sequences(dtype, N):
    """More offsets than a workgroup keeps in LDS."""
    rng = np.random.default_rng(N)
    lens, start = rng.integers(0, 6, N).tolist(), rng.integers(0, 40, N).tolist()
    table, P = pages([a + b for a, b in zip(start, lens)], 16, N)
    codes, scales = kla.kv4_cache(P, 2, 16, 64, DEV)
    k, v = make_kv(lens, 2, 64, dtype, N)
    cu, host = packed(lens)
    kla.kv4_append(k, v, codes, scales, table, i32(start), cu, host)
    got = kla.kv4_read(codes, scales, table, i32(start), cu, dtype, host)
    for x, y in ((k, got[0]), (v, got[1])):
        np.testing.assert_array_equal(f64(y), values(*quantise(f64(x))))
    # each token is where the table says
    tb, b = table.cpu(), host.tolist()
    for n in (0, 1, N // 2, N - 1, int(np.argmax(lens))):
        for i in range(lens[n]):
            pos = start[n] + i
            want = quantise(f64(k)[0, :, b[n] + i])[1]
            np.testing.assert_array_equal(scales[int(tb[n, pos // 16]), 0, :, pos % 16].cpu().numpy(), want)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("D", [64, 128])
def test_every_scale_byte_reads_as_it_is_defined(dtype, D):
    """2^(s - 127), with the smallest byte 0 and the largest numbers beyond the type, and NaN for 255."""
    codes, scales = kla.kv4_cache(16, 1, 16, D, DEV)
    codes.copy_(torch.randint(0, 256, codes.shape, generator=torch.Generator().manual_seed(D)).to(torch.uint8))
    scales.view(16, 2, 16, D // 32).copy_(torch.arange(256, device=DEV).view(16, 1, 16, 1).to(torch.uint8).expand(16, 2, 16, D // 32))
    table = torch.arange(16, dtype=torch.int32, device=DEV)[None]
    cu, host = packed([256])
    got = kla.kv4_read(codes, scales, table, i32([0]), cu, dtype, host)
    for j in (0, 1):
        c = codes[:, j, 0].cpu().numpy().reshape(256, D // 2)
        nib = np.stack([c & 15, c >> 4], -1).reshape(256, D)
        want = torch.from_numpy(values(nib[:255], scales[:, j, 0].cpu().numpy().reshape(256, -1)[:255])).to(dtype)
        y = got[j][0, 0].cpu()
        assert torch.equal(y[:255], want)
        assert y[255].isnan().all()


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("D,Hq,Hkv", [(64, 4, 1), (128, 6, 2)])
def test_decode_over_small_scales(dtype, D, Hq, Hkv):
    """Blocks whose scale byte is 0 or 1 among ordinary ones."""
    lens = [130, 33]
    codes, scales, table, kv = fill(lens, Hkv, D, 16)
    tb = table.cpu()
    for n, pos, j, byte in ((0, 3, 0, 0), (0, 100, 1, 0), (0, 129, 1, 1), (1, 32, 0, 0), (1, 0, 1, 0)):
        p, at = int(tb[n, pos // 16]), pos % 16
        old = int(scales[p, j, 0, at, 0])
        scales[p, j, 0, at, 0] = byte
        kv[n][j][0, pos, :32] *= 2.0 ** (byte - old)
    q = torch.randn(2, Hq, D, device=DEV).to(dtype)
    check(kla.attn_kv4_decode_step(q, codes, scales, table, i32(lens)), q, kv, D ** -0.5, dtype)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("length,at", [(40, 0), (40, 39), (1, 0), (5000, 2500), (5000, 4999)])
def test_decode_over_a_block_of_nan(dtype, length, at):
    """A key that holds a NaN makes its heads' outputs NaN, a value its 32 channels; other heads
    and sequences do not see it, nor does a sequence that ends before it."""
    lens = [length, 70]
    codes, scales, table, kv = fill(lens, 2, 64, 16)
    q = torch.randn(2, 6, 64, device=DEV).to(dtype)

    def step(n=lens):
        return kla.attn_kv4_decode_step(q, codes, scales, table, i32(n), max_len=max(lens))

    clean = step()
    check(clean, q, kv, 0.125, dtype)
    page = int(table[0, at // 16])
    for j in (0, 1):
        old = scales[page, j, 1, at % 16, 1].clone()
        scales[page, j, 1, at % 16, 1] = 255
        o = step()
        bad = o.isnan()
        assert bad[0, 3:, 32 if j else 0:].all() and int(bad.sum()) == 3 * (32 if j else 64)
        assert torch.equal(o[~bad], clean[~bad])
        short = step([at, 70])
        check(short[:1], q[:1], [(kv[0][0][:, :at], kv[0][1][:, :at])], 0.125, dtype)
        scales[page, j, 1, at % 16, 1] = old
    assert torch.equal(step(), clean)
