"""Few new tokens over caches whose codes are read past the memory-side cache, as the bound on
the lengths says: a large bound over a small cache, of which nothing beyond seq_lens is read."""

import pytest
import torch

from test_gpu_kv4_chunk import BF, F32, Cache, run

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a GPU")]


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("D,page", [(64, 16), (128, 64)])
@pytest.mark.parametrize("new", [[1, 2, 0, 3, 1], [20, 0, 9, 31, 33]])
def test_large_bounds(dtype, D, page, new):
    """Tiles of 16 rows and, in bf16, of 32."""
    Hkv, G, bound = 3, 4, 131072
    lens = [700, 5, 64, 2500, 40]
    lens = [max(a, b) for a, b in zip(lens, new)]
    rows = -(-sum(new) * G // len(new))
    assert rows <= 16 if sum(new) < 10 else 16 < rows <= 128
    assert len(new) * Hkv * bound * (D + D // 16) >= 96 << 20
    run(Cache(lens, Hkv, D, page), new, Hkv * G, dtype, max_len=bound)
