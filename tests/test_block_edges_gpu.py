"""The 8-bit block-scaled cache where its calls can go wrong, on the GPU against the float64
definitions of block_ref."""
import numpy as np
import pytest
import torch

from tests import block_ref as R
from tests.test_block_gpu import DT, check, dev, filled, gen

pytestmark = pytest.mark.gpu


def poke_nan_value(cache, page, offset):
    """NaN into the value code of one token, all kv heads and dims."""
    places = torch.from_numpy(R.PLACES[1][offset % 16]).cuda() + offset // 16 * 4112
    cache.pages[int(page)][:, places] = 0x7F


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("T,hq,hkv", [(1, 4, 4), (7, 8, 2), (4, 16, 4), (5, 20, 4), (9, 40, 2)])  # 1, 28, 16, 25, 180 rows
def test_tree_mask_of_the_first_draft(dtype, T, hq, hkv):
    """Sixteen lengths, so that draft 0 stands at every place of a tile, its last one included, where a
    chain's rows would all see it.  Rows without its bit do not see it, not even if its value is NaN."""
    rng, dtype, P, B = gen(T * hq), DT[dtype], 16, 16
    cache, table, lens = filled(rng, hq, hkv, P, [T + 33 + i for i in range(B)], dtype, t=T)
    mask = rng.integers(0, 2 ** 63, (B, T), dtype=np.uint64) & np.uint64((1 << T) - 1)
    without = rng.random((B, T)) < 0.5
    without[:, 0] = np.arange(B) % 3 > 0
    without[(lens - T) % 16 == 15, 0] = True
    mask = np.where(without, mask & ~np.uint64(1), mask | np.uint64(1))
    q = dev(rng.standard_normal((B, T, hq, 128)) / 4, dtype)  # no weight below fp16's range
    call = lambda: cache.tree_verify(q, dev(mask.view(np.int64)), dev(table), dev(lens))  # noqa: E731
    out = call()

    def see(b, j, p):
        i = p - (lens[b] - T)
        return (i < 0) | (mask[b, j] >> np.maximum(i, 0).astype(np.uint64) & np.uint64(1)).astype(bool)
    check(cache, table, lens, q, out, see, "tree verify")
    for b in range(B):
        at = int(lens[b]) - T
        poke_nan_value(cache, table[b, at // P], at % P)
    again = call()
    blind = torch.from_numpy(without).cuda()
    assert torch.equal(again[blind], out[blind])
    assert torch.isnan(again[~blind]).all()
