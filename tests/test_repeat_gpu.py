"""A call's result does not depend on what ran before it on the same SMs: shared memory keeps an
earlier launch's tiles, and a pair's missing second tile must not be read from there."""
import numpy as np
import pytest
import torch

from rotation_quantized_kv_rq_gb300 import rq, synth

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("mode,bits", [(synth.PLANAR, 3), (synth.ISO, 4), (synth.DENSE, 2)])
def test_decode_after_large_value_norms(mode, bits):
    rng = np.random.default_rng(3)
    hq, hkv, P, lens = 32, 8, 16, np.array([5000, 3000, 777, 12345], np.int32)
    need = (lens + P - 1) // P
    table = np.zeros((4, need.max()), np.int32)
    for b, at in enumerate(np.cumsum(need) - need):
        table[b, :need[b]] = np.arange(at, at + need[b])
    n = int(need.sum()) * P
    rot_k, rot_v = (synth.rotation_params(mode, hkv, rng) for _ in range(2))
    caches = []
    for scale in (1.0, 60.0):  # value norms of about 11, and of about 680
        c = rq.KVCache(mode, bits, hq, hkv, P, int(need.sum()), rot_k, rot_v, max_batch=4, max_pages_per_seq=int(need.max()))
        g = torch.Generator(device="cuda").manual_seed(5)
        k, v = (torch.randn((n, hkv, 128), generator=g, device="cuda") for _ in range(2))
        c.append(k.half(), (v * scale).half(), torch.arange(n, dtype=torch.int32, device="cuda"))
        caches.append(c)
    q = torch.from_numpy(rng.standard_normal((4, hq, 128))).half().cuda()
    bt, sl = torch.from_numpy(table).cuda(), torch.from_numpy(lens).cuda()
    for _ in range(8):
        caches[0].decode(q, bt, sl)  # shared memory holds small norms only
    want = caches[0].decode(q, bt, sl)
    for i in range(24):  # other lengths: other units, with tiles where the call has none
        caches[1].decode(q, bt, torch.from_numpy(rng.integers(1, lens + 1, dtype=np.int32)).cuda())
        assert torch.equal(caches[0].decode(q, bt, sl), want), i
