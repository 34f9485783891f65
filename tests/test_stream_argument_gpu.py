"""Calls of KVCache and Rope with stream=: the outputs that they make are the stream's own memory."""
import pytest
import torch

from rotation_quantized_kv_rq_gb300 import rq
from tests.test_block_gpu import dev, filled, gen
from tests.test_latent_edges_gpu import beside

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("raw", [False, True])
def test_outputs_of_calls_with_a_stream(raw):
    rng, dtype, T, heads = gen(3), torch.bfloat16, 64, 32
    cache, table, lens = filled(rng, heads, 4, 16, [300, 70, 129, 64], dtype, t=T)
    tab, lens = dev(table), dev(lens)
    q = dev(rng.standard_normal((4, T, heads, 128)), dtype)
    one, mask = q[:, 0].contiguous(), dev(rng.integers(1, 1 << 62, (4, T)))
    new = dev(rng.standard_normal((2, 4, 4, 128)), dtype)
    handle = lambda s: s.cuda_stream if raw else s  # noqa: E731
    beside(lambda s: cache.decode(one, tab, lens, stream=handle(s)), one.numel() * 2)
    beside(lambda s: cache.decode_step(one, new[0], new[1], tab, lens, stream=handle(s)), one.numel() * 2)
    for call in (cache.verify, cache.extend):
        beside(lambda s: call(q, tab, lens, stream=handle(s)), q.numel() * 2)
    beside(lambda s: cache.tree_verify(q, mask, tab, lens, stream=handle(s)), q.numel() * 2)
    rope, flat = rq.Rope(128), q.view(4 * T, heads, 128)
    pos = torch.arange(4 * T, dtype=torch.int32, device="cuda")
    beside(lambda s: rope.apply(flat, flat, pos, stream=handle(s)), q.numel() * 2)
    kv, slots = flat[:, :4], torch.full((4 * T,), -1, dtype=torch.int32, device="cuda")
    beside(lambda s: cache.append_rope(kv, kv, slots, rope, pos, q=flat, stream=handle(s)), q.numel() * 2)
