"""The 8-bit block-scaled cache's refusals at the ends of its ranges, on a host without a GPU."""
import ctypes

import pytest

from rotation_quantized_kv_rq_gb300 import rq
from tests.test_block_cpu import config


@pytest.mark.parametrize("page_size", [16, 48, 256])
def test_create_refuses_positions_near_the_end_of_int32(page_size):
    """Positions are 32 bits wide, and an attention kernel looks up pages some way past a sequence's end."""
    ctx = ctypes.c_void_p(1)
    cfg = config(page_size=page_size, max_pages_per_seq=(2 ** 31 - 1) // page_size)
    assert rq.lib().rq_create(ctypes.byref(ctx), ctypes.byref(cfg)) == rq.RQ_ERR_UNSUPPORTED
    assert ctx.value is None
