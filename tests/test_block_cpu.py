"""The 8-bit block-scaled cache and the position rotation on a host without a GPU: what the calls
refuse before they touch CUDA, the byte places of a block, and the frequencies' fixed-point form."""
import ctypes

import numpy as np
import pytest

from rotation_quantized_kv_rq_gb300 import rq
from tests import block_ref as R


def config(**over):
    base = dict(head_dim=128, num_q_heads=32, num_kv_heads=8, bits=8, mode=rq.RQ_FP8, page_size=16, num_pages=64,
                max_batch=4, max_query_tokens=1, max_pages_per_seq=8, sm_scale=0.0, io_type=0)
    base.update(over)
    cfg = rq.rq_config()
    for k, v in base.items():
        setattr(cfg, k, v)
    cfg.device = -1
    return cfg


@pytest.mark.parametrize("over,code", [
    (dict(bits=4), rq.RQ_ERR_UNSUPPORTED),
    (dict(head_dim=64), rq.RQ_ERR_UNSUPPORTED),
    (dict(page_size=24), rq.RQ_ERR_UNSUPPORTED),
    (dict(page_size=512), rq.RQ_ERR_UNSUPPORTED),
    (dict(num_q_heads=30), rq.RQ_ERR_INVALID),
    (dict(io_type=2), rq.RQ_ERR_INVALID),
    (dict(mode=7), rq.RQ_ERR_INVALID),
    (dict(mode=rq.RQ_PLANAR, bits=4, io_type=rq.RQ_BF16), rq.RQ_ERR_UNSUPPORTED),
    (dict(sm_scale=-1.0), rq.RQ_ERR_INVALID),
    (dict(num_pages=2 ** 28, page_size=16), rq.RQ_ERR_UNSUPPORTED),
    (dict(num_kv_heads=40000, num_q_heads=40000, page_size=256), rq.RQ_ERR_UNSUPPORTED),
])
def test_create_refuses(over, code):
    ctx = ctypes.c_void_p(1)
    assert rq.lib().rq_create(ctypes.byref(ctx), ctypes.byref(config(**over))) == code
    assert ctx.value is None


def test_create_refuses_a_codebook():
    book = np.zeros(256, np.float32)
    cfg = config()
    cfg.codebook = book.ctypes.data_as(ctypes.POINTER(ctypes.c_float))
    ctx = ctypes.c_void_p()
    assert rq.lib().rq_create(ctypes.byref(ctx), ctypes.byref(cfg)) == rq.RQ_ERR_INVALID
    with pytest.raises(rq.RQError):
        rq.rq_create(rq.RQ_FP8, 8, 32, 8, 16, 64, np.zeros((8, 128)), None, max_batch=1)


def test_noalloc_refuses_the_mode():
    cfg = config(bits=8)
    assert rq.lib().rq_decode_attention_noalloc(ctypes.byref(cfg), 16, 16, 16, 16, 16, 16, 1, 16, 1, 16, None,
                                                None) == rq.RQ_ERR_UNSUPPORTED


@pytest.mark.parametrize("over", [
    dict(rotary_dim=-8), dict(rotary_dim=136), dict(rotary_dim=12), dict(num_axes=0), dict(num_axes=9),
    dict(freq=-1.0), dict(freq=float("nan")), dict(freq=float("inf")), dict(freq=1e6), dict(freq=None),
    dict(axis=1), dict(axis=-1), dict(scale=float("inf")),
])
def test_rope_create_refuses(over):
    a = dict(rotary_dim=64, num_axes=1, freq=1.0, axis=0, scale=1.0)
    a.update(over)
    f = np.full(64, 0.0 if a["freq"] is None else a["freq"])
    ax = np.full(64, a["axis"], np.intc)
    cfg = rq.rq_rope_config(a["rotary_dim"], 0, a["num_axes"],
                            None if a["freq"] is None else f.ctypes.data_as(ctypes.POINTER(ctypes.c_double)),
                            ax.ctypes.data_as(ctypes.POINTER(ctypes.c_int)), a["scale"], -1)
    rope = ctypes.c_void_p(1)
    assert rq.lib().rq_rope_create(ctypes.byref(rope), ctypes.byref(cfg)) == rq.RQ_ERR_INVALID
    assert rope.value is None


def rows(x=0x10000, stride=1024, heads=8, weight=None, out=0x90000, out_stride=1024):
    return rq.rq_rows(x, stride, heads, weight, out, out_stride)


N = 4  # tokens of the refused calls: rows of 8 heads at 0x10000 end at 0x12000


@pytest.mark.parametrize("q,k", [
    (None, None),
    (rows(x=None), None),
    (rows(x=0x10008), None),
    (rows(out=None), None),
    (rows(out=0x90008), None),
    (rows(weight=0x50004), None),
    (rows(heads=0), None),
    (rows(stride=1016), None),               # a token's heads overlap the next token's
    (rows(stride=1028), None),
    (rows(out_stride=896), None),
    (rows(out=0x10100), None),               # out over x, not in place
    (rows(out=0x10000, out_stride=2048), None),
    (rows(), rows(x=0x90400)),               # k inside q's out
    (rows(), rows(x=0x20000, out=0x90800)),  # both outs over each other
    (rows(x=0x10000, out=0x90000, stride=2048, out_stride=2048), rows(x=0x10400, out=0x90400, stride=2048, out_stride=2048)),
], ids=str)
def test_norm_rope_refuses(q, k):
    ref = lambda r: None if r is None else ctypes.byref(r)  # noqa: E731
    assert rq.lib().rq_norm_rope(None, ref(q), ref(k), 0, 1e-6, None, N, None) == rq.RQ_ERR_INVALID


@pytest.mark.parametrize("io,eps,n", [(2, 1e-6, 4), (-1, 1e-6, 4), (0, -1.0, 4), (0, float("nan"), 4),
                                      (0, float("inf"), 4), (0, 1e-6, -1)])
def test_norm_rope_refuses_scalars(io, eps, n):
    assert rq.lib().rq_norm_rope(None, ctypes.byref(rows()), None, io, eps, None, n, None) == rq.RQ_ERR_INVALID


def test_null_calls():
    L = rq.lib()
    L.rq_rope_free(None)
    assert L.rq_rope_create(None, None) == rq.RQ_ERR_INVALID
    assert L.rq_norm_rope(None, ctypes.byref(rows()), None, 0, 1e-6, None, 0, None) == rq.RQ_OK
    assert L.rq_rope_append(None, None, None, None, None, 1024, 1e-6, None, None, 1, None, None,
                            None) == rq.RQ_ERR_INVALID


def test_places_are_a_permutation_of_the_block():
    both = np.concatenate([p.reshape(-1) for p in R.PLACES])
    assert np.array_equal(np.sort(both), np.arange(4096))


@pytest.mark.parametrize("amax,e", [(0.0, -60), (448.0, 0), (449.0, 1), (224.0, -1), (224.5, 0), (65504.0, 8),
                                    (1e-30, -60), (3e38, 60)])
def test_exponent_of_the_definition(amax, e):
    assert R.exponent(amax) == e
