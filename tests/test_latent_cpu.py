"""Latent attention on a host without a GPU: what the calls refuse before they touch CUDA, and the cache's byte places."""
import ctypes

import numpy as np
import pytest

from rotation_quantized_kv_rq_gb300 import rq
from tests import latent_ref as L


def config(**over):
    base = dict(num_heads=16, latent_dim=512, position_dim=64, page_size=16, num_pages=64, max_batch=4, max_query_tokens=1,
                max_pages_per_seq=8, sm_scale=0.0, io_type=0)
    base.update(over)
    cfg = rq.rq_latent_config()
    for k, v in base.items():
        setattr(cfg, k, v)
    cfg.device = -1
    return cfg


@pytest.mark.parametrize("over,code", [
    (dict(num_heads=0), rq.RQ_ERR_INVALID),
    (dict(num_heads=1025), rq.RQ_ERR_UNSUPPORTED),
    (dict(latent_dim=256), rq.RQ_ERR_UNSUPPORTED),
    (dict(position_dim=32), rq.RQ_ERR_UNSUPPORTED),
    (dict(latent_dim=-1), rq.RQ_ERR_INVALID),
    (dict(page_size=24), rq.RQ_ERR_UNSUPPORTED),
    (dict(page_size=272), rq.RQ_ERR_UNSUPPORTED),
    (dict(page_size=0), rq.RQ_ERR_INVALID),
    (dict(num_pages=0), rq.RQ_ERR_INVALID),
    (dict(num_pages=2 ** 27), rq.RQ_ERR_UNSUPPORTED),
    (dict(max_pages_per_seq=2 ** 27 - 8), rq.RQ_ERR_UNSUPPORTED),
    (dict(max_batch=0), rq.RQ_ERR_INVALID),
    (dict(max_batch=8001), rq.RQ_ERR_UNSUPPORTED),
    (dict(max_query_tokens=2 ** 27), rq.RQ_ERR_UNSUPPORTED),
    (dict(sm_scale=-1.0), rq.RQ_ERR_INVALID),
    (dict(sm_scale=float("nan")), rq.RQ_ERR_INVALID),
    (dict(sm_scale=float("inf")), rq.RQ_ERR_INVALID),
    (dict(io_type=2), rq.RQ_ERR_INVALID),
])
def test_create_refuses(over, code):
    ctx = ctypes.c_void_p(1)
    assert rq.lib().rq_latent_create(ctypes.byref(ctx), ctypes.byref(config(**over))) == code
    assert ctx.value is None


def test_null_calls():
    lib = rq.lib()
    lib.rq_latent_free(None)
    assert lib.rq_latent_page_bytes(None) == 0
    assert lib.rq_latent_create(None, None) == rq.RQ_ERR_INVALID
    assert lib.rq_latent_append(None, None, 16, 576, None, 1e-6, 16, 576, None, None, None, 16, 1, 16, None,
                                None) == rq.RQ_ERR_INVALID
    assert lib.rq_latent_attention(None, None, None, 1, None, 16, 16, 1, 16, 1, 16, None, None) == rq.RQ_ERR_INVALID
    assert lib.rq_latent_read(None, 16, 16, 1, None, 16, 1, 1, 16, 16, None, None) == rq.RQ_ERR_INVALID
    assert lib.rq_prompt_attention(None, None, None) == rq.RQ_ERR_INVALID


def prompt(**over):
    heads = lambda at, dims, h=4: dict(x=at, stride=h * dims, head_stride=dims, heads=h)  # noqa: E731
    base = dict(q=heads(0x10000, 192), k=heads(0x20000, 128), v=heads(0x30000, 128), k_pe=0x40000, k_pe_stride=64, out=0x50000,
                q_offsets=0x60000, k_offsets=0x60100, B=2, nq=8, nk=8, max_new=8, sm_scale=0.0, io_type=0,
                workspace=0x100000, workspace_bytes=1 << 30)
    for key, value in over.items():
        base[key] = dict(base[key], **value) if isinstance(value, dict) else value
    args = rq.rq_prompt()
    for key, value in base.items():
        setattr(args, key, rq.rq_heads(**value) if isinstance(value, dict) else value)
    return args


@pytest.mark.parametrize("over", [
    dict(q=dict(x=None)), dict(q=dict(x=0x10008)), dict(q=dict(heads=0)), dict(q=dict(stride=764)), dict(q=dict(head_stride=184)),
    dict(q=dict(stride=-768)), dict(k=dict(heads=3)), dict(v=dict(heads=5)), dict(k=dict(head_stride=120)),
    dict(k=dict(x=0x20002)), dict(v=dict(stride=4)), dict(v=dict(x=None)), dict(k_pe=None), dict(k_pe=0x40004),
    dict(k_pe_stride=60), dict(k_pe_stride=56), dict(out=None), dict(out=0x50008), dict(q_offsets=None), dict(k_offsets=None),
    dict(B=-1), dict(B=65536), dict(nq=-1), dict(nk=-1), dict(max_new=-1), dict(sm_scale=-1.0), dict(sm_scale=float("nan")),
    dict(io_type=3), dict(workspace=None), dict(workspace=0x100004),
], ids=str)
def test_prompt_refuses(over):
    assert rq.lib().rq_prompt_attention(ctypes.byref(prompt(**over)), None, None) == rq.RQ_ERR_INVALID


@pytest.mark.parametrize("over", [dict(B=0), dict(nq=0), dict(max_new=0)], ids=str)
def test_prompt_of_nothing(over):
    assert rq.lib().rq_prompt_attention(ctypes.byref(prompt(**over)), None, None) == rq.RQ_OK


@pytest.mark.parametrize("P", [16, 48, 256])
def test_places_are_a_permutation_of_the_page(P):
    r = np.arange(P)[:, None]
    part = L.part_place(P, r, L.PART).reshape(-1)
    every = np.concatenate([L.code_place(P, r, L.DIM).reshape(-1), part, part + 1, 640 * P + np.arange(P)])
    assert np.array_equal(np.sort(every), np.arange(641 * P))


@pytest.mark.parametrize("top,e", [((0.0, 0.0), -60), ((448.0, 0.0), 0), ((449.0, 0.0), 1), ((1.0, 65536.0), 1),
                                   ((1.0, 32768.0), 0), ((1.0, 1.0), -8), ((3e38, 0.0), 60)])
def test_exponent_of_the_definition(top, e):
    assert L.exponent(*top) == e
