"""The 8-bit block-scaled cache where its calls can go wrong, on the GPU against the float64
definitions of block_ref."""
import math

import numpy as np
import pytest
import torch

from rotation_quantized_kv_rq_gb300 import rq
from tests import block_ref as R
from tests.test_block_gpu import DT, check, dev, filled, gen, host, wide, within

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


CALLS = ["decode", "verify", "tree", "extend", "extend, own kernel"]


@pytest.mark.parametrize("dtype,sm_scale", [("bf16", 0.0), ("f16", 0.0), ("f16", 1e-30), ("bf16", 1e-30)])
@pytest.mark.parametrize("values", [False, True])
@pytest.mark.parametrize("call", CALLS)
def test_zero_queries_over_zero_keys(call, values, dtype, sm_scale):
    """The product of the factors of a score (of the query row, of the softmax, of the keys' block) can be
    below f32's range: what a row may not see keeps no weight all the same, and what it sees has equal
    weights.  values: keys of zeros were appended with values; else a pool of zeros as it is made."""
    dtype, rng, P, hq, hkv = DT[dtype], gen(50), 16, 4, 2
    T = 1 if call == "decode" else 3
    lens = np.array([1, 15, 17, 0, 40, 300], np.int32)
    need = (lens + P - 1) // P
    width = max(int(need.max()), wide(len(lens), T, hq, P) if "own" in call else 0)
    table = np.zeros((len(lens), width), np.int32)
    for b, at in enumerate(np.cumsum(need) - need):
        table[b, :need[b]] = np.arange(at, at + need[b])
    cache = rq.KVCache(rq.RQ_FP8, 8, hq, hkv, P, int(need.sum()), None, None, max_batch=len(lens), max_query_tokens=T,
                       max_pages_per_seq=width, sm_scale=sm_scale, dtype=dtype)
    lens = np.where((lens > 0) & (lens < T), T, lens).astype(np.int32)  # (a sequence holds its query tokens)
    if values:
        for b, L in enumerate(lens):
            if L:
                pos = np.arange(L)
                v = dev(rng.standard_normal((L, hkv, 128)), dtype)
                cache.append(torch.zeros_like(v), v, dev((table[b, pos // P] * P + pos % P).astype(np.int32)))
    q = torch.zeros((len(lens), T, hq, 128), dtype=dtype, device="cuda")
    args = dev(table), dev(lens)
    if call == "decode":
        out = cache.decode(q[:, 0].contiguous(), *args)[:, None]
    elif call == "tree":
        out = cache.tree_verify(q, torch.tensor([[1, 3, 5]] * len(lens), device="cuda"), *args)
    else:
        out = (cache.verify if call == "verify" else cache.extend)(q, *args)

    def see(b, j, p):
        i = p - (lens[b] - T)
        return i <= (0, 1, 2)[j] if call != "tree" else (i < 0) | ((1, 3, 5)[j] >> np.maximum(i, 0) & 1).astype(bool)
    check(cache, table, lens, q, out, see, call)
    if not values:
        assert (out == 0).all()


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("call", ["decode", "extend"])
def test_a_long_flat_tail_beside_a_heavy_token(call, dtype):
    """One token with a value of 0, and 2^17 with values of 1 whose weights are 2^-26 of its own: the result
    is 2^-9.  Many sequences on the same pages, so that all of one is summed in few places.  A weight's
    step is at most 2^-31 of the row's largest weight, half of which a token may lose."""
    dtype, N, P = DT[dtype], 1 << 17, 256
    B, hq, T = (640, 1, 1) if call == "decode" else (160, 64, 1)
    cache = rq.KVCache(rq.RQ_FP8, 8, hq, 1, P, N // P + 1, None, None, max_batch=B, dtype=dtype)
    k, v = torch.zeros((N + 1, 1, 128), dtype=dtype, device="cuda"), torch.ones((N + 1, 1, 128), dtype=dtype, device="cuda")
    k[0, 0, 0], v[0] = 1, 0
    cache.append(k, v, torch.arange(N + 1, dtype=torch.int32, device="cuda"))
    q = torch.zeros((B, T, hq, 128), dtype=dtype, device="cuda")
    q[..., 0] = 26 * math.log(2) * math.sqrt(128)
    table = torch.arange(N // P + 1, dtype=torch.int32, device="cuda").repeat(B, 1)
    lens = torch.full((B,), N + 1, dtype=torch.int32, device="cuda")
    out = cache.decode(q[:, 0], table, lens)[:, None] if call == "decode" else cache.extend(q, table, lens)
    tail = N * math.exp(-float(q[0, 0, 0, 0]) / math.sqrt(128))
    ref = np.full(tuple(out.shape), tail / (1 + tail))
    within(host(out), ref, N * 2.0 ** -32 + (2.0 ** -11 + 2.0 ** -20) * ref + R.half_step(dtype, ref) * (1 + 2.0 ** -8))


@pytest.mark.parametrize("which", ["k", "v"])
def test_append_reports_clipped_values(which):
    """A finite magnitude above 448 * 2^60 is stored as that, and reported; one of just that is not."""
    cache = rq.KVCache(rq.RQ_FP8, 8, 2, 2, 16, 2, None, None, max_batch=1, dtype=torch.bfloat16)
    x = dict(k=torch.ones((2, 2, 128), dtype=torch.bfloat16, device="cuda"), v=torch.ones((2, 2, 128), dtype=torch.bfloat16, device="cuda"))
    x[which][0, 0, 5] = -448 * 2.0 ** 60
    slots = torch.tensor([0, 16], dtype=torch.int32, device="cuda")
    cache.append(x["k"], x["v"], slots)
    assert int(cache.status.item()) == 0
    x[which][1, 1, 7] = 450 * 2.0 ** 60
    cache.append(x["k"], x["v"], slots)
    assert int(cache.status.item()) == rq.RQ_STATUS_NORM_OVERFLOW
    codes, exps = R.unpack(cache.pages.cpu().numpy(), 16)
    kind = "kv".index(which)
    assert exps[kind][0, 0, 0] == exps[kind][1, 1, 0] == 60
    assert codes[kind][0, 0, 0, 5] == -448 and codes[kind][1, 1, 0, 7] == 448


@pytest.mark.parametrize("slots,written", [
    ([3, -1, 4], []), ([3, -1, 5], [3]), ([0, 1, -1, 2], [0, 1]), ([3, 5], []), ([6, 5], []), ([16, 18, 17], [16]), ([5, 5], []),
    ([9, 40, 10, 41, 20], [20]),                                      # [token][sequence]
    ([0, 16, 32, 1, 17, 33], [0, 16, 32]),
    ([-1, 9, 10, -1, 40, 41, -1, -1], [9, 10, 40, 41]),               # in order, padded
    (list(range(7, 39)) + [6], list(range(16, 39))),                  # a stray token of the first run's block
], ids=str)
@pytest.mark.parametrize("more", [0, 300, 2200])
def test_append_reports_tokens_apart(slots, written, more):
    """Tokens of one block that do not stand together: at most one run of them is written, the one that
    starts the block if the call has it, and that is reported.  more: tokens of a further sequence behind them, which are all written."""
    rng, hkv, hq, P = gen(len(slots) + more), 2, 3, 16
    caches = [rq.KVCache(rq.RQ_FP8, 8, hkv, hkv, P, 160, None, None, max_batch=1) for _ in range(2)]
    fill = dev(rng.standard_normal((48, hkv, 128)), torch.float16)
    for c in caches:
        c.append(fill, fill, torch.arange(48, dtype=torch.int32, device="cuda"))
    extra = list(range(53, 53 + more))
    all_slots = np.array(slots + extra, np.int32)
    n = len(all_slots)
    q, k, v = (dev(rng.standard_normal((n, h, 128)) * 4, torch.float16) for h in (hq, hkv, hkv))
    rope, pos = rq.Rope(128), torch.arange(n, dtype=torch.int32, device="cuda")
    out = caches[0].append_rope(k, v, dev(all_slots), rope, pos, q=q)
    keep = np.array([i for i, s in enumerate(all_slots) if s in written or s in extra], np.int64)
    if keep.size:
        at = torch.from_numpy(keep).cuda()
        caches[1].append_rope(k[at], v[at], dev(all_slots[keep]), rope, pos[at])
    assert torch.equal(caches[0].pages, caches[1].pages)
    assert torch.equal(out, rope.apply(q, None, pos)[0])
    assert int(caches[1].status.item()) == 0
    apart = sum(s >= 0 for s in slots) > len(written)
    assert int(caches[0].status.item()) == (rq.RQ_STATUS_BAD_ORDER if apart else 0)


@pytest.mark.parametrize("slots,dropped", [
    (list(range(5, 2605)) + [3], list(range(5, 16)) + [3]),
    (list(range(5, 805)) + list(range(806, 2606)) + [805], list(range(806, 816)) + [805]),
    ([2605] + list(range(5, 2605)), [2605]),                    # its block's start comes last
])
@pytest.mark.parametrize("skip", [0, 1, 3])
def test_append_reports_a_stray_token_of_a_long_call(slots, dropped, skip):
    """The same far apart in a call of many tokens, slots at every alignment."""
    rng, n = gen(skip), len(slots)
    caches = [rq.KVCache(rq.RQ_FP8, 8, 1, 1, 32, 82, None, None, max_batch=1, dtype=torch.bfloat16) for _ in range(2)]
    k, v = (dev(rng.standard_normal((n, 1, 128)), torch.bfloat16) for _ in range(2))
    s = torch.tensor([0] * skip + slots, dtype=torch.int32, device="cuda")[skip:]
    caches[0].append(k, v, s)
    at = torch.tensor([i for i in range(n) if slots[i] not in dropped], device="cuda")
    caches[1].append(k[at], v[at], s[at])
    assert torch.equal(caches[0].pages, caches[1].pages)
    assert [int(c.status.item()) for c in caches] == [rq.RQ_STATUS_BAD_ORDER, 0]


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("P,hkv,B", [(16, 1, 1), (32, 3, 40), (256, 8, 9)])
def test_decode_step_over_a_cache_in_use(dtype, P, hkv, B):
    """Steps one after the other against append and decode of the same tokens: the same pages and results."""
    dtype, rng, hq = DT[dtype], gen(60 + B), 2 * hkv
    start = rng.integers(0, 3 * P, B)
    a, table, lens = filled(rng, hq, hkv, P, start, dtype)
    extra = make_wider(a, table, start, 20)
    pages = extra.max() + 1
    caches = [rq.KVCache(rq.RQ_FP8, 8, hq, hkv, P, int(pages), None, None, max_batch=B, dtype=dtype) for _ in range(2)]
    for c in caches:
        c.pages[:a.num_pages] = a.pages
    for i in range(18):
        lens = (start + i + 1).astype(np.int32)
        q, k, v = (dev(rng.standard_normal((B, h, 128)) * 2.0 ** rng.integers(-2, 3), dtype) for h in (hq, hkv, hkv))
        got = caches[0].decode_step(q, k, v, dev(extra), dev(lens))
        slots = extra[np.arange(B), (lens - 1) // P] * P + (lens - 1) % P
        caches[1].append(k, v, dev(slots.astype(np.int32)))
        assert torch.equal(got, caches[1].decode(q, dev(extra), dev(lens))), i
    assert torch.equal(caches[0].pages, caches[1].pages)
    check(caches[0], extra, lens, q[:, None], got[:, None], lambda b, j, p: p <= lens[b] - 1, "step")


def make_wider(cache, table, start, more):
    """The block table with pages of their own for `more` further tokens of every sequence."""
    P = cache.page_size
    need = (start + more + P - 1) // P
    out, at = np.zeros((len(start), need.max()), np.int32), cache.num_pages
    for b, s in enumerate(start):
        have = (s + P - 1) // P
        out[b, :have] = table[b, :have]
        out[b, have:need[b]] = np.arange(at, at + need[b] - have)
        at += need[b] - have
    return out
