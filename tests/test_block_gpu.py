"""The 8-bit block-scaled cache, the norms and position rotation before it, and attention over it,
on the GPU against the float64 definitions of block_ref."""
import numpy as np
import pytest
import torch

from rotation_quantized_kv_rq_gb300 import rq
from tests import block_ref as R

pytestmark = pytest.mark.gpu

DT = {"f16": torch.float16, "bf16": torch.bfloat16}
# f32 arithmetic of the norm and the rotation, relative to |a| + |b| of a pair: the mean of 128
# squares (12 roundings, halved by the root), the root, two products: 9 * 2^-24; the angle rounded to
# 24 bits within an eighth of a turn (pi / 4 * 2^-24), sincospif (2^-23), the rotation's three roundings
TURN_ERR = 9 * 2.0 ** -24 + np.pi / 4 * 2.0 ** -24 + 2.0 ** -23 + 3 * 2.0 ** -24


def gen(seed):
    return np.random.default_rng(seed)


def dev(x, dtype=None):
    t = torch.from_numpy(np.ascontiguousarray(x)).cuda()
    return t if dtype is None else t.to(dtype)


def host(t):
    return t.detach().cpu().double().numpy()


def fused(rng, n, hq, hkv, dtype):
    """q, k, v as slices of one projection's output."""
    x = rng.standard_normal((n, hq + 2 * hkv, 128))
    x[:, :, 3] *= 10
    t = dev(x, dtype)
    return t[:, :hq], t[:, hq:hq + hkv], t[:, hq + hkv:]


def within(got, ref, tol, what=""):
    err = np.abs(got - ref)
    bad = ~(err <= tol)
    assert not bad.any(), f"{what}: {bad.sum()} of {bad.size} off, worst {np.nanmax(err / np.maximum(tol, 1e-300)):.3g} of the tolerance"


# ------------------------------------------------------------------------- norms and rotation

@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("n,hq,hkv,rotary,interleaved,sections,norm,far", [
    (1, 1, 1, 128, False, None, True, 100),
    (5, 7, 3, 64, True, None, True, 1 << 20),
    (3, 64, 8, 96, False, (16, 16, 16), True, 1 << 15),
    (700, 12, 4, 128, False, (24, 20, 20), False, 1 << 17),
    (130, 5, 1, 8, True, (1, 3), True, 2 ** 31 - 1),
    (2, 3, 2, 0, False, None, True, 10),
])
def test_norm_rope(dtype, n, hq, hkv, rotary, interleaved, sections, norm, far):
    dtype, rng = DT[dtype], gen(n)
    q, k, _ = fused(rng, n, hq, hkv, dtype)
    axes = len(sections) if sections else 1
    pos = rng.integers(-far, far, (axes, n)).astype(np.int32)
    wq, wk = (1 + 0.2 * rng.standard_normal((2, 128)).astype(np.float32)) if norm else (None, None)
    freq = 10000.0 ** (-2.0 * np.arange(rotary // 2) / max(rotary, 1))
    rope = rq.Rope(rotary, sections=sections, interleaved=interleaved, scale=1.25)
    dw = [None if w is None else dev(w) for w in (wq, wk)]
    before = q.clone(), k.clone()
    outs = rope.apply(q, k, dev(pos), *dw, eps=1e-5)
    axis = None if sections is None else np.repeat(np.arange(axes), sections)
    for x, o, w in ((q, outs[0], wq), (k, outs[1], wk)):
        ref, size = R.turn(host(x), w, 1e-5, pos, freq, axis, interleaved, 1.25)
        within(host(o), ref, R.half_step(dtype, ref) * (1 + 2.0 ** -10) + TURN_ERR * size)
    assert torch.equal(q, before[0]) and torch.equal(k, before[1])
    # one of the two alone, and in place inside the fused rows: the same values
    assert torch.equal(rope.apply(None, k, dev(pos), k_weight=dw[1], eps=1e-5)[1], outs[1])
    rope.apply(q, k, dev(pos), *dw, eps=1e-5, q_out=q, k_out=k)
    assert torch.equal(q, outs[0]) and torch.equal(k, outs[1])


def test_norm_rope_refuses():
    rope = rq.Rope(128, sections=(32, 16, 16))
    q, k, _ = fused(gen(0), 4, 4, 2, torch.float16)
    pos = torch.zeros((3, 4), dtype=torch.int32, device="cuda")
    w = torch.ones(128, device="cuda")
    ok = lambda **o: rope.apply(**{**dict(q=q, k=k, positions=pos, q_weight=w), **o})  # noqa: E731
    ok()
    for bad in (dict(positions=pos[:1].contiguous()), dict(positions=pos.long()), dict(positions=None),
                dict(positions=pos.cpu()), dict(q=q.float(), k=None), dict(k=k.bfloat16()), dict(k=k[:3]),
                dict(q_weight=w.half()), dict(q_weight=w[:64]), dict(q_weight=w.cpu()), dict(q=None, k=None),
                dict(q=q[..., :64]), dict(q=q.transpose(0, 1)), dict(q_out=k), dict(k=k.cpu()),
                dict(q_out=torch.empty(4, 4, 128, device="cuda")), dict(eps=-1.0)):
        with pytest.raises(rq.RQError) as e:
            ok(**bad)
        assert e.value.code == rq.RQ_ERR_INVALID
    for bad in (dict(rotary_dim=12), dict(sections=(32, 31)), dict(scale=0.0), dict(inv_freq=[1.0])):
        with pytest.raises(rq.RQError):
            rq.Rope(**bad)
    e = rope.apply(q[:0], k[:0], pos[:, :0].contiguous())
    assert e[0].shape == (0, 4, 128)


# ------------------------------------------------------------------------------------ append

def make(hq, hkv, P, pages, dtype, batch=4, t=1, fill=0, max_pages=None):
    cache = rq.KVCache(rq.RQ_FP8, 8, hq, hkv, P, pages, None, None, max_batch=batch, max_query_tokens=t,
                       max_pages_per_seq=max_pages, dtype=dtype)
    cache.pages.fill_(fill)
    return cache


def same_cache(cache, ref, slots, key_tol=None):
    """The pool's codes and scales at `slots` against the model's.  key_tol: the keys' relative f32
    error by token [n][H][128] (None: exact inputs, equal codes)."""
    codes, exps = R.unpack(cache.pages.cpu().numpy(), cache.page_size)
    P = cache.page_size
    for kind in (0, 1):
        e = exps[kind].transpose(0, 2, 1).reshape(-1, cache.num_kv_heads)
        assert np.array_equal(e[slots // 16], ref.exps[kind][slots // 16]), "scales"
        got = codes[kind][slots // P, :, slots % P]
        want = ref.codes[kind][slots // 16, :, slots % 16]
        if kind == 1 or key_tol is None:
            assert np.array_equal(got, want, equal_nan=True), f"kind {kind}"
        else:
            diff = got != want
            # another code only where the exact value stands within its error of the two codes' middle
            mid = np.abs((got + want) / 2 - key_tol[0])
            assert (mid[diff] <= key_tol[1][diff]).all() and diff.mean() < 1e-3
            steps = np.maximum(R.step_of(got), R.step_of(want))
            assert (np.abs(got - want) <= steps).all()


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("hkv,P,calls", [
    (1, 16, [[(0, 0, 1)]]),
    (3, 32, [[(0, 0, 5)], [(0, 5, 1), (1, 0, 33)], [(0, 6, 30), (1, 33, 2)]]),
    (8, 16, [[(b, 0, 17 + b) for b in range(4)]] + [[(b, 17 + b + s, 1) for b in range(4)] for s in range(20)]),
    (9, 64, [[(0, 0, 5000)], [(0, 5000, 4900), (1, 0, 3)]]),   # long appends, a start inside a block
    (2, 48, [[(0, 0, 16)], [(0, 9, 3)], [(0, 12, 40)]]),       # a rewind, as after rejected drafts
])
def test_append_codes_and_scales(dtype, hkv, P, calls):
    """(sequence, first position, tokens) of each call.  Magnitudes differ by token, so that scales
    grow inside blocks and old codes are rescaled."""
    dtype, rng = DT[dtype], gen(hkv)
    per = 9920 // P + 1
    table = rng.permutation(4 * per).reshape(4, per)
    cache, ref = make(hkv, hkv, P, 4 * per, dtype), R.Cache(4 * per, hkv, P)
    seen = set()
    for call in calls:
        pos = [(b, p) for b, start, cnt in call for p in range(start, start + cnt)]
        slots = np.array([table[b, p // P] * P + p % P for b, p in pos], np.int32)
        n = len(slots)
        kv = rng.standard_normal((2, n, hkv, 128)) * 2.0 ** rng.integers(-8, 9, (2, n, 1, 1))
        kv[0, :, :, 5] *= 10
        k, v = dev(kv[0], dtype), dev(kv[1], dtype)
        if n > 2:  # padding, in the middle of the call but not of a run
            cut = next((i for i in range(1, n) if pos[i][0] != pos[i - 1][0]), n)
            k, v = (torch.cat((x[:cut], x[:1], x[cut:])) for x in (k, v))
            slots = np.insert(slots, cut, -1).astype(np.int32)
        cache.append(k, v, dev(slots))
        ref.append(host(k), host(v), slots)
        seen |= set(slots[slots >= 0].tolist())
    same_cache(cache, ref, np.array(sorted(seen)))
    assert int(cache.status.item()) == 0


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("n,start,hq,hkv,interleaved,norm", [(1, 3, 4, 2, False, True), (37, 5, 8, 8, True, True),
                                                             (5000, 11, 3, 1, False, False), (4900, 0, 8, 3, False, True)])
def test_append_rope(dtype, n, start, hq, hkv, interleaved, norm):
    dtype, rng, P = DT[dtype], gen(n), 32
    pages = (start + n) // P + 1
    cache, ref = make(hkv, hkv, P, pages, dtype), R.Cache(pages, hkv, P)  # the queries' heads are the call's
    old = dev(rng.standard_normal((start, hkv, 128)), dtype)
    if start:
        cache.append(old, old, torch.arange(start, dtype=torch.int32, device="cuda"))
        ref.append(host(old), host(old), np.arange(start))
    q, k, v = fused(rng, n, hq, hkv, dtype)
    w = 1 + 0.2 * rng.standard_normal((2, 128)).astype(np.float32) if norm else None
    pos = rng.integers(0, 1 << 20, (2, n)).astype(np.int32)
    rope = rq.Rope(128, sections=(40, 24), interleaved=interleaved)
    freq = 10000.0 ** (-2.0 * np.arange(64) / 128)
    axis = np.repeat((0, 1), (40, 24))
    slots = np.arange(start, start + n, dtype=np.int32)
    wq, wk = (dev(w[0]), dev(w[1])) if norm else (None, None)
    out = cache.append_rope(k, v, dev(slots), rope, dev(pos), q=q, q_weight=wq, k_weight=wk)
    assert torch.equal(out, rope.apply(q, None, dev(pos), q_weight=wq)[0])
    turned, size = R.turn(host(k), w[1] if norm else None, 1e-6, pos, freq, axis, interleaved)
    ref.append(turned, host(v), slots)
    down = 2.0 ** -ref.exps[0][slots // 16].astype(float)[..., None]
    same_cache(cache, ref, slots, key_tol=(turned * down, TURN_ERR * size * down))
    assert int(cache.status.item()) == 0


def test_append_not_finite():
    cache = make(2, 2, 16, 2, torch.float16)
    k = torch.ones((3, 2, 128), dtype=torch.float16, device="cuda")
    k[0, 0, 0], k[1, 0, 1], k[2, 0, 2] = float("inf"), float("nan"), -float("inf")
    cache.append(k, torch.ones_like(k), torch.arange(3, dtype=torch.int32, device="cuda"))
    codes, exps = R.unpack(cache.pages.cpu().numpy(), 16)
    assert int(cache.status.item()) == rq.RQ_STATUS_NOT_FINITE
    assert exps[0][0, 0, 0] == R.exponent(1.0) == exps[0][0, 1, 0]
    c = codes[0][0, 0]
    assert c[0, 0] == 448 and np.isnan(c[1, 1]) and c[2, 2] == -448 and c[0, 1] == 256


@pytest.mark.parametrize("slots", [[-1, 32, 0], [2 ** 31 - 1, -5, 1]])
def test_append_skips_padding_and_refuses_slots(slots):
    cache = make(2, 2, 16, 2, torch.bfloat16, fill=0x5A)
    k = torch.ones((3, 2, 128), dtype=torch.bfloat16, device="cuda")
    before = cache.pages.clone()
    cache.append(k, k, torch.tensor(slots, dtype=torch.int32, device="cuda"))
    assert int(cache.status.item()) == rq.RQ_STATUS_BAD_SLOT
    changed = (cache.pages != before).any(-1)
    assert changed.tolist() == [[True, True], [False, False]]
    kept = R.unpack(cache.pages.cpu().numpy(), 16)[0][1][0, 0]  # rows other than the written one
    other = [r for r in range(16) if r != slots[2]]
    if slots[2] == 0:
        assert (kept[other] == R.VALUES[0x5A]).all()


def test_append_refusals():
    cache = make(4, 2, 16, 2, torch.float16)
    planar = rq.KVCache(rq.RQ_PLANAR, 4, 4, 2, 16, 2, np.ones((2, 128)), np.ones((2, 128)), max_batch=1)
    q, k, v = fused(gen(1), 3, 4, 2, torch.float16)
    slots, pos = torch.arange(3, dtype=torch.int32, device="cuda"), torch.arange(3, dtype=torch.int32, device="cuda")
    rope = rq.Rope(128)
    ok = lambda c=cache, **o: c.append_rope(**{**dict(k=k, v=v, slot_mapping=slots, rope=rope, positions=pos, q=q), **o})  # noqa: E731
    ok()
    with pytest.raises(rq.RQError) as e:
        ok(planar)
    assert e.value.code == rq.RQ_ERR_UNSUPPORTED
    for bad in (dict(k=k[:2]), dict(k=k.bfloat16()), dict(v=v[:, :1]), dict(q_out=k.expand(3, 2, 128)),
                dict(slot_mapping=slots.long()), dict(positions=None), dict(k=q), dict(eps=-1.0), dict(v=None),
                dict(q_out=torch.empty_strided((3, 4, 128), (0, 128, 1), dtype=torch.float16, device="cuda"))):
        with pytest.raises(rq.RQError) as e:
            ok(**bad)
        assert e.value.code == rq.RQ_ERR_INVALID, bad
    with pytest.raises(rq.RQError) as e:
        planar.codes()
    assert e.value.code == rq.RQ_ERR_UNSUPPORTED
    with pytest.raises(rq.RQError) as e:
        cache.codebook()
    assert e.value.code == rq.RQ_ERR_UNSUPPORTED


# --------------------------------------------------------------------------------- attention

def wide(B, T, hq, P):
    """Block-table width from which an extend call has its own kernel (narrower, smaller calls share the split-K one)."""
    return 2 ** 23 // (B * T * hq * P) + 1


def filled(rng, hq, hkv, P, lens, dtype, t=1, spread=0, width=0):
    """A cache of sequences of `lens` tokens on random pages; what no token was written to holds NaN
    codes and the largest exponents.  spread: keys and values of blocks differ by up to 2^spread."""
    need = [(int(x) + P - 1) // P for x in lens]
    width = max(max(need) + 1, 2, width)
    pages = sum(need) + 2
    table = np.zeros((len(lens), width), np.int32)
    order = rng.permutation(pages)
    i = 0
    for b, m in enumerate(need):
        table[b, :m] = order[i:i + m]
        i += m
    cache = make(hq, hkv, P, pages, dtype, batch=len(lens), t=t, fill=0xFF, max_pages=width)
    for b, L in enumerate(lens):
        if L == 0:
            continue
        kv = rng.standard_normal((2, L, hkv, 128))
        kv[0, :, :, 7] *= 10
        kv[1] *= 2.0 ** rng.integers(-spread, spread + 1, (L // 16 + 1, 1, 1)).repeat(16, 0)[:L]
        kv[0] *= 2.0 ** rng.integers(-(spread > 0), 1 + (spread > 0), (L // 16 + 1, 1, 1)).repeat(16, 0)[:L]
        pos = np.arange(L)
        slots = (table[b, pos // P] * P + pos % P).astype(np.int32)
        cache.append(dev(kv[0], dtype), dev(kv[1], dtype), dev(slots))
    return cache, table, np.asarray(lens, np.int32)


def model(cache):
    codes, exps = R.unpack(cache.pages.cpu().numpy(), cache.page_size)
    H = cache.num_kv_heads
    return ([c.transpose(0, 2, 1, 3).reshape(-1, 16, H, 128).transpose(0, 2, 1, 3) for c in codes],
            [e.transpose(0, 2, 1).reshape(-1, H) for e in exps])


def check(cache, table, lens, q, out, visible, what):
    codes, exps = model(cache)
    ref, tol = R.attention(q, codes, exps, table, lens, cache.page_size, visible)
    within(host(out), ref, tol + R.half_step(q.dtype, ref) * (1 + 2.0 ** -8), what)
    assert int(cache.status.item()) == 0


CASES = [
    # Hq, Hkv, P, lens, spread
    (32, 8, 16, [1024], 0),
    (8, 8, 16, [0, 1, 15, 16, 17, 31, 33], 0),
    (12, 4, 48, [95, 257, 2, 500], 3),
    (64, 8, 64, [700, 64, 65, 63], 0),
    (40, 2, 32, [333, 1], 6),      # 20 query heads per kv head
    (25, 1, 256, [600, 255, 4097], 2),
    (16, 16, 16, [129] * 9, 0),
]


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("hq,hkv,P,lens,spread", CASES)
def test_decode(dtype, hq, hkv, P, lens, spread):
    rng, dtype = gen(hq * P), DT[dtype]
    cache, table, lens = filled(rng, hq, hkv, P, lens, dtype, spread=spread)
    q = dev(rng.standard_normal((len(lens), 1, hq, 128)), dtype)
    out = cache.decode(q[:, 0].contiguous(), dev(table), dev(lens))
    check(cache, table, lens, q, out[:, None], lambda b, j, p: p <= lens[b] - 1, "decode")
    again = cache.decode(q[:, 0].contiguous(), dev(table), dev(lens))
    assert torch.equal(out, again)


VERIFY = [
    (6, 32, 8, 16, [70, 100, 6, 7, 0], 0), (2, 5, 5, 32, [2, 33], 2), (5, 24, 2, 16, [90, 1033], 0),
    (3, 64, 1, 64, [1500, 3, 64], 3), (64, 4, 4, 16, [64, 200], 0), (17, 1, 1, 16, [17, 300], 0),
]
EXTEND = VERIFY + [
    (300, 32, 8, 16, [300, 555, 1024], 0), (129, 12, 4, 48, [129, 0, 700], 3), (513, 3, 1, 64, [2000], 0),
    (100, 40, 2, 16, [101, 115, 117], 5), (1, 4, 4, 16, [1, 128, 129, 4000], 2), (257, 1, 1, 256, [257, 300, 9000], 0),
]


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("T,hq,hkv,P,lens,spread", VERIFY)
def test_verify(dtype, T, hq, hkv, P, lens, spread):
    rng, dtype = gen(T * hq), DT[dtype]
    cache, table, lens = filled(rng, hq, hkv, P, lens, dtype, t=T, spread=spread)
    q = dev(rng.standard_normal((len(lens), T, hq, 128)), dtype)
    out = cache.verify(q, dev(table), dev(lens))
    check(cache, table, lens, q, out, lambda b, j, p: p <= lens[b] - T + j, "verify")
    assert torch.equal(out, cache.verify(q, dev(table), dev(lens)))


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("own_kernel", [False, True])
@pytest.mark.parametrize("T,hq,hkv,P,lens,spread", EXTEND)
def test_extend(dtype, own_kernel, T, hq, hkv, P, lens, spread):
    rng, dtype = gen(T * hq), DT[dtype]
    width = wide(len(lens), T, hq, P) if own_kernel else 0
    # max_query_tokens is 1: no limit here
    cache, table, lens = filled(rng, hq, hkv, P, lens, dtype, spread=spread, width=width)
    q = dev(rng.standard_normal((len(lens), T, hq, 128)), dtype)
    out = cache.extend(q, dev(table), dev(lens))
    check(cache, table, lens, q, out, lambda b, j, p: p <= lens[b] - T + j, "extend")
    assert torch.equal(out, cache.extend(q, dev(table), dev(lens)))


@pytest.mark.parametrize("call", ["verify", "extend", "extend, own kernel"])
@pytest.mark.parametrize("value", [float("nan"), float("inf")])
def test_what_is_not_finite_reaches_the_rows_that_see_it(call, value):
    """Key and value of new token 3 not finite: rows 0-2 do not see it.  A NaN value shows in its dim
    only, a NaN key in all; infinities are stored as the largest value."""
    T, L, hq = 6, 40, 4
    cache, table, lens = filled(gen(12), hq, 2, 16, [L, 300], torch.float16, t=T,
                                width=wide(2, T, hq, 16) if "own" in call else 0)
    kv = torch.ones((2, 1, 2, 128), dtype=torch.float16, device="cuda")
    kv[1, 0, 0, 37] = value  # value of kv head 0
    kv[0, 0, 1, 5] = value   # key of kv head 1
    at = L - T + 3
    cache.append(kv[0], kv[1], torch.tensor([table[0, at // 16] * 16 + at % 16], dtype=torch.int32, device="cuda"))
    assert int(cache.status.item()) == rq.RQ_STATUS_NOT_FINITE
    q = dev(gen(13).standard_normal((2, T, hq, 128)), torch.float16)
    out = (cache.verify if call == "verify" else cache.extend)(q, dev(table), dev(lens))
    fin = torch.isfinite(out)
    assert fin[1].all() and fin[0, :3].all()
    if value != value:
        want = torch.ones((3, hq, 128), dtype=torch.bool, device="cuda")
        want[:, :2, 37], want[:, 2:] = False, False
        assert torch.equal(fin[0, 3:], want)
    else:
        assert fin.all()


@pytest.mark.parametrize("T,hq,hkv,P,lens", [(7, 32, 8, 16, [7, 40, 300]), (64, 4, 2, 32, [64, 90]), (1, 3, 3, 16, [1, 50])])
def test_tree_verify(T, hq, hkv, P, lens):
    rng = gen(T)
    cache, table, lens = filled(rng, hq, hkv, P, lens, torch.float16, t=T)
    mask = rng.integers(0, 2 ** 63, (len(lens), T), dtype=np.uint64) * 2 + rng.integers(0, 2, (len(lens), T), dtype=np.uint64)
    mask[0, 0] = 0  # an empty prefix and no draft: sees nothing
    q = dev(rng.standard_normal((len(lens), T, hq, 128)), torch.float16)
    out = cache.tree_verify(q, dev(mask.view(np.int64)), dev(table), dev(lens))

    def see(b, j, p):
        i = p - (lens[b] - T)
        return (i < 0) | (mask[b, j] >> np.maximum(i, 0).astype(np.uint64) & np.uint64(1)).astype(bool)
    check(cache, table, lens, q, out, see, "tree verify")
    if T < lens[0] + 1 and lens[0] == T:
        assert (out[0, 0] == 0).all()
    chain = np.array([[(1 << (j + 1)) - 1 for j in range(T)]] * len(lens), np.uint64)
    a = cache.tree_verify(q, dev(chain.view(np.int64)), dev(table), dev(lens))
    assert torch.equal(a, cache.verify(q, dev(table), dev(lens)))


def test_large_scores_and_equal_scores():
    """Scores far apart (one key takes all the weight) and all equal (a mean)."""
    rng = gen(3)
    cache, table, lens = filled(rng, 4, 2, 16, [200, 333], torch.bfloat16)
    q = torch.zeros((2, 1, 4, 128), dtype=torch.bfloat16, device="cuda")
    q[1] = dev(rng.standard_normal((1, 4, 128)) * 300, torch.bfloat16)
    q[1, 0, 0] *= 1e6
    out = cache.decode(q[:, 0].contiguous(), dev(table), dev(lens))
    check(cache, table, lens, q, out[:, None], lambda b, j, p: p <= lens[b] - 1, "decode")


@pytest.mark.parametrize("call", ["verify", "tree", "extend", "extend, own kernel"])
def test_scores_near_the_ends_of_the_range(call):
    """Scores of about -1e32: the one key of half the size takes all the weight.  Scores of minus
    infinity only: a softmax of 0 / 0, where a row that sees nothing is 0."""
    T, lens = 6, [40, 300, 6, 4]
    width = wide(4, T, 4, 16) if "own" in call else 0
    cache, table, lens = filled(gen(20), 4, 2, 16, lens, torch.bfloat16, t=T, width=width)
    want = torch.empty((4, 2, 128), dtype=torch.bfloat16, device="cuda")
    for b, L in enumerate(lens):
        pos = np.arange(L)
        k = torch.ones((L, 2, 128), dtype=torch.bfloat16, device="cuda")
        k[2] = 0.5
        v = dev(gen(21 + b).integers(-8, 9, (L, 2, 128)), torch.bfloat16)
        cache.append(k, v, dev((table[b, pos // 16] * 16 + pos % 16).astype(np.int32)))
        want[b] = v[2]
    q = torch.full((4, T, 4, 128), -1e31, dtype=torch.bfloat16, device="cuda")
    q[:, :, 1] = 0
    q[:, :, 1, 0] = -float("inf")
    if call == "tree":
        mask = torch.full((4, T), 0x3F, dtype=torch.int64, device="cuda")
        mask[2, 0], mask[3, 5], mask[3, 4] = 0, 3, ~63  # bits of drafts that the sequence does not hold
        out = cache.tree_verify(q, mask, dev(table), dev(lens))
        rows = {0: range(6), 1: range(6), 2: range(1, 6), 3: range(4)}
        blind = [(2, 0), (3, 4), (3, 5)]
    else:
        out = (cache.verify if call == "verify" else cache.extend)(q, dev(table), dev(lens))
        rows = {0: range(6), 1: range(6), 2: range(2, 6), 3: range(4, 6)}
        blind = [(3, 0), (3, 1)]
        assert torch.isnan(out[2, :, 1]).all() and torch.isnan(out[3, 2:, 1]).all()
    for b in rows:
        for j in rows[b]:
            for head in (0, 2, 3):
                assert torch.equal(out[b, j, head], want[b, head // 2]), (b, j, head)
            assert torch.isnan(out[b, j, 1]).all()
    for b, j in blind:
        assert (out[b, j] == 0).all(), (b, j)


def test_nan_key_reaches_its_readers_only():
    cache, table, lens = filled(gen(4), 2, 2, 16, [40, 40], torch.float16)
    k = torch.ones((1, 2, 128), dtype=torch.float16, device="cuda")
    k[0, 1, 9] = float("nan")
    cache.append(k, torch.ones_like(k), torch.tensor([table[0, 1] * 16 + 3], dtype=torch.int32, device="cuda"))
    q = torch.ones((2, 2, 128), dtype=torch.float16, device="cuda")
    out = cache.decode(q, dev(table), dev(lens))
    assert torch.isfinite(out[0, 0]).all() and torch.isnan(out[0, 1]).all() and torch.isfinite(out[1]).all()
    short = cache.decode(q, dev(table), dev(np.array([19, 40], np.int32)))  # it stands at position 19, unseen
    assert torch.isfinite(short).all()


def test_decode_step_equals_append_and_decode():
    rng = gen(5)
    lens = [1, 16, 17, 100, 0]
    a, table, ln = filled(rng, 8, 2, 16, [0, 15, 16, 99, 0], torch.bfloat16)
    b = make(8, 2, 16, a.num_pages, torch.bfloat16, batch=5, max_pages=table.shape[1])
    used = set(table[1, :1]) | set(table[2, :1]) | set(table[3, :7])
    table[0, 0], table[2, 1] = [p for p in range(a.num_pages) if p not in used]  # pages for the new tokens
    b.pages.copy_(a.pages)
    lens = np.array(lens, np.int32)
    k, v = (dev(rng.standard_normal((5, 2, 128)) * 3, torch.bfloat16) for _ in range(2))
    q = dev(rng.standard_normal((5, 8, 128)), torch.bfloat16)
    got = a.decode_step(q, k, v, dev(table), dev(lens))
    at = np.maximum(lens - 1, 0)
    slots = np.where(lens > 0, table[np.arange(5), at // 16] * 16 + at % 16, -1).astype(np.int32)
    b.append(k, v, dev(slots))
    assert torch.equal(got, b.decode(q, dev(table), dev(lens)))
    assert torch.equal(a.pages, b.pages) and int(a.status.item()) == 0


@pytest.mark.parametrize("fault", ["page", "negative page", "length", "negative length", "short"])
@pytest.mark.parametrize("call", ["decode", "verify", "extend", "extend, own kernel", "step"])
def test_faults_are_reported_and_clamped(fault, call):
    if fault == "short" and call in ("decode", "step"):
        return
    cache, table, lens = filled(gen(6), 4, 2, 16, [50, 40], torch.float16, t=3,
                                width=wide(2, 3, 4, 16) if "own" in call else 0)
    want = rq.RQ_STATUS_BAD_PAGE if "page" in fault else rq.RQ_STATUS_BAD_LEN
    if "page" in fault:
        table[0, 3] = 2 ** 31 - 1 if fault == "page" else -7  # the newest token's
    else:
        lens[0] = dict([("length", 16 * table.shape[1] + 1), ("negative length", -1), ("short", 2)])[fault]
    good = lens[1]
    q = dev(gen(7).standard_normal((2, 3, 4, 128)), torch.float16)
    k = torch.ones((2, 2, 128), dtype=torch.float16, device="cuda")
    fn = dict(decode=lambda: cache.decode(q[:, 0].contiguous(), dev(table), dev(lens))[:, None],
              step=lambda: cache.decode_step(q[:, 0].contiguous(), k, k, dev(table), dev(lens))[:, None],
              verify=lambda: cache.verify(q, dev(table), dev(lens)),
              extend=lambda: cache.extend(q, dev(table), dev(lens)))[call.split(",")[0]]
    out = fn()
    torch.cuda.synchronize()
    assert int(cache.status.item()) == want
    cache.status.zero_()
    if call != "step":
        T = out.shape[1]
        lens2 = np.array([0, good], np.int32)
        check(cache, table, lens2, q[:, :T], torch.cat((torch.zeros_like(out[:1]), out[1:])),
              lambda b, j, p: p <= lens2[b] - T + j, call)


def test_refusals_of_attention():
    cache, table, lens = filled(gen(8), 4, 2, 16, [50, 40], torch.bfloat16, t=2)
    q = torch.zeros((2, 3, 4, 128), dtype=torch.bfloat16, device="cuda")
    with pytest.raises(rq.RQError) as e:
        cache.verify(q, dev(table), dev(lens))
    assert e.value.code == rq.RQ_ERR_CAPACITY
    with pytest.raises(AssertionError):
        cache.verify(q[:, :2].contiguous().half(), dev(table), dev(lens))
    with pytest.raises(rq.RQError):
        rq.KVCache(rq.RQ_FP8, 8, 4, 2, 16, 2, None, None, max_batch=1, dtype=torch.float32)
    with pytest.raises(rq.RQError):
        rq.KVCache(rq.RQ_FP8, 8, 4, 2, 16, 2, None, None, max_batch=1,
                   pages=torch.zeros((2, 2, 4111), dtype=torch.uint8, device="cuda"))
    empty = cache.decode(q[:0, 0].contiguous(), dev(table)[:0], dev(lens)[:0])
    assert empty.shape == (0, 4, 128)


# -------------------------------------------------------------------------- as they are used

def test_a_model_s_steps_together():
    """A chunk appended and attended, three decode steps of it captured in a graph and replayed on a
    side stream, against the definitions on the cache as it stands."""
    rng, hq, hkv, P, B = gen(9), 8, 2, 16, 3
    start = [40, 7, 100]
    cache, table, lens = filled(rng, hq, hkv, P, start, torch.bfloat16, t=1)
    need = [(s + 20 + P - 1) // P for s in start]
    cache2 = rq.KVCache(rq.RQ_FP8, 8, hq, hkv, P, sum(need), None, None, max_batch=B, max_pages_per_seq=max(need),
                        dtype=torch.bfloat16)
    table = np.zeros((B, max(need)), np.int32)
    o = 0
    for b, m in enumerate(need):
        table[b, :m] = np.arange(o, o + m)
        o += m
    rope, w = rq.Rope(128), dev(np.ones(128, np.float32))
    T = max(start)  # chunks, padded to the longest with slot -1 in front
    qkv = dev(rng.standard_normal((B, T, hq + 2 * hkv, 128)), torch.bfloat16)
    pos = np.stack([np.arange(T) - (T - s) for s in start])
    slots = np.where(pos >= 0, np.take_along_axis(table, np.maximum(pos, 0) // P, 1) * P + pos % P, -1).astype(np.int32)
    x = qkv.view(B * T, hq + 2 * hkv, 128)
    q = cache2.append_rope(x[:, hq:hq + hkv], x[:, hq + hkv:], dev(slots.reshape(-1)), rope,
                           dev(pos.reshape(-1).astype(np.int32)), q=x[:, :hq], q_weight=w, k_weight=w)
    # one sequence's chunk attends by itself
    b = 2
    out = cache2.extend(q.view(B, T, hq, 128)[b:b + 1].contiguous(), dev(table[b:b + 1]), dev(np.array([T], np.int32)))
    check(cache2, table[b:], [T], q.view(B, T, hq, 128)[b:], out, lambda _, j, p: p <= j, "chunk")

    # decode steps: buffers that the graph reads
    step_qkv = dev(rng.standard_normal((B, hq + 2 * hkv, 128)), torch.bfloat16)
    d_pos, d_slots, d_lens = (torch.zeros(B, dtype=torch.int32, device="cuda") for _ in range(3))
    d_table = dev(table)
    qs, outs = torch.empty((B, hq, 128), dtype=torch.bfloat16, device="cuda"), torch.empty((B, hq, 128), dtype=torch.bfloat16, device="cuda")

    def step():
        cache2.append_rope(step_qkv[:, hq:hq + hkv], step_qkv[:, hq + hkv:], d_slots, rope, d_pos, q=step_qkv[:, :hq],
                           q_weight=w, k_weight=w, q_out=qs)
        cache2.decode(qs, d_table, d_lens, out=outs)

    def feed(i):
        p = np.array(start, np.int32) + i
        d_pos.copy_(dev(p))
        d_slots.copy_(dev((table[np.arange(B), p // P] * P + p % P).astype(np.int32)))
        d_lens.copy_(dev(p + 1))
        step_qkv.copy_(dev(gen(100 + i).standard_normal((B, hq + 2 * hkv, 128)), torch.bfloat16))
        return p + 1
    side = torch.cuda.Stream()
    ln = feed(0)
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    side.synchronize()
    check(cache2, table, ln, qs[:, None].clone(), outs[:, None], lambda b, j, p: p <= ln[b] - 1, "eager step")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for i in range(1, 4):
        ln = feed(i)
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            graph.replay()
        side.synchronize()
        check(cache2, table, ln, qs[:, None].clone(), outs[:, None], lambda b, j, p: p <= ln[b] - 1, f"step {i}")


def test_long_appends_equal_short_ones():
    """Three sequences of 8,229 tokens in one call, their starts inside blocks, against calls that end at
    block ends: the same bytes, and the queries as Rope.apply turns them."""
    rng, hq, hkv, P = gen(31), 5, 2, 32
    n, starts = [5003, 9, 3217], [7, 0, 21]
    per = 5024 // P + 1
    a, b = (make(hkv, hkv, P, 3 * per, torch.bfloat16) for _ in range(2))
    table = rng.permutation(3 * per).reshape(3, per)
    pos = np.concatenate([np.arange(s, s + m) for s, m in zip(starts, n)])
    seq = np.repeat(np.arange(3), n)
    slots = (table[seq, pos // P] * P + pos % P).astype(np.int32)
    q, k, v = fused(rng, sum(n), hq, hkv, torch.bfloat16)
    rope, w = rq.Rope(128), dev((1 + 0.2 * rng.standard_normal(128)).astype(np.float32))
    d_pos, d_slots = dev(pos.astype(np.int32)), dev(slots)
    out = a.append_rope(k, v, d_slots, rope, d_pos, q=q, q_weight=w, k_weight=w)
    assert torch.equal(out, rope.apply(q, None, d_pos, q_weight=w)[0])
    at = 0
    while at < len(pos):
        to = min(at + 1000, len(pos))
        while to < len(pos) and pos[to] % 16 and seq[to] == seq[to - 1]:
            to -= 1
        part = b.append_rope(k[at:to], v[at:to], d_slots[at:to], rope, d_pos[at:to], q=q[at:to], q_weight=w, k_weight=w)
        assert torch.equal(part, out[at:to])
        at = to
    assert torch.equal(a.pages, b.pages) and int(a.status.item()) == 0


def test_tokens_of_many_sequences():
    """One token each of 2,500 sequences, in one call of either kind and in calls of 100."""
    rng, B = gen(32), 2500
    caches = [make(1, 1, 16, B, torch.float16, batch=B) for _ in range(3)]
    off = rng.integers(0, 16, B)
    slots = (rng.permutation(B) * 16 + off).astype(np.int32)
    lens = np.where(np.arange(B) % 7 == 3, 0, off + 1).astype(np.int32)
    first = [dev(rng.standard_normal((16 * B, 1, 128)), torch.float16) for _ in range(2)]
    k, v = (dev(rng.standard_normal((B, 1, 128)) * 2.0 ** rng.integers(-4, 5, (B, 1, 1)), torch.float16) for _ in range(2))
    q = dev(rng.standard_normal((B, 1, 128)), torch.float16)
    table = dev((slots // 16)[:, None].astype(np.int32))
    given = dev(np.where(lens > 0, slots, -1).astype(np.int32))
    for c in caches:
        c.append(*first, torch.arange(16 * B, dtype=torch.int32, device="cuda"))
    caches[0].append(k, v, given)
    out = caches[1].decode_step(q, k, v, table, dev(lens))
    for i in range(0, B, 100):
        caches[2].append(k[i:i + 100].contiguous(), v[i:i + 100].contiguous(), given[i:i + 100].contiguous())
    assert torch.equal(caches[0].pages, caches[2].pages) and torch.equal(caches[1].pages, caches[2].pages)
    assert torch.equal(out, caches[0].decode(q, table, dev(lens)))
    check(caches[0], table.cpu().numpy(), lens, q[:, None], out[:, None], lambda b, j, p: p <= lens[b] - 1, "decode")


@pytest.mark.parametrize("B,T,hq", [(700, 1, 8), (300, 2, 8)])
def test_many_sequences(B, T, hq):
    rng = gen(B)
    lens = np.where(rng.random(B) < 0.1, 0, rng.integers(T, 300, B))
    cache, table, lens = filled(rng, hq, 1, 32, lens, torch.bfloat16, t=T)
    q = dev(rng.standard_normal((B, T, hq, 128)), torch.bfloat16)
    check(cache, table, lens, q, cache.verify(q, dev(table), dev(lens)), lambda b, j, p: p <= lens[b] - T + j, "verify")


def test_many_rows_of_a_kv_head():
    rng = gen(33)  # 64 drafts x 64 heads of one kv head: 512 groups of 8 rows
    cache, table, lens = filled(rng, 64, 1, 16, [64, 333], torch.float16, t=64)
    q = dev(rng.standard_normal((2, 64, 64, 128)), torch.float16)
    check(cache, table, lens, q, cache.verify(q, dev(table), dev(lens)), lambda b, j, p: p <= lens[b] - 64 + j, "verify")


def test_two_contexts_at_once():
    """Calls of two contexts on two streams, eagerly and replayed from two graphs."""
    sets = []
    for i in range(2):
        cache, table, lens = filled(gen(40 + i), 16, 4, 16, [3000, 70 + i, 1200], torch.bfloat16, t=9, width=300)
        q = dev(gen(42 + i).standard_normal((3, 9, 16, 128)), torch.bfloat16)
        calls = [lambda o, c=cache, a=(q, dev(table), dev(lens)): c.verify(*a, out=o),
                 lambda o, c=cache, a=(q.repeat(1, 60, 1, 1)[:, :70].contiguous(), dev(table), dev(lens)): c.extend(*a, out=o)]
        outs = [torch.empty((3, t, 16, 128), dtype=torch.bfloat16, device="cuda") for t in (9, 70)]
        for call, o in zip(calls, outs):
            call(o)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        again = [torch.empty_like(o) for o in outs]
        with torch.cuda.graph(graph):
            for call, o in zip(calls, again):
                call(o)
        sets.append((calls, outs, again, graph, torch.cuda.Stream()))
    for replay in (False, True):
        for calls, outs, again, graph, stream in sets:
            for o in again:
                o.zero_()
            stream.wait_stream(torch.cuda.current_stream())
        for _ in range(10):
            for calls, outs, again, graph, stream in sets:
                with torch.cuda.stream(stream):
                    if replay:
                        graph.replay()
                    else:
                        for call, o in zip(calls, again):
                            call(o)
        torch.cuda.synchronize()
        for calls, outs, again, graph, stream in sets:
            assert all(torch.equal(a, o) for a, o in zip(again, outs))


def test_offsets_past_32_bits():
    """Pages past 4 GiB of the pool: append, then decode and extend over them."""
    hkv, P, pages = 8, 256, 8300  # 526 KB a page of all heads
    cache = make(hkv, hkv, P, pages, torch.float16, batch=1, max_pages=2)
    table, L = np.array([[pages - 1, pages - 2]], np.int32), 300
    rng = gen(11)
    pos = np.arange(L)
    slots = (table[0, pos // P] * P + pos % P).astype(np.int32)
    k, v = (dev(rng.standard_normal((L, hkv, 128)), torch.float16) for _ in range(2))
    cache.append(k, v, dev(slots))
    small = make(hkv, hkv, P, 2, torch.float16, batch=1, max_pages=2)
    small.append(k, v, dev(pos.astype(np.int32)))
    assert torch.equal(cache.pages[pages - 1], small.pages[0]) and torch.equal(cache.pages[pages - 2], small.pages[1])
    q = dev(rng.standard_normal((1, 290, hkv, 128)), torch.float16)
    ln, near = dev(np.array([L], np.int32)), dev(np.array([[0, 1]], np.int32))
    assert torch.equal(cache.extend(q[:, :20].contiguous(), dev(table), ln), small.extend(q[:, :20].contiguous(), near, ln))
    far = cache, np.pad(table, ((0, 0), (0, 20))), small, np.pad(near.cpu().numpy(), ((0, 0), (0, 20)))
    for c in (cache, small):  # contexts of wide tables over the same pools: the extend kernel of its own
        c.wide = rq.KVCache(rq.RQ_FP8, 8, hkv, hkv, P, c.num_pages, None, None, max_batch=1, max_pages_per_seq=22, pages=c.pages)
    assert torch.equal(far[0].wide.extend(q, dev(far[1]), ln), far[2].wide.extend(q, dev(far[3]), ln))
    assert torch.equal(cache.decode(q[:, 0].contiguous(), dev(table), ln), small.decode(q[:, 0].contiguous(), near, ln))
