"""Latent attention on the GPU against the float64 definitions of latent_ref: the append, attention in the absorbed form,
reading back, and attention in the expanded form."""
import math

import numpy as np
import pytest
import torch

from rotation_quantized_kv_rq_gb300 import rq
from tests import block_ref as R
from tests import latent_ref as L

pytestmark = pytest.mark.gpu

DT = {"f16": torch.float16, "bf16": torch.bfloat16}
# relative to |a| + |b| of a pair: the angle rounded to 24 bits within an eighth of a turn (pi / 4 * 2^-24), sincospif (2^-23), the
# rotation's three roundings
TURN_ERR = np.pi / 4 * 2.0 ** -24 + 2.0 ** -23 + 3 * 2.0 ** -24
# the mean of 512 squares: sums of 16 in a lane and five steps over the warp, 21 roundings halved by the root, the root, the factor
# and the product
NORM_ERR = 15 * 2.0 ** -24


def gen(seed):
    return np.random.default_rng(seed)


def dev(x, dtype=None):
    t = torch.from_numpy(np.ascontiguousarray(x)).cuda()
    return t if dtype is None else t.to(dtype)


def host(t):
    return t.detach().cpu().double().numpy()


def within(got, ref, tol, what=""):
    err = np.abs(got - ref)
    bad = ~(err <= tol)
    assert not bad.any(), f"{what}: {bad.sum()} of {bad.size} off, worst {np.nanmax(err / np.maximum(tol, 1e-300)):.3g} of the tolerance"


def int32(x):
    return dev(np.asarray(x, np.int32))


def make(heads, P, pages, dtype, batch=8, t=1, **over):
    return rq.LatentCache(heads, P, pages, max_batch=batch, max_query_tokens=t, dtype=dtype, **over)


# ------------------------------------------------------------------------------------ append

def check_pool(cache, before, want, what):
    """The pool's tokens against want {slot: (codes, position part, exponent byte)} with tolerances (codes' exact values
    and error, parts' tolerance), or None for NaN; every other byte as before."""
    P, dtype = cache.page_size, cache.dtype
    now = cache.pages.cpu().numpy()
    codes, part, byte = L.unpack(now, P, dtype)
    rest = now.copy()
    for slot, w in want.items():
        n, r = divmod(slot, P)
        for at in (L.code_place(P, r, L.DIM), L.part_place(P, r, L.PART), L.part_place(P, r, L.PART) + 1, 640 * P + r):
            rest[n, at] = before[n, at]
        if w is None:
            assert byte[slot] == 255 and not codes[slot].any() and not part[slot].any(), what
            continue
        (c, c_err), (p, p_tol), e = w
        assert byte[slot] == e + 127, f"{what}: exponent of slot {slot}"
        exact = c * 2.0 ** -e
        ref = R.round_e4m3(exact)
        diff = codes[slot] != ref
        mid = np.abs((codes[slot] + ref) / 2 - exact)  # another code only next to the middle of two
        assert (mid[diff] <= c_err[diff] * 2.0 ** -e).all(), f"{what}: codes of slot {slot}"
        within(part[slot], np.clip(p * 2.0 ** -e, -32768, 32768), p_tol * 2.0 ** -e, what)
    assert np.array_equal(rest, before), f"{what}: bytes outside the tokens"


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("n,heads,P,rotary,interleaved,norm,far", [
    (1, 1, 16, 64, True, True, 100),
    (5, 3, 48, 64, False, True, 1 << 20),
    (33, 128, 64, 64, True, False, 1 << 15),
    (130, 17, 256, 32, False, True, 2 ** 31 - 1),
    (64, 5, 16, 8, True, True, 1 << 17),
    (3, 2, 32, 40, False, False, 1000),
    (7, 0, 16, 0, False, True, 10),
])
def test_append(dtype, n, heads, P, rotary, interleaved, norm, far):
    dtype, rng = DT[dtype], gen(n + heads)
    pages = (n + P - 1) // P + 2
    cache = make(max(heads, 1), P, pages, dtype)
    before = rng.integers(0, 256, tuple(cache.pages.shape)).astype(np.uint8)
    cache.pages.copy_(torch.from_numpy(before))
    down = dev(rng.standard_normal((n, 512 + 64 + 8)) * 2.0 ** rng.uniform(-3, 3, (n, 1)), dtype)
    c, k_pe = down[:, :512], down[:, 512:576]
    q = dev(rng.standard_normal((n, max(heads, 1), 192)), dtype)
    q_pe = q[..., 128:] if heads else None
    slots = rng.permutation(pages * P)[:n]
    pos = rng.integers(-far, far, n).astype(np.int32)
    w = (1 + 0.2 * rng.standard_normal(512)).astype(np.float32) if norm else None
    freq = 10000.0 ** (-2.0 * np.arange(rotary // 2) / max(rotary, 1))
    rope = rq.Rope(rotary, interleaved=interleaved, scale=1.25) if rotary else None
    call = dict(rope=rope, positions=dev(pos) if rotary else None, weight=None if w is None else dev(w), eps=1e-5)
    turned = cache.append(c, k_pe, int32(slots), q_pe=q_pe, **call)
    x = host(c)
    if norm:
        x = x / np.sqrt((x * x).mean(-1, keepdims=True) + 1e-5) * w.astype(np.float64)
    p, size = R.turn(host(k_pe)[:, None], None, 0, pos[None], freq, None, interleaved, 1.25)
    p, size = p[:, 0], size[:, 0]
    want = {}
    for i, s in enumerate(slots):
        e = L.exponent(np.abs(x[i]).max(), np.abs(p[i]).max())
        p_tol = R.half_step(dtype, p[i] * 2.0 ** -e) * 2.0 ** e * (1 + 2.0 ** -10) + TURN_ERR * size[i]
        want[int(s)] = (x[i], NORM_ERR * np.abs(x[i]) if norm else np.zeros(512)), (p[i], p_tol), e
    check_pool(cache, before, want, "append")
    assert int(cache.status.item()) == 0
    if heads:
        ref, size = R.turn(host(q_pe), None, 0, pos[None], freq, None, interleaved, 1.25)
        within(host(turned), ref, R.half_step(dtype, ref) * (1 + 2.0 ** -10) + TURN_ERR * size, "queries")
        rest = q[..., :128].clone()
        again = cache.append(c, k_pe, int32(slots), q_pe=q_pe, q_pe_out=q_pe, **call)
        assert again is q_pe and torch.equal(q_pe, turned) and torch.equal(q[..., :128], rest)
    pool = cache.pages.clone()
    cache.pages.copy_(torch.from_numpy(before))
    cache.append(c, k_pe, int32(slots), **call)
    assert torch.equal(cache.pages, pool)


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_append_range_and_faults(dtype):
    """Zeros, subnormals, the borders of a scale, magnitudes past the largest scale, infinities and NaN, padding and slots past
    the pool; without norm and rotation the codes are exact."""
    dtype, P, rng = DT[dtype], 16, gen(5)
    rows = np.zeros((12, 576))
    rows[1, :512] = rng.standard_normal(512)
    rows[2, 3], rows[2, 4] = 448.0, 447.0
    rows[3, 3] = 449.0 if dtype == torch.float16 else 450.0
    rows[4, 512], rows[4, 0] = 32768.0, 1.0
    rows[5, 512], rows[5, 0] = 32768.0 + (32.0 if dtype == torch.float16 else 256.0), 1.0
    rows[6, :] = 2.0 ** -24
    rows[7, 511] = np.inf
    rows[8, 575] = np.nan
    rows[9, :512] = rng.standard_normal(512) * 1e4
    if dtype == torch.bfloat16:
        rows[10, 5], rows[10, 6], rows[10, 520] = 2.0 ** 100, 1e-30, -2.0 ** 90
    t = dev(rows, dtype)
    slots = np.arange(12) + 9
    slots[11] = -1
    cache = make(1, P, 2, dtype)
    cache.append(t[:, :512], t[:, 512:], int32(slots))
    want, x = {}, host(t)
    for i in range(11):
        c, p = x[i, :512], x[i, 512:]
        tok = L.coded(c, p, dtype)
        if tok is not None:
            e = tok[2]
            # a value past the largest scale is stored as the largest there is
            c = np.clip(c, -448 * 2.0 ** e, 448 * 2.0 ** e)
            tok = (c, np.zeros(512)), (p, R.half_step(dtype, p * 2.0 ** -e) * 2.0 ** e), e
        want[int(slots[i])] = tok
    check_pool(cache, np.zeros((2, 641 * P), np.uint8), want, "range")
    bits = rq.RQ_STATUS_NOT_FINITE | (rq.RQ_STATUS_NORM_OVERFLOW if dtype == torch.bfloat16 else 0)
    assert int(cache.status.item()) == bits
    cache.status.zero_()
    before = cache.pages.clone()
    cache.append(t[:1, :512], t[:1, 512:], int32([2 * P]))
    assert int(cache.status.item()) == rq.RQ_STATUS_BAD_SLOT and torch.equal(cache.pages, before)
    cache.append(t[:0, :512], t[:0, 512:], int32([]))


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_append_norm_of_rows_apart(dtype):
    """With the norm: a row of zeros, one value in a row, values far apart, and (bf16) squares past float32's range, which are not
    finite."""
    dtype, P = DT[dtype], 16
    rows = np.zeros((4, 576))
    rows[1, 7] = -3.0
    rows[2, :512] = 2.0 ** -10
    rows[2, 100] = 4096.0
    rows[3, :512] = 1.0 if dtype == torch.float16 else 2.0 ** 100
    t, w, eps = dev(rows, dtype), dev(np.full(512, 1.5), torch.float32), 1e-6
    cache = make(1, P, 1, dtype)
    before = cache.pages.cpu().numpy().copy()
    cache.append(t[:, :512], t[:, 512:], int32([3, 0, 9, 15]), weight=w, eps=eps)
    x = host(t)[:, :512]
    x = x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * 1.5
    want = {}
    for i, s in enumerate((3, 0, 9, 15)):
        e = L.exponent(np.abs(x[i]).max(), 0.0)
        want[s] = (x[i], NORM_ERR * np.abs(x[i])), (np.zeros(64), np.zeros(64)), e
    if dtype == torch.bfloat16:
        want[15] = None
    check_pool(cache, before, want, "norm")
    assert int(cache.status.item()) == (rq.RQ_STATUS_NOT_FINITE if dtype == torch.bfloat16 else 0)


def test_append_refuses():
    cache = make(4, 16, 4, torch.float16)
    x = torch.zeros(6, 576, dtype=torch.float16, device="cuda")
    q = torch.zeros(6, 4, 192, dtype=torch.float16, device="cuda")
    pos = torch.zeros(6, dtype=torch.int32, device="cuda")
    rope = rq.Rope(64)
    w = torch.ones(512, device="cuda")
    ok = lambda **o: cache.append(**{**dict(c=x[:, :512], k_pe=x[:, 512:], slot_mapping=int32(range(6)), rope=rope,  # noqa: E731
                                            positions=pos, weight=w, q_pe=q[..., 128:]), **o})
    ok()
    for bad in (dict(c=x[:, :256]), dict(c=x[:5, :512]), dict(c=x[:, :512].float()), dict(c=x[:, :512].cpu()),
                dict(c=x[:, 4:516]), dict(k_pe=x[:, 510:574]), dict(k_pe=x[:, 512:544]), dict(slot_mapping=pos.long()),
                dict(slot_mapping=pos[:5]), dict(slot_mapping=pos.cpu()), dict(positions=None), dict(positions=pos[:5]),
                dict(positions=pos.long()), dict(weight=w.half()), dict(weight=w[:256]), dict(weight=w.cpu()), dict(eps=-1.0),
                dict(eps=math.inf), dict(eps=math.nan), dict(rope=rq.Rope(128)), dict(q_pe=q), dict(q_pe=q[:5, :, 128:]),
                dict(q_pe=q[..., 128:].bfloat16()), dict(q_pe=None, q_pe_out=q[..., 128:]), dict(q_pe_out=q[:, :2, 128:]),
                dict(q_pe_out=q.view(6, 4, 192)[..., 120:184]), dict(q_pe_out=q[..., 64:128]),
                dict(q_pe=q[:, :1, 128:].expand(6, 4, 64)), dict(q_pe=q[..., 124:188]),
                dict(q_pe=x[:, None, 448:512], q_pe_out=x[:, None, 448:512])):
        with pytest.raises(rq.RQError) as e:
            ok(**bad)
        assert e.value.code == rq.RQ_ERR_INVALID, bad.keys()
    for bad in (dict(page_size=24), dict(num_heads=0), dict(dtype=torch.float32), dict(pages=torch.zeros(4, 641 * 16)),
                dict(pages=torch.zeros(4, 640 * 16, dtype=torch.uint8, device="cuda"))):
        with pytest.raises(rq.RQError):
            rq.LatentCache(**{**dict(num_heads=4, page_size=16, num_pages=4, max_batch=1), **bad})


def test_append_in_place_beside_the_latents():
    """Queries, latents and position parts in one buffer, the queries turned in place between them."""
    rng, n, heads = gen(8), 9, 3
    x = dev(rng.standard_normal((n, heads * 192 + 576)), torch.bfloat16)
    q = x[:, :heads * 192].unflatten(1, (heads, 192))[..., 128:]
    pos = int32(rng.integers(0, 1000, n))
    rope = rq.Rope(64, interleaved=True)
    caches = [make(heads, 16, 2, torch.bfloat16) for _ in range(2)]
    c, pe = x[:, heads * 192:heads * 192 + 512], x[:, heads * 192 + 512:]
    apart = caches[0].append(c.clone(), pe.clone(), int32(range(n)), rope, pos, q_pe=q.clone())
    caches[1].append(c, pe, int32(range(n)), rope, pos, q_pe=q, q_pe_out=q)
    assert torch.equal(q, apart) and torch.equal(caches[0].pages, caches[1].pages)


# --------------------------------------------------------------------------- the absorbed form

class Case:
    """Sequences over a pool in a random order of pages; bytes of no sequence are garbage."""

    def __init__(self, seed, lens, T, heads, P, dtype, sm_scale=0.0, gain=1.0, spread=1.0):
        rng = gen(seed)
        self.lens, self.T, self.heads, self.P, self.dtype = np.asarray(lens, np.int32), T, heads, P, dtype
        B = len(lens)
        width = max(1, int(np.maximum(self.lens, 0).max() + P - 1) // P + 1)
        need = (np.maximum(self.lens, 0) + P - 1) // P
        total = int(need.sum()) + 2
        order = rng.permutation(total)
        self.table = np.full((B, width), order[-1], np.int32)
        at = 0
        pages = L.fill(P, total, dtype, rng, garbage=True)
        for b in range(B):
            n = int(self.lens[b])
            self.table[b, :need[b]] = order[at:at + need[b]]
            at += need[b]
            if n > 0:
                slots = self.slots(b, np.arange(n))
                L.put(pages, P, slots, rng.standard_normal((n, 512)) * 2.0 ** rng.uniform(-spread, spread, (n, 1)),
                      2 * rng.standard_normal((n, 64)), dtype)
        self.pages = pages
        self.scale = sm_scale or 192 ** -0.5
        self.q_c = (gain * dev(rng.standard_normal((heads, B * T, 512)), torch.float64)).to(dtype)  # head after head
        self.q_c = self.q_c.transpose(0, 1).unflatten(0, (B, T))
        self.q_pe = (gain * dev(rng.standard_normal((B, T, heads, 192)), torch.float64)).to(dtype)[..., 128:]
        self.cache = make(heads, P, total, dtype, batch=B, t=T, sm_scale=sm_scale, max_pages_per_seq=width)
        self.load()

    def slots(self, b, pos):
        return self.table[b, pos // self.P].astype(np.int64) * self.P + pos % self.P

    def load(self):
        self.cache.pages.copy_(torch.from_numpy(self.pages))

    def run(self, mask=None, **over):
        a = dict(q_c=self.q_c, q_pe=self.q_pe, block_table=dev(self.table), seq_lens=dev(self.lens))
        a.update(over)
        if mask is not None:
            return self.cache.tree_verify(tree_mask=dev(mask), **a)
        return self.cache.verify(**a)

    def check(self, out, mask=None, what=""):
        see = L.chain(self.T) if mask is None else L.tree(mask, self.T)
        ref, tol = L.attention(host(self.q_c), host(self.q_pe), self.pages, self.table, self.lens, self.P, see, self.scale, self.dtype)
        within(host(out), ref, tol + R.half_step(self.dtype, ref) * (1 + 2.0 ** -8), what)


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("lens,T,heads,P", [
    ([1], 1, 1, 16),
    ([0, 1, 2, 17, 255, 256, 257], 1, 16, 16),
    ([700, 1, 513], 1, 128, 64),
    ([300, 64, 65], 3, 5, 48),
    ([1000, 4, 259], 4, 40, 32),          # 160 rows: two row tiles
    ([130, 40, 511], 6, 128, 256),        # six row tiles, row tiles that start inside a token's heads
    ([2000], 33, 20, 16),
    ([3001], 1, 130, 16),                 # more heads than a tile has rows
    ([90, 20000], 1, 8, 64),
    ([1, 1, 1], 1, 64, 16),
])
def test_attention(dtype, lens, T, heads, P):
    case = Case(len(lens) + heads, lens, T, heads, P, DT[dtype])
    out = case.run()
    case.check(out)
    assert int(case.cache.status.item()) == 0
    assert torch.equal(out, case.run()), "repeated calls give the same bits"
    if T == 1:
        got = case.cache.decode(case.q_c[:, 0], case.q_pe[:, 0], dev(case.table), dev(case.lens))
        assert torch.equal(got, out[:, 0])


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("lens,T,heads,P", [([13, 500, 77], 13, 20, 32), ([64, 300], 64, 3, 16), ([2], 2, 1, 16), ([9000, 260], 7, 16, 64),
                                            ([500, 40, 6], 6, 5, 16), ([2000, 31], 16, 2, 32), ([1025], 20, 3, 64)])
def test_tree(dtype, lens, T, heads, P):
    """Random trees, with a row that sees no draft and, in a sequence of drafts only, a row that sees nothing."""
    case = Case(T, lens, T, heads, P, DT[dtype])
    rng = gen(T)
    mask = np.zeros((len(lens), T), np.uint64)
    for b in range(len(lens)):
        for j in range(1, T):
            up = int(rng.integers(-1, j))
            mask[b, j] = (mask[b, up] if up >= 0 else np.uint64(0)) | np.uint64(1 << j)
    mask[:, 1:2] |= np.uint64(1 << min(63, T + 3))  # bits past the drafts mean nothing
    out = case.run(mask.view(np.int64))
    case.check(out, mask)
    if lens[0] == T:
        assert not out[0, 0].any()
    full = np.array([[(1 << (j + 1)) - 1 for j in range(T)]] * len(lens), np.uint64)
    assert torch.equal(case.run(full.view(np.int64)), case.run()), "a chain as a tree"


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("heads", [1, 16, 33, 128])
def test_attention_over_many_tiles(dtype, heads):
    """Many tiles to a pair of SMs, whose second SM may have no rows: the tokens over and over, which changes no softmax."""
    case = Case(5, [2048], 1, heads, 64, DT[dtype])
    times, batch = 12, 40
    cache = make(heads, 64, case.pages.shape[0], DT[dtype], batch=batch, max_pages_per_seq=32 * times)
    cache.pages.copy_(case.cache.pages)
    table = dev(np.tile(case.table[:, :32], (batch, times)))
    every = lambda x: x.expand(batch, -1, -1, -1).contiguous()  # noqa: E731
    out = cache.verify(every(case.q_c), every(case.q_pe), table, int32([2048 * times] * batch))
    assert int(cache.status.item()) == 0
    for b in (0, 17, batch - 1):
        case.check(out[b:b + 1], what=f"sequence {b}")


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_attention_scales_and_queries(dtype):
    """Scales far apart in one sequence, queries of any size, zero rows, large scores."""
    dtype = DT[dtype]
    for seed, gain, spread, sm in ((1, 1.0, 12.0, 0.0), (2, 0.0, 1.0, 0.0), (3, 2.0 ** -12, 1.0, 0.0), (4, 1.0, 1.0, 1e-30),
                                   (5, 4.0, 1.0, 0.5), (6, 100.0 if dtype == torch.float16 else 2.0 ** 40, 1.0, 1e-3 if dtype == torch.float16 else 2.0 ** -40)):
        case = Case(seed, [400, 30], 2, 9, 16, dtype, sm_scale=sm, gain=gain, spread=spread)
        if seed == 1:
            case.q_c[0, 1] = 0
            case.q_pe[0, 1, 3] = 0
        case.check(case.run(), what=f"seed {seed}")


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_attention_one_token_is_its_latent(dtype):
    case = Case(3, [1, 5], 1, 4, 16, DT[dtype], spread=0.0)
    codes, _, byte = L.unpack(case.pages, case.P, case.dtype)
    s = case.slots(0, np.arange(1))
    want = torch.from_numpy(codes[s[0]] * L.scale(byte[s[0]])).to(case.dtype)
    assert torch.equal(case.run()[0, 0].cpu(), want.expand(4, 512))


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_attention_heavy_token_beside_many_light_ones(dtype):
    """One token of weight 1 and n of 2^-17 each: they sum to as much as it, and are not lost."""
    n, P, dtype = 1 << 17, 256, DT[dtype]
    c = np.zeros((n + 1, 512))
    c[0, 0], c[1:, 1] = 1.0, 1.0
    gap = 17 * math.log(2)  # of the scores: q . c with q = (gap, 0, ...)
    q_c = np.zeros((1, 1, 2, 512))
    q_c[..., 0] = np.array([1.0, 1.0])
    pages = np.zeros((n // P + 1, 641 * P), np.uint8)
    L.put(pages, P, np.arange(n + 1), c, np.zeros((n + 1, 64)), dtype)
    cache = make(2, P, n // P + 1, dtype, sm_scale=gap)
    cache.pages.copy_(torch.from_numpy(pages))
    out = host(cache.decode(dev(q_c[0], dtype), torch.zeros(1, 2, 64, dtype=dtype, device="cuda"),
                            int32(np.arange(n // P + 1))[None], int32([n + 1])))
    assert np.abs(out[..., :2] - 0.5).max() < 2.0 ** -9, out[..., :2]


@pytest.mark.parametrize("heads", [3, 8, 30])
def test_attention_nan_tokens_reach_rows_that_see_them(heads):
    """A token stored as NaN among the drafts, and garbage behind the sequence."""
    case = Case(9, [270, 300], 6, heads, 16, torch.bfloat16)
    clean = case.run()
    bad = case.slots(0, np.array([270 - 6 + 3]))[0]
    case.pages[bad // 16, 640 * 16 + bad % 16] = 255
    case.load()
    out = case.run()
    assert torch.equal(out[0, :3], clean[0, :3]) and torch.isnan(out[0, 3:]).all() and torch.equal(out[1], clean[1])
    mask = np.array([[1 << j for j in range(6)]] * 2, np.int64)
    out = case.run(mask)
    assert torch.isnan(out[0, 3]).all() and not torch.isnan(out[0, [0, 1, 2, 4, 5]]).any() and not torch.isnan(out[1]).any()


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("value", [math.nan, math.inf, -math.inf])
@pytest.mark.parametrize("heads", [10, 30, 70])
def test_attention_queries_not_finite(dtype, value, heads):
    case = Case(4, [600, 0], 2, heads, 16, DT[dtype])
    clean = case.run()
    case.q_c[0, 1, 2, 7] = value
    case.q_pe[0, 0, heads - 1, 3] = value
    case.q_c[1, 0, 0, 0] = value
    out = case.run()
    hit = torch.zeros(2, 2, heads, dtype=torch.bool, device="cuda")
    hit[0, 1, 2] = hit[0, 0, heads - 1] = True
    assert torch.isnan(out[hit]).all() and torch.equal(out[~hit], clean[~hit])
    assert not out[1].any()


def test_attention_faults():
    """Lengths and pages out of range are reported, and the other sequences are as they would be."""
    case = Case(6, [100, 200, 300], 2, 16, 16, torch.float16)
    clean = case.run()
    for lens, what in (([100, -5, 300], rq.RQ_STATUS_BAD_LEN), ([100, 100000, 300], rq.RQ_STATUS_BAD_LEN), ([100, 1, 300], rq.RQ_STATUS_BAD_LEN)):
        case.cache.status.zero_()
        out = case.run(seq_lens=int32(lens))
        assert int(case.cache.status.item()) & what and torch.equal(out[[0, 2]], clean[[0, 2]])
    for page in (-1, 1 << 30):
        case.cache.status.zero_()
        table = case.table.copy()
        table[1, 3] = page
        out = case.run(block_table=dev(table))
        assert int(case.cache.status.item()) == rq.RQ_STATUS_BAD_PAGE and torch.equal(out[[0, 2]], clean[[0, 2]])
    case.cache.status.zero_()
    table = case.table.copy()
    table[:, -1] = -1  # behind every sequence: not looked at
    assert torch.equal(case.run(block_table=dev(table)), clean) and int(case.cache.status.item()) == 0


def test_attention_refuses():
    case = Case(1, [40, 50], 3, 8, 16, torch.float16)
    c = case.cache
    q, p, tab, lens = case.q_c, case.q_pe, dev(case.table), dev(case.lens)
    mask = torch.ones(2, 3, dtype=torch.int64, device="cuda")
    ok = lambda **o: c.tree_verify(**{**dict(q_c=q, q_pe=p, tree_mask=mask, block_table=tab, seq_lens=lens), **o})  # noqa: E731
    ok()
    inv, cap = rq.RQ_ERR_INVALID, rq.RQ_ERR_CAPACITY
    four = q.new_zeros(2, 4, 8, 512), p.new_zeros(2, 4, 8, 64), torch.ones(2, 4, dtype=torch.int64, device="cuda")
    for bad, code in ((dict(q_c=q[..., :256]), inv), (dict(q_c=q.bfloat16()), inv), (dict(q_c=q[:1]), inv), (dict(q_pe=p[:, :2]), inv),
                      (dict(q_c=q[:, :, :4]), inv), (dict(q_c=q.cpu()), inv), (dict(seq_lens=lens.long()), inv), (dict(seq_lens=lens[:1]), inv),
                      (dict(block_table=tab.long()), inv), (dict(block_table=tab[:1]), inv), (dict(block_table=tab.t().contiguous().t()), inv),
                      (dict(tree_mask=mask.int()), inv), (dict(tree_mask=mask[:, :2]), inv), (dict(tree_mask=None), inv),
                      (dict(tree_mask=mask.cpu()), inv), (dict(out=torch.empty(2, 3, 8, 512, device="cuda")), inv),
                      (dict(q_c=q[:, 0]), inv), (dict(q_c=q.new_zeros(2, 4, 8, 512)[:, :3]), inv),
                      (dict(q_c=four[0], q_pe=four[1], tree_mask=four[2]), cap),
                      (dict(block_table=torch.zeros(2, 99, dtype=torch.int32, device="cuda")), cap),
                      (dict(q_c=q.new_zeros(5, 3, 8, 512), q_pe=p.new_zeros(5, 3, 8, 64), tree_mask=mask.new_ones(5, 3),
                            block_table=tab.new_zeros(5, 2), seq_lens=lens.new_zeros(5)), cap)):
        with pytest.raises(rq.RQError) as e:
            ok(**bad)
        assert e.value.code == code, bad.keys()
    big = rq.LatentCache(1, 16, 4, max_batch=1, max_query_tokens=65)
    with pytest.raises(rq.RQError):
        big.tree_verify(q.new_zeros(1, 65, 1, 512), p.new_zeros(1, 65, 1, 64), mask.new_zeros(1, 65), tab[:1], lens[:1])
    assert c.verify(q[:0], p[:0], tab[:0], lens[:0]).shape == (0, 3, 8, 512)


# ---------------------------------------------------------------------------------- reading back

@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("lens,P,starts,gap", [([1], 16, None, 0), ([0, 5, 0, 100, 0], 16, None, 0), ([300, 17], 48, [7, 100], 3),
                                               ([2000, 1, 999], 256, None, 2)])
def test_read(dtype, lens, P, starts, gap):
    dtype = DT[dtype]
    whole = [n + (starts[i] if starts else 0) for i, n in enumerate(lens)]
    case = Case(len(lens), whole, 1, 1, P, dtype, spread=6.0)
    codes, part, byte = L.unpack(case.pages, P, dtype)
    off = np.concatenate([[0], np.cumsum(lens)]) + gap
    n = int(off[-1]) + gap
    c = torch.full((n, 512), 7.0, dtype=dtype, device="cuda")
    pe = torch.full((n, 64), 7.0, dtype=dtype, device="cuda")
    got = case.cache.read(dev(case.table), int32(off), n, starts=None if starts is None else int32(starts), c=c, k_pe=pe)
    assert got[0] is c and got[1] is pe
    for b in range(len(lens)):
        s = case.slots(b, np.arange(lens[b]) + (starts[b] if starts else 0))
        want = torch.from_numpy(codes[s] * L.scale(byte[s])[:, None]).to(dtype), torch.from_numpy(part[s] * L.scale(byte[s])[:, None]).to(dtype)
        for t, w in zip((c, pe), want):
            assert torch.equal(t[off[b]:off[b + 1]].cpu(), w)
    for t in (c, pe):
        assert (t[:gap] == 7).all() and (t[n - gap:] == 7).all()
    assert int(case.cache.status.item()) == 0


def test_read_faults():
    case = Case(2, [100, 60], 1, 1, 16, torch.bfloat16)
    cache, tab = case.cache, dev(case.table)
    nan = case.slots(1, np.array([8]))[0]
    cache.pages[nan // 16, 640 * 16 + nan % 16] = 255
    c, pe = cache.read(tab, int32([0, 100, 160]), 160)
    assert torch.isnan(c[108]).all() and torch.isnan(pe[108]).all() and torch.isnan(c).sum() == 512
    full = lambda: (torch.full((160, 512), 7.0, dtype=torch.bfloat16, device="cuda"),  # noqa: E731
                    torch.full((160, 64), 7.0, dtype=torch.bfloat16, device="cuda"))
    for starts, offsets, page, bit in (([0, -1], [0, 100, 160], None, rq.RQ_STATUS_BAD_LEN), ([0, 1 << 30], [0, 100, 160], None, rq.RQ_STATUS_BAD_LEN),
                                       (None, [0, 100, 160], -3, rq.RQ_STATUS_BAD_PAGE), (None, [0, 100, 160], 1 << 20, rq.RQ_STATUS_BAD_PAGE)):
        cache.status.zero_()
        t2 = case.table.copy()
        if page is not None:
            t2[1, 0] = page
        x, y = full()
        cache.read(dev(t2), int32(offsets), 160, starts=None if starts is None else int32(starts), c=x, k_pe=y)
        assert int(cache.status.item()) == bit
        assert torch.equal(x[:100], c[:100]) and (x[100] == 7).all() and (y[100] == 7).all()
    for offsets in ([0, 160, 100], [-50, 100, 160], [200, 100, 50]):  # falling or outside: whatever is read stays inside
        x, y = full()
        cache.read(tab, int32(offsets), 160, c=x, k_pe=y)
        torch.cuda.synchronize()
    cache.status.zero_()
    for bad in (dict(offsets=int32([0, 160])), dict(offsets=int32([0, 100, 160]).long()), dict(block_table=tab.long()), dict(n=-1),
                dict(starts=int32([0])), dict(c=torch.empty(160, 512, device="cuda")), dict(k_pe=torch.empty(159, 64, dtype=torch.bfloat16, device="cuda"))):
        with pytest.raises(rq.RQError):
            cache.read(**{**dict(block_table=tab, offsets=int32([0, 100, 160]), n=160), **bad})
    assert cache.read(tab[:0], int32([0]), 0)[0].shape == (0, 512)


# ---------------------------------------------------------------------------- the expanded form

def prompt_case(seed, new, old, heads, dtype, gain=1.0, gap=0):
    rng = gen(seed)
    qo = np.concatenate([[0], np.cumsum(new)]) + gap
    ko = np.concatenate([[0], np.cumsum(np.asarray(new) + old)]) + gap
    nq, nk = int(qo[-1]) + gap, int(ko[-1]) + gap
    q = dev(rng.standard_normal((nq, heads, 192)) * gain, dtype)
    kv = dev(rng.standard_normal((nk, heads, 256)), dtype)
    pe = dev(rng.standard_normal((nk, 72)), dtype)[:, :64]
    return q, kv[..., :128], pe, kv[..., 128:], qo, ko


def check_prompt(out, q, k, pe, v, qo, ko, dtype, sm=0.0):
    ref, tol = L.prompt(host(q), host(k), host(pe), host(v), qo, ko, sm or 192 ** -0.5, dtype)
    rows = slice(qo[0], qo[-1])
    within(host(out)[rows], ref[rows], (tol + R.half_step(dtype, ref) * (1 + 2.0 ** -8))[rows], "prompt")


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("new,old,heads", [
    ([1], [0], 1),
    ([1, 2, 127, 128, 129], [0, 0, 0, 0, 0], 3),
    ([257, 0, 64], [0, 100, 0], 2),
    ([5, 1, 300], [1000, 127, 128], 5),
    ([600], [400], 1),
    ([1, 1], [511, 0], 16),
    ([3, 200], [5000, 9000], 2),     # few units: a cluster shares each one's keys
    ([2, 1, 300], [0, 7000, 900], 3),
    ([256, 129, 7], [130, 0, 1024], 4),
    ([100, 30, 0, 1], [4000, 333, 5, 0], 70),  # more units than pairs of SMs, no more than 256 queries
    ([1100, 513], [20, 0], 3),       # rows of several sizes, cut
    ([64, 2], [5000, 3000], 2),      # no more than 256 queries, cut
    ([600], [0], 130),
])
def test_prompt(dtype, new, old, heads):
    dtype = DT[dtype]
    q, k, pe, v, qo, ko = prompt_case(len(new) + heads, new, old, heads, dtype, gap=2)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = torch.full((q.shape[0], heads, 128), 7.0, dtype=dtype, device="cuda")
    got = rq.prompt_attention(q, k, pe, v, int32(qo), int32(ko), max(new), out=out, status=status)
    assert got is out and int(status.item()) == 0
    check_prompt(out, q, k, pe, v, qo, ko, dtype)
    assert (out[:2] == 7).all() and (out[-2:] == 7).all(), "rows of no sequence are left as they are"
    again = rq.prompt_attention(q, k, pe, v, int32(qo), int32(ko), max(new))
    assert torch.equal(again[2:-2], out[2:-2])
    # other strides: heads outside tokens, contiguous copies
    t = [x.transpose(0, 1).contiguous().transpose(0, 1) for x in (q, k, v)]
    assert torch.equal(rq.prompt_attention(t[0], t[1], pe.contiguous(), t[2], int32(qo), int32(ko), max(new))[2:-2], out[2:-2])
    # a larger bound may lay the work out otherwise, and so add in another order
    check_prompt(rq.prompt_attention(q, k, pe, v, int32(qo), int32(ko), max(new) + 100), q, k, pe, v, qo, ko, dtype)


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_prompt_scores_of_any_size(dtype):
    dtype = DT[dtype]
    for seed, gain, sm in ((1, 0.0, 0.0), (2, 20.0, 0.0), (3, 1.0, 1e-30), (4, 300.0, 1.0)):
        q, k, pe, v, qo, ko = prompt_case(seed, [200, 3], [50, 0], 2, dtype, gain)
        check_prompt(rq.prompt_attention(q, k, pe, v, int32(qo), int32(ko), 200, sm_scale=sm), q, k, pe, v, qo, ko, dtype, sm)


def test_prompt_rising_scores():
    """Scores that rise along the keys move the running maximum in every tile."""
    q, k, pe, v, qo, ko = prompt_case(3, [300], [700], 1, torch.float16)
    q.fill_(1.0)
    k.copy_(torch.linspace(-1, 1, 1000, device="cuda")[:, None, None].expand(1000, 1, 128))
    check_prompt(rq.prompt_attention(q, k, pe, v, int32(qo), int32(ko), 300, sm_scale=1.0), q, k, pe, v, qo, ko, torch.float16, 1.0)


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("value", [math.nan, math.inf, -math.inf])
@pytest.mark.parametrize("n", [300, 200])
def test_prompt_values_that_are_not_finite(dtype, value, n):
    """A value that is not finite reaches the rows that see it, in its dim, and no other; nor does a key's, or one of the
    next sequence."""
    dtype = DT[dtype]
    q, k, pe, v, qo, ko = prompt_case(7, [n, 40], [37, 5], 2, dtype)
    clean = rq.prompt_attention(q, k, pe, v, int32(qo), int32(ko), n)
    for pos in (37 + 1, 37 + 130, 37 + n - 1, 10, ko[1]):
        v2 = v.clone()
        v2[pos, 1, 5] = value
        out = rq.prompt_attention(q, k, pe, v2, int32(qo), int32(ko), n)
        hit = torch.zeros_like(out, dtype=torch.bool)
        hit[max(0, pos - 37):n if pos < ko[1] else n + 40, 1, 5] = True
        if pos == ko[1]:
            hit[:n] = False
        assert not torch.isfinite(out[hit]).any() and torch.equal(out[~hit], clean[~hit]), pos
        k2, pe2 = k.clone(), pe.clone()
        k2[pos, 0, 3] = value
        out = rq.prompt_attention(q, k2, pe, v, int32(qo), int32(ko), n)
        hit.zero_()
        hit[max(0, pos - 37):n, 0] = True
        if pos == ko[1]:
            hit[:n] = False
            hit[n:, 0] = True
        assert torch.equal(out[~hit], clean[~hit])
        if math.isnan(value):
            assert torch.isnan(out[hit]).all()
            pe2[pos, 9] = value
            out = rq.prompt_attention(q, k, pe2, v, int32(qo), int32(ko), n)
            hit |= hit.any(1, keepdim=True)
            assert torch.isnan(out[hit]).all() and torch.equal(out[~hit], clean[~hit])


def test_prompt_rows_that_see_nothing():
    """More queries than keys: the first see nothing and are zeros."""
    rng = gen(1)
    q = dev(rng.standard_normal((200, 2, 192)), torch.float16)
    kv = dev(rng.standard_normal((50, 2, 128)), torch.float16)
    pe = dev(rng.standard_normal((50, 64)), torch.float16)
    for nk in (50, 0):
        out = rq.prompt_attention(q, kv[:nk], pe[:nk], kv[:nk], int32([0, 200]), int32([0, nk]), 200)
        assert not out[:200 - nk].any()
        check_prompt(out, q, kv[:nk], pe[:nk], kv[:nk], [0, 200], [0, nk], torch.float16)


def test_prompt_faults_and_refusals():
    q, k, pe, v, qo, ko = prompt_case(5, [30, 20, 10], [5, 0, 7], 2, torch.bfloat16)
    clean = rq.prompt_attention(q, k, pe, v, int32(qo), int32(ko), 30)
    for qb, kb, most in (([0, 30, 25, 60], ko, 30), ([0, 30, 50, 61], ko, 30), ([-1, 30, 50, 60], ko, 31), (qo, [0, 35, 30, 72], 30),
                         (qo, [0, 35, 55, 73], 30), (qo, [-2, 35, 55, 72], 30), (qo, ko, 29)):
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        out = torch.full_like(clean, 7.0)
        rq.prompt_attention(q, k, pe, v, int32(qb), int32(kb), most, out=out, status=status)
        assert int(status.item()) == rq.RQ_STATUS_BAD_LEN
        for b in range(3):
            if qb[b] == qo[b] and qb[b + 1] == qo[b + 1] and kb[b] == ko[b] and kb[b + 1] == ko[b + 1] and qo[b + 1] - qo[b] <= most:
                assert torch.equal(out[qo[b]:qo[b + 1]], clean[qo[b]:qo[b + 1]])
    ok = lambda **o: rq.prompt_attention(**{**dict(q=q, k=k, k_pe=pe, v=v, q_offsets=int32(qo), k_offsets=int32(ko), max_new=30), **o})  # noqa: E731
    for bad in (dict(q=q[..., :128]), dict(q=q.float()), dict(q=q.cpu()), dict(k=k.half()), dict(k=k[:5]), dict(k=k[:, :1]), dict(v=v[..., :64]),
                dict(k_pe=pe[:, :32]), dict(k_pe=pe[:5]), dict(k_pe=pe.cpu()), dict(q_offsets=int32(qo).long()), dict(k_offsets=int32(ko)[:2]),
                dict(max_new=-1), dict(sm_scale=-1.0), dict(out=torch.empty(60, 2, 128, device="cuda")), dict(k=k[:, :1].expand(-1, 2, -1)),
                dict(q=q.transpose(1, 2)), dict(status=torch.zeros(1, device="cuda")), dict(k_offsets=int32(ko).cpu()),
                dict(v=v.new_zeros(72, 2, 132)[..., 4:])):
        with pytest.raises(rq.RQError) as e:
            ok(**bad)
        assert e.value.code == rq.RQ_ERR_INVALID, bad.keys()
    assert rq.prompt_attention(q[:0], k, pe, v, int32([0]), int32([0]), 0).shape == (0, 2, 128)


# ------------------------------------------------------------------------------------ together

def serve(dtype, cache, stream=None):
    """A prompt and four decode steps through append, read, the expansion and both forms of attention."""
    rng, heads, n = gen(11), 4, 90
    w_k, w_v = (dev(rng.standard_normal((heads, 128, 512)) / 16, dtype) for _ in range(2))
    rope = rq.Rope(64, interleaved=True)
    weight = dev(1 + 0.1 * rng.standard_normal(512), torch.float32)
    table = int32(rng.permutation(8)[None])
    down = dev(rng.standard_normal((n + 4, 576)), dtype)
    q = dev(rng.standard_normal((n + 4, heads, 192)), dtype)
    slot_of = lambda p: table[0, p // 16].long() * 16 + p % 16  # noqa: E731
    every = torch.arange(n + 4, device="cuda")
    slots, pos = slot_of(every).int(), every.int()
    outs = []
    q_pe = q[..., 128:]
    cache.append(down[:n, :512], down[:n, 512:], slots[:n], rope, pos[:n], weight, q_pe=q_pe[:n], q_pe_out=q_pe[:n])
    for step in range(5):
        end = n + step
        first = 0 if step == 0 else end - 1
        if step:
            cache.append(down[end - 1:end, :512], down[end - 1:end, 512:], slots[end - 1:end], rope, pos[end - 1:end], weight,
                         q_pe=q_pe[end - 1:end], q_pe_out=q_pe[end - 1:end])
        c, pe = cache.read(table, int32([0, end]), end)
        k, v = (torch.einsum("nc,hdc->nhd", c, w) for w in (w_k, w_v))
        expanded = rq.prompt_attention(q[first:end], k, pe, v, int32([0, end - first]), int32([0, end]), end - first)
        q_c = torch.einsum("nhd,hdc->hnc", q[first:end, :, :128], w_k).transpose(0, 1)[None]
        lat = cache.verify(q_c, q_pe[first:end][None], table, int32([end]))[0]
        outs.append((expanded, torch.einsum("nhc,hdc->nhd", lat, w_v)))
    return outs


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_both_forms_agree_over_a_prompt_and_decode_steps(dtype):
    """The two forms differ by the roundings of keys, values and absorbed queries to 16 bits: of each score and of each output
    some 4 eps of the magnitudes, which are a few units here."""
    dtype = DT[dtype]
    cache = make(4, 16, 8, dtype, batch=1, t=90)
    for expanded, absorbed in serve(dtype, cache):
        a, b = host(expanded), host(absorbed)
        assert np.abs(a - b).max() <= 32 * torch.finfo(dtype).eps * np.abs(a).max() and np.abs(a).max() > 0.1
    assert int(cache.status.item()) == 0


def test_on_another_stream_and_captured():
    """A decode step, append and attention, on a stream of the caller's, then captured once and replayed on new inputs."""
    case = Case(12, [300, 40, 0], 1, 16, 16, torch.bfloat16)
    cache, tab, lens = case.cache, dev(case.table), dev(case.lens)
    rope = rq.Rope(64)
    rng = gen(2)
    x = dev(rng.standard_normal((3, 576)), torch.bfloat16)
    slots = int32(list(case.slots(0, np.array([299]))) + list(case.slots(1, np.array([39]))) + [-1])
    pos = int32([299, 39, 0])
    q_c, q_pe = case.q_c[:, 0].contiguous(), case.q_pe[:, 0].contiguous()
    out = torch.empty_like(q_c)
    turned = torch.empty_like(q_pe)

    def step():
        cache.append(x[:, :512], x[:, 512:], slots, rope, pos, q_pe=q_pe, q_pe_out=turned)
        cache.decode(q_c, turned, tab, lens, out=out)

    step()
    want = out.clone()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        out.zero_()
        step()
        got = out.clone()
    s.synchronize()
    assert torch.equal(got, want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    x.copy_(torch.randn_like(x))
    q_c.copy_(torch.randn_like(q_c))
    step()
    want = out.clone()
    out.zero_()
    graph.replay()
    assert torch.equal(out, want)


def test_outputs_over_inputs():
    """Attention may write over its latent queries; an output over other inputs is refused."""
    for T in (1, 3):
        case = Case(3, [5000, 40, 700], T, 60, 16, torch.bfloat16)  # (cut, and of several units)
        case.q_c = case.q_c.contiguous()
        want, q = case.run(), case.q_c.clone()
        assert case.run(q_c=q, out=q) is q and torch.equal(q, want)
    big = torch.zeros(3 * 3 * 60 * 512 + 512, dtype=torch.bfloat16, device="cuda")
    for bad in (dict(q_c=big[:-512].view(3, 3, 60, 512), out=big[512:].view(3, 3, 60, 512)),
                dict(q_pe=big[:3 * 3 * 60 * 64].view(3, 3, 60, 64), out=big[:-512].view(3, 3, 60, 512)),
                dict(q_c=big[:-512].view(3, 60, 3, 512).transpose(1, 2), out=big[:-512].view(3, 3, 60, 512))):
        with pytest.raises(rq.RQError) as e:
            case.run(**bad)
        assert e.value.code == rq.RQ_ERR_INVALID
    rows = torch.zeros(64 * 1024, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(rq.RQError) as e:
        case.cache.read(dev(case.table[:1]), int32([0, 40]), 40, c=rows[:40 * 512].view(40, 512), k_pe=rows[512:512 + 40 * 64].view(40, 64))
    assert e.value.code == rq.RQ_ERR_INVALID
    q, k, pe, v, qo, ko = prompt_case(2, [30], [10], 2, torch.float16)
    k, v = k.contiguous(), v.contiguous()
    for out in (k[10:], v[:30], q.flatten()[:30 * 256].view(30, 2, 128)):
        with pytest.raises(rq.RQError) as e:
            rq.prompt_attention(q, k, pe, v, int32(qo), int32(ko), 30, out=out)
        assert e.value.code == rq.RQ_ERR_INVALID


def test_views_of_the_pool():
    case = Case(2, [20], 1, 1, 32, torch.float16)
    codes, part, byte = L.unpack(case.pages, 32, torch.float16)
    c, p, s = case.cache.codes(), case.cache.position_parts(), case.cache.scales()
    assert c.shape == (case.pages.shape[0], 4, 32, 128) and p.shape[1:] == (32, 64) and s.shape[1:] == (32,)
    slot = case.slots(0, np.array([19]))[0]
    n, r = divmod(int(slot), 32)
    got = c[n, :, r].float().cpu().numpy().reshape(4, 8, 16)[:, np.arange(8) ^ (r % 8)].reshape(512)
    assert np.array_equal(got, codes[slot]) and float(s[n, r]) == 2.0 ** (byte[slot] - 127)


def test_prompt_on_another_stream_and_captured():
    """Calls of several cuts on two streams at once, each with its own workspace, then one captured and replayed on new inputs."""
    cases = [prompt_case(i, new, old, 3, torch.bfloat16) for i, (new, old) in enumerate((([64], [4000]), ([1100, 3], [0, 700]), ([700], [90])))]
    run = lambda c: rq.prompt_attention(*c[:4], int32(c[4]), int32(c[5]), int(np.diff(c[4]).max()))  # noqa: E731
    want = [run(c) for c in cases]
    streams = [torch.cuda.Stream() for _ in cases]
    torch.cuda.synchronize()
    got = []
    for _ in range(3):
        for c, s in zip(cases, streams):
            with torch.cuda.stream(s):
                got.append(run(c))
    torch.cuda.synchronize()
    assert all(torch.equal(g, want[i % len(cases)]) for i, g in enumerate(got))
    q, k, pe, v, qo, ko = cases[0]
    qo, ko = int32(qo), int32(ko)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = rq.prompt_attention(q, k, pe, v, qo, ko, 64)
    q.copy_(torch.randn_like(q))
    v.copy_(torch.randn_like(v))
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, rq.prompt_attention(q, k, pe, v, qo, ko, 64))


def test_prompt_workspace_is_checked():
    q, k, pe, v, qo, ko = prompt_case(1, [5], [3], 2, torch.float16)
    out = torch.full((5, 2, 128), 7.0, dtype=torch.float16, device="cuda")
    small = torch.empty(rq.rq_prompt_workspace(0) - 16, dtype=torch.uint8, device="cuda")
    with pytest.raises(rq.RQError) as e:
        rq.rq_prompt_attention(q, k, pe, v, int32(qo), int32(ko), 5, out, small)
    assert e.value.code == rq.RQ_ERR_CAPACITY and (out == 7).all()


def test_two_caches_on_two_streams_at_once():
    """Each cache has its own workspace: calls that are cut over many tokens, in flight together."""
    cases = [Case(seed, [5000, 300], 1, 20, 32, torch.float16) for seed in (1, 2)]
    want = [c.run() for c in cases]
    streams = [torch.cuda.Stream() for _ in cases]
    args = [(c.q_c, c.q_pe, dev(c.table), dev(c.lens)) for c in cases]
    torch.cuda.synchronize()
    got = []
    for _ in range(5):
        for c, s, a in zip(cases, streams, args):
            with torch.cuda.stream(s):
                got.append(c.cache.verify(*a))
    torch.cuda.synchronize()
    assert all(torch.equal(g, want[i % 2]) for i, g in enumerate(got))


def test_offsets_past_32_bits():
    """A pool past 4 GiB, and rows past 2^31 elements in every tensor, against small ones."""
    P, dtype, heads, rng = 64, torch.bfloat16, 128, gen(4)
    x = dev(rng.standard_normal((70, 576)), dtype)
    small, big = make(heads, P, 2, dtype, batch=4096, t=9), make(heads, P, 110000, dtype, batch=4096, t=9)
    first, far = np.arange(70), np.arange(70) + np.where(np.arange(70) < 64, 109999, 107000 - 1) * 64
    small.append(x[:, :512], x[:, 512:], int32(first))
    big.append(x[:, :512], x[:, 512:], int32(far))
    assert torch.equal(big.pages[109999], small.pages[0])
    near_table, far_table = int32([[0, 1]]), int32([[109999, 107000]])
    q_c, q_pe = dev(rng.standard_normal((1, 9, heads, 512)), dtype), dev(rng.standard_normal((1, 9, heads, 64)), dtype)
    want = small.verify(q_c, q_pe, near_table, int32([70]))
    assert torch.equal(big.verify(q_c, q_pe, far_table, int32([70])), want)

    q_many, out = torch.zeros(4096, 9, heads, 512, dtype=dtype, device="cuda"), torch.empty(4096, 9, heads, 512, dtype=dtype, device="cuda")
    pe_many = torch.zeros(4096, 9, heads, 64, dtype=dtype, device="cuda")
    q_many[-1], pe_many[-1] = q_c[0], q_pe[0]
    lens, tables = int32([0] * 4095 + [70]), far_table.expand(4096, 2).contiguous()
    big.verify(q_many, pe_many, tables, lens, out=out)
    ref, tol = L.attention(host(q_c), host(q_pe), small.pages.cpu().numpy(), np.array([[0, 1]]), np.array([70]), P, L.chain(9), 192 ** -0.5, dtype)
    within(host(out[-1:]), ref, tol + R.half_step(dtype, ref) * (1 + 2.0 ** -8))
    assert not out[0].any() and not out[4094].any()
    del q_many, pe_many, out

    c, pe = small.read(near_table, int32([0, 70]), 70)
    n = 4_300_000
    c_far, pe_far = torch.empty(n, 512, dtype=dtype, device="cuda"), torch.empty(n, 64, dtype=dtype, device="cuda")
    big.read(far_table, int32([n - 70, n]), n, c=c_far, k_pe=pe_far)
    assert torch.equal(c_far[-70:], c) and torch.equal(pe_far[-70:], pe)
    del c_far, pe_far

    n = 100_000
    down, q = torch.zeros(n, 576, dtype=dtype, device="cuda"), torch.zeros(n, heads, 192, dtype=dtype, device="cuda")
    down[-70:], q[-9:, :, 128:] = x, q_pe[0]
    rope, slots, pos = rq.Rope(64), torch.full((n,), -1, dtype=torch.int32, device="cuda"), torch.arange(n, dtype=torch.int32, device="cuda")
    slots[-70:] = int32(first)
    big.append(down[:, :512], down[:, 512:], slots, rope, pos, q_pe=q[..., 128:], q_pe_out=q[..., 128:])
    turned = small.append(x[:, :512], x[:, 512:], int32(first), rope, pos[-70:], q_pe=torch.cat([torch.zeros(61, heads, 64, dtype=dtype, device="cuda"), q_pe[0]]))
    near = lambda a, b: np.abs(host(a) - host(b)).max() <= torch.finfo(dtype).eps * np.abs(host(b)).max()  # noqa: E731
    assert near(q[-9:, :, 128:], turned[-9:])  # (a long call and a short one round apart)
    (c, pe), (c_ref, pe_ref) = (m.read(near_table, int32([0, 70]), 70) for m in (big, small))
    assert torch.equal(c, c_ref) and near(pe, pe_ref)
    assert int(big.status.item()) == 0 and int(small.status.item()) == 0
    del q, big

    nq = 140_000
    q = torch.empty(nq, heads, 192, dtype=dtype, device="cuda")
    kv, k_pe = torch.empty(nq, 64 + heads, 128, dtype=dtype, device="cuda"), torch.empty(nq, 64, dtype=dtype, device="cuda")
    q[-9:] = dev(rng.standard_normal((9, heads, 192)), dtype)
    kv[-300:] = dev(rng.standard_normal((300, 64 + heads, 128)), dtype)
    k_pe[-300:] = dev(rng.standard_normal((300, 64)), dtype)
    k, v = kv[:, 64:], kv[:, :heads]
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = rq.prompt_attention(q, k, k_pe, v, int32([nq - 9, nq]), int32([nq - 300, nq]), 9, status=status)
    check_prompt(out[-9:], q[-9:], k[-300:], k_pe[-300:], v[-300:], [0, 9], [0, 300], dtype)
    assert int(status.item()) == 0
