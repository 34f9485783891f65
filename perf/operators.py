"""Measured cases of the 8-bit block-scaled KV cache and of what stands before it: the norms and
position rotation of queries and keys, the append that applies them on the way, and attention
(decode, verify, extend) over the cache.

`run` computes each operator in elementary torch operations, or, with `own`, through the
framework's entry points; `exact` gives the same from the definition in 64 bits.

The cache: a block is 16 tokens of one kv head, 4112 bytes: 2048 key codes, 2048 value codes (e4m3),
the exponent bytes of the two scales (e8m0: 2^(byte - 127)), 14 unused bytes.  Key code of token r,
dim d at (((r/8)*2 + d/64)*32 + (r%8)*4 + d%64/16)*16 + d%16; value code at
(d/32*32 + d/4%8*4 + r%8/2)*16 + d%4*4 + r/8*2 + r%2.  A page holds page_size/16 blocks per kv head.
"""
import math

import torch

own = False

D = 128
BLOCK = 16
BLOCK_BYTES = 4112
E_MIN, E_MAX = -60, 60


# ------------------------------------------------------------------------------------- cases

def listed():
    return [
        # one decode step of 16 sequences: latency
        dict(name="norm_rope step 16", op="norm_rope", n=16, hq=32, hkv=8, dtype="float16", rotary=128, axes=1,
             interleaved=False, norm=True, far=32768),
        # a prefill chunk of image and text tokens: three position axes, rows inside the fused projection's output
        dict(name="norm_rope prefill 16384", op="norm_rope", n=16384, hq=64, hkv=8, dtype="bfloat16", rotary=128,
             axes=3, interleaved=False, norm=True, far=131072),
        # odd sizes, half of the head rotated, pairs interleaved, no norm, far positions
        dict(name="norm_rope odd 1013", op="norm_rope", n=1013, hq=12, hkv=4, dtype="float16", rotary=64, axes=1,
             interleaved=True, norm=False, far=1048576),
        # the newest token of 64 sequences: queries, keys and values of a decode step in one call
        dict(name="append step 64", op="append", batch=64, new=1, start=4097, hq=64, hkv=8, page=16,
             dtype="bfloat16", axes=1, norm=True),
        # a prefill chunk of one sequence that starts inside a block
        dict(name="append prefill 32768", op="append", batch=1, new=32768, start=1000, hq=32, hkv=8, page=64,
             dtype="bfloat16", axes=3, norm=True),
        # one short sequence: latency
        dict(name="decode 1x1024", op="attend", batch=1, least=1024, most=1024, t=1, hq=32, hkv=8, page=16,
             dtype="float16"),
        # a server's batch of ragged lengths
        dict(name="decode 32x1K-32K", op="attend", batch=32, least=1024, most=32768, t=1, hq=64, hkv=8, page=16,
             dtype="bfloat16"),
        # many sequences of equal length
        dict(name="decode 64x16K", op="attend", batch=64, least=16384, most=16384, t=1, hq=64, hkv=8, page=64,
             dtype="float16"),
        # speculative verify of 6 drafts
        dict(name="verify 8x16K+6", op="attend", batch=8, least=16390, most=16390, t=6, hq=32, hkv=8, page=16,
             dtype="float16"),
        # chunked prefill, 1,024 new tokens over 15K cached ones
        dict(name="extend 8x1024 of 16K", op="extend", batch=8, least=16384, most=16384, t=1024, hq=32, hkv=8,
             page=16, dtype="bfloat16"),
        # a short ragged chunk of odd sizes
        dict(name="extend 3x77 of 2K", op="extend", batch=3, least=77, most=2048, t=77, hq=12, hkv=4, page=32,
             dtype="float16"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm_rope", "append", "attend", "attend", "extend"])
    hkv = rng.choice([1, 2, 4, 8])
    hq = hkv * rng.choice([1, 2, 3, 4, 5, 8])
    dtype = rng.choice(["float16", "bfloat16"])
    if op == "norm_rope":
        axes = rng.choice([1, 1, 2, 3])
        return dict(op=op, n=_log(rng, 1, 16384), hq=hq, hkv=hkv, dtype=dtype, rotary=rng.choice([32, 64, 96, 128, 128]),
                    axes=axes, interleaved=rng.random() < 0.4, norm=rng.random() < 0.7, far=_log(rng, 4096, 1 << 20))
    page = rng.choice([16, 32, 64, 128])
    if op == "append":
        if rng.random() < 0.5:
            batch, new = _log(rng, 1, 256), rng.choice([1, 1, 2, 5, 8])
        else:
            batch = rng.randint(1, 4)
            new = _log(rng, 16, 32768 // batch)
        return dict(op=op, batch=batch, new=new, start=_log(rng, 1, 8192) - 1, hq=hq, hkv=hkv, page=page, dtype=dtype,
                    axes=rng.choice([1, 3]), norm=rng.random() < 0.7)
    if op == "attend":
        t = rng.choice([1, 1, 2, 4, 6, 8])
        batch = _log(rng, 1, 64)
        most = _log(rng, 64, min(32768, 64 * 16384 // batch))
        return dict(op=op, batch=batch, least=max(t, most // rng.choice([1, 4, 32])), most=max(t, most), t=t, hq=hq,
                    hkv=hkv, page=page, dtype=dtype)
    batch = rng.randint(1, 8)
    t = _log(rng, 32, 1024)
    most = t + _log(rng, 1, 15360)
    return dict(op=op, batch=batch, least=max(t, most // rng.choice([1, 2, 8])), most=most, t=t, hq=min(hq, 32),
                hkv=hkv if hq <= 32 else 4, page=page, dtype=dtype)


# ------------------------------------------------------------------------------------ inputs

BASE = 500000.0
EPS = 1e-6


def _sections(pairs, axes):
    """Pairs per axis, the first axis taking what is left over."""
    each = pairs // axes // 4 * 4
    return [pairs - each * (axes - 1)] + [each] * (axes - 1)


def _lens(case, gen, device):
    lens = torch.randint(case["least"], case["most"] + 1, (case["batch"],), generator=gen, device=device)
    lens[0] = case["most"]
    return lens.to(torch.int32)


def _exponent(amax):
    """The smallest E in [E_MIN, E_MAX] with amax <= 448 * 2^E (448 = 0.875 * 2^9)."""
    m, e = torch.frexp(amax)
    return torch.where(amax > 0, torch.where(m <= 0.875, e - 9, e - 8), E_MIN).clamp(E_MIN, E_MAX)


def _to_layout_k(codes):  # [..., 16 tokens, 128 dims] -> [..., 2048]
    s = codes.shape[:-2]
    n = len(s)
    x = codes.reshape(*s, 2, 8, 2, 4, 16)  # r/8, r%8, d/64, d/16%4, d%16
    return x.permute(*range(n), n, n + 2, n + 1, n + 3, n + 4).reshape(*s, 2048)


def _to_layout_v(codes):
    s = codes.shape[:-2]
    n = len(s)
    x = codes.reshape(*s, 2, 4, 2, 4, 8, 4)  # r/8, r%8/2, r%2, d/32, d/4%8, d%4
    return x.permute(*range(n), n + 3, n + 4, n + 1, n + 5, n, n + 2).reshape(*s, 2048)


def _from_layout_k(raw):
    s = raw.shape[:-1]
    n = len(s)
    x = raw.reshape(*s, 2, 2, 8, 4, 16)
    return x.permute(*range(n), n, n + 2, n + 1, n + 3, n + 4).reshape(*s, 16, 128)


def _from_layout_v(raw):
    s = raw.shape[:-1]
    n = len(s)
    x = raw.reshape(*s, 4, 8, 4, 4, 2, 2)
    return x.permute(*range(n), n + 4, n + 2, n + 5, n, n + 1, n + 3).reshape(*s, 16, 128)


def _pool(num_blocks, hkv, per_page, gen, device):
    """A cache in use: pages [pages, hkv, page bytes] of coded keys (4 channels of each head ten
    times larger) and values.  num_blocks: blocks of 16 tokens, a multiple of per_page."""
    pages = torch.zeros((num_blocks // per_page, hkv, per_page, BLOCK_BYTES), dtype=torch.uint8, device=device)
    gain = torch.ones((hkv, 1, 1, D), device=device)
    gain.view(hkv, D).scatter_(1, torch.rand((hkv, D), generator=gen, device=device).argsort(1)[:, :4], 10.0)
    step = max(1, (1 << 25) // (hkv * per_page * BLOCK * D))
    for lo in range(0, pages.shape[0], step):
        part = pages[lo:lo + step]
        for at, scale in ((0, gain), (2048, 1.0)):
            x = torch.randn((part.shape[0], hkv, per_page, BLOCK, D), generator=gen, device=device) * scale
            e = _exponent(x.abs().amax((-1, -2)))
            codes = torch.ldexp(x, -e[..., None, None]).to(torch.float8_e4m3fn).view(torch.uint8)
            part[..., at:at + 2048] = (_to_layout_k if at == 0 else _to_layout_v)(codes)
            part[..., 4096 + at // 2048] = (e + 127).to(torch.uint8)
    return pages.view(pages.shape[0], hkv, per_page * BLOCK_BYTES)


def _table(lens, page, gen, device):
    """Pages of all sequences in a random order: block table [batch, most pages], pages in all."""
    need = (lens.cpu() + page - 1) // page
    width, total = int(need.max()), int(need.sum())
    order = torch.randperm(total, generator=gen, device=device).to(torch.int32)
    table = torch.zeros((len(lens), width), dtype=torch.int32, device=device)
    mask = torch.arange(width, device=device)[None] < need.to(device)[:, None]
    table[mask] = order
    return table, total


def _handles(case, state, device):
    """What a program of the framework keeps: the cache and the rotation."""
    from rotation_quantized_kv_rq_gb300 import rq
    if case["op"] != "norm_rope":
        state["cache"] = rq.KVCache(rq.RQ_FP8, 8, case["hq"], case["hkv"], case["page"], state["pages"].shape[0], None,
                                    None, max_batch=case["batch"], max_query_tokens=case.get("t", 1),
                                    max_pages_per_seq=state["table"].shape[1], device=device, pages=state["pages"],
                                    dtype=getattr(torch, case["dtype"]))
    if case["op"] in ("norm_rope", "append"):
        state["rope"] = rq.Rope(state["rotary"], base=BASE, sections=state["sections"],
                                interleaved=state["interleaved"], device=device)


def prepare(case, seed):
    device = torch.device("cuda", torch.cuda.current_device())
    gen = torch.Generator(device=device)
    gen.manual_seed(seed)
    dtype = getattr(torch, case["dtype"])
    hq, hkv = case["hq"], case["hkv"]
    state = dict(op=case["op"], hq=hq, hkv=hkv)
    if case["op"] in ("norm_rope", "append"):
        n = case["n"] if case["op"] == "norm_rope" else case["batch"] * case["new"]
        qkv = torch.randn((n, hq + 2 * hkv, D), generator=gen, device=device)
        qkv[:, hq:hq + hkv, :4] *= 10.0
        qkv = qkv.to(dtype)  # the fused projection's output; its three parts are slices of it
        state.update(q=qkv[:, :hq], k=qkv[:, hq:hq + hkv], v=qkv[:, hq + hkv:])
        state["rotary"] = case.get("rotary", D)
        state["interleaved"] = case.get("interleaved", False)
        state["sections"] = _sections(state["rotary"] // 2, case["axes"])
        state["wq"] = state["wk"] = None
        if case["norm"]:
            state["wq"], state["wk"] = 1 + 0.1 * torch.randn((2, D), generator=gen, device=device)
    if case["op"] == "norm_rope":
        state["positions"] = torch.randint(0, case["far"], (case["axes"], n), generator=gen, device=device,
                                           dtype=torch.int32)
    elif case["op"] == "append":
        batch, new, start, page = case["batch"], case["new"], case["start"], case["page"]
        first = start + torch.arange(batch, device=device) % 32  # sequences stand at different places of a block
        state["table"], pages = _table(first + new, page, gen, device)
        pos = first[:, None] + torch.arange(new, device=device)
        seq = torch.arange(batch, device=device)[:, None]
        state["slots"] = (state["table"][seq, pos // page] * page + pos % page).reshape(-1).to(torch.int32)
        axis = torch.arange(1, case["axes"] + 1, device=device)[:, None]
        state["positions"] = (pos.reshape(1, -1) // axis).to(torch.int32).contiguous()
        state["pages"] = _pool(pages * page // BLOCK, hkv, page // BLOCK, gen, device)
        state["page"] = page
    else:
        state["lens"] = _lens(case, gen, device)
        state["table"], pages = _table(state["lens"], case["page"], gen, device)
        state["pages"] = _pool(pages * case["page"] // BLOCK, hkv, case["page"] // BLOCK, gen, device)
        state["q"] = torch.randn((case["batch"], case["t"], hq, D), generator=gen, device=device).to(dtype)
        state["page"] = case["page"]
    if own:
        _handles(case, state, device)
    return state


# ----------------------------------------------------------------------------------- plain forms

def _turned(x, weight, positions, state):
    """The norm and position rotation of rows x [n, heads, 128], in 32 bits; angles in 64."""
    x = x.float()
    if weight is not None:
        x = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS) * weight
    r = state["rotary"]
    i = torch.arange(r // 2, device=x.device, dtype=torch.float64)
    axis = torch.repeat_interleave(torch.arange(len(state["sections"]), device=x.device),
                                   torch.tensor(state["sections"], device=x.device))
    angle = positions.double()[axis].T * torch.pow(BASE, -2.0 * i / r)
    cos, sin = angle.cos().float()[:, None], angle.sin().float()[:, None]
    turn, rest = x[..., :r], x[..., r:]
    if state["interleaved"]:
        a, b = turn[..., 0::2], turn[..., 1::2]
        turn = torch.stack((a * cos - b * sin, a * sin + b * cos), -1).flatten(-2)
    else:
        a, b = turn[..., :r // 2], turn[..., r // 2:]
        turn = torch.cat((a * cos - b * sin, a * sin + b * cos), -1)
    return torch.cat((turn, rest), -1)


def _plain_norm_rope(s):
    return (_turned(s["q"], s["wq"], s["positions"], s).to(s["q"].dtype),
            _turned(s["k"], s["wk"], s["positions"], s).to(s["k"].dtype))


def _blocks(s):
    """The pool as [blocks, hkv, 4112]: block id = slot / 16 (a copy)."""
    per = s["page"] // BLOCK
    p = s["pages"].view(-1, s["hkv"], per, BLOCK_BYTES)
    return p.transpose(1, 2).clone(memory_format=torch.contiguous_format).view(-1, s["hkv"], BLOCK_BYTES)


def _rows_into(blocks, at, rows, slots, touched, place):
    """Codes rows [n, hkv, 128] into the key (at = 0) or value (at = 2048) part of the blocks
    `touched` (their ids; place: each token's row among them); the scales grow as they must, and
    start anew in a block whose first token is among the rows."""
    off = slots.long() % BLOCK
    n, hkv = rows.shape[:2]
    most = torch.zeros((len(touched), hkv), device=rows.device)
    most.scatter_reduce_(0, place[:, None].expand(n, hkv), rows.abs().amax(-1), "amax")
    fresh = torch.zeros(len(touched), dtype=torch.bool, device=rows.device)
    fresh[place[off == 0]] = True
    old = blocks[touched]
    e_old = old[..., 4096 + at // 2048].int() - 127
    e_new = _exponent(most)
    e = torch.where(fresh[:, None], e_new, torch.maximum(e_old, e_new))
    part = (_from_layout_k if at == 0 else _from_layout_v)(old[..., at:at + 2048]).view(torch.float8_e4m3fn).float()
    part = torch.where((fresh[:, None] | (e == e_old))[..., None, None], part,
                       torch.ldexp(part, (e_old - e)[..., None, None]))
    part = part.to(torch.float8_e4m3fn).view(torch.uint8)
    part[place, :, off] = torch.ldexp(rows, -e[place][..., None]).to(torch.float8_e4m3fn).view(torch.uint8)
    old[..., at:at + 2048] = (_to_layout_k if at == 0 else _to_layout_v)(part)
    old[..., 4096 + at // 2048] = (e + 127).to(torch.uint8)
    blocks[touched] = old


def _views(pages, hkv):
    """The pool's codes and scales as the values that they are."""
    p = pages.view(pages.shape[0], hkv, -1, BLOCK_BYTES)
    return p[..., :4096].view(torch.float8_e4m3fn), p[..., 4096:4098].view(torch.float8_e8m0fnu)


def _plain_append(s):
    q = _turned(s["q"], s["wq"], s["positions"], s).to(s["q"].dtype)
    k = _turned(s["k"], s["wk"], s["positions"], s)
    blocks = _blocks(s)
    touched, place = torch.unique(s["slots"].long() // BLOCK, return_inverse=True)
    _rows_into(blocks, 0, k, s["slots"], touched, place)
    _rows_into(blocks, 2048, s["v"].float(), s["slots"], touched, place)
    per = s["page"] // BLOCK
    s["pages"].view(-1, s["hkv"], per, BLOCK_BYTES).copy_(
        blocks.view(-1, per, s["hkv"], BLOCK_BYTES).transpose(1, 2))
    return (q,) + _views(s["pages"], s["hkv"])


def _tokens(s):
    """Keys and values [batch, hkv, length, 128] of the sequences' pages, in 32 bits."""
    p = s["pages"][s["table"].long()]  # [batch, width, hkv, page bytes]
    b, w, h = p.shape[:3]
    p = p.view(b, w, h, -1, BLOCK_BYTES).transpose(1, 2).reshape(b, h, -1, BLOCK_BYTES)
    out = []
    for at, put in ((0, _from_layout_k), (2048, _from_layout_v)):
        e = p[..., 4096 + at // 2048].int() - 127
        codes = put(p[..., at:at + 2048]).view(torch.float8_e4m3fn).float()
        out.append(torch.ldexp(codes, e[..., None, None]).reshape(b, h, -1, D))
    return out


def _plain_attend(s):
    k, v = _tokens(s)
    q = s["q"]
    b, t, hq = q.shape[:3]
    g = hq // s["hkv"]
    rows = q.float().view(b, t, s["hkv"], g, D).permute(0, 2, 1, 3, 4).reshape(b, s["hkv"], t * g, D)
    score = rows @ k.transpose(-1, -2) * D ** -0.5
    seen = (s["lens"].long()[:, None] - t + torch.arange(t, device=q.device)).repeat_interleave(g, 1)
    hide = torch.arange(k.shape[2], device=q.device)[None, None] > seen[..., None]  # [b, rows, length]
    score = score.masked_fill_(hide[:, None], -math.inf)
    score = torch.exp(score - score.amax(-1, keepdim=True))
    out = score @ v / score.sum(-1, keepdim=True)
    return out.view(b, s["hkv"], t, g, D).permute(0, 2, 1, 3, 4).reshape(b, t, hq, D).to(q.dtype)


# ------------------------------------------------------------------------------------ the pass

def run(state):
    if not own:
        if state["op"] == "norm_rope":
            return _plain_norm_rope(state)
        return _plain_append(state) if state["op"] == "append" else _plain_attend(state)
    s = state
    if s["op"] == "norm_rope":
        return s["rope"].apply(s["q"], s["k"], s["positions"], q_weight=s["wq"], k_weight=s["wk"], eps=EPS)
    cache = s["cache"]
    if s["op"] == "append":
        q = cache.append_rope(s["k"], s["v"], s["slots"], s["rope"], s["positions"], q=s["q"], q_weight=s["wq"],
                              k_weight=s["wk"], eps=EPS)
        return q, cache.codes(), cache.scales()
    if s["op"] == "extend":
        return cache.extend(s["q"], s["table"], s["lens"])
    if s["q"].shape[1] == 1:
        return cache.decode(s["q"][:, 0], s["table"], s["lens"])[:, None]
    return cache.verify(s["q"], s["table"], s["lens"])


# ------------------------------------------------------------------------------------- the work

def work(case):
    hq, hkv = case["hq"], case["hkv"]
    if case["op"] == "norm_rope":
        n = case["n"]
        return dict(bytes=n * (hq + hkv) * 2 * 2 * D + 4 * n * case["axes"], flops=n * (hq + hkv) * D * 7)
    if case["op"] == "append":
        n = case["batch"] * case["new"]
        coded = 2 * D + 2 / BLOCK
        return dict(bytes=n * (hq * 4 * D + hkv * (4 * D + coded)) + 4 * n * (1 + case["axes"]),
                    flops=n * (hq + 2 * hkv) * D * 7)
    mean = case["most"] if case["least"] == case["most"] else (case["least"] + case["most"]) / 2
    tokens = case["most"] + (case["batch"] - 1) * mean  # expected: the first sequence is the longest
    t, b = case["t"], case["batch"]
    seen = tokens * t - b * t * (t - 1) / 2  # visible (query token, cached token) pairs
    return dict(bytes=tokens * hkv * (2 * D + 2 / BLOCK) + 2 * 2 * D * b * t * hq + 4 * tokens / case["page"],
                flops=4 * D * hq * seen)


# ------------------------------------------------------------------------------- 64-bit definition

def _e4m3_values(device):
    """The value of each e4m3 byte, from the format: sign, 4 exponent bits (bias 7), 3 mantissa bits."""
    v = []
    for byte in range(256):
        e, m = byte >> 3 & 15, byte & 7
        x = math.nan if e == 15 and m == 7 else m / 8 * 2.0 ** -6 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7)
        v.append(-x if byte >> 7 else x)
    return torch.tensor(v, dtype=torch.float64, device=device)


def _places(device):
    """Byte of token r, dim d inside a block: [16, 128] for keys and for values."""
    r = torch.arange(16, device=device)[:, None]
    d = torch.arange(128, device=device)[None]
    k = (((r // 8) * 2 + d // 64) * 32 + (r % 8) * 4 + d % 64 // 16) * 16 + d % 16
    v = 2048 + (d // 32 * 32 + d // 4 % 8 * 4 + r % 8 // 2) * 16 + d % 4 * 4 + r // 8 * 2 + r % 2
    return k, v


def _round_e4m3(x):
    """The nearest e4m3 value (ties to even) of x, |x| <= 448, as its value in 64 bits."""
    _, e = torch.frexp(x)
    step = torch.ldexp(torch.ones_like(x), (e - 1).clamp(min=-6) - 3)
    return torch.round(x / step) * step


def _exact_turn(x, weight, s):
    x = x.double()
    if weight is not None:
        x = x / torch.sqrt((x * x).sum(-1, keepdim=True) / D + EPS) * weight.double()
    r = s["rotary"]
    out = x.clone()
    i = 0
    for axis, pairs in enumerate(s["sections"]):
        for _ in range(pairs):
            angle = s["positions"][axis].double() * BASE ** (-2.0 * i / r)
            a, b = (2 * i, 2 * i + 1) if s["interleaved"] else (i, i + r // 2)
            z = torch.complex(x[..., a], x[..., b]) * torch.polar(torch.ones_like(angle), angle)[:, None]
            out[..., a], out[..., b] = z.real, z.imag
            i += 1
    return out


def _exact_append(s):
    dev = s["q"].device
    per, hkv = s["page"] // BLOCK, s["hkv"]
    value, places = _e4m3_values(dev), _places(dev)
    new = (_exact_turn(s["k"], s["wk"], s), s["v"].double())
    pages = s["pages"].view(-1, hkv, per, BLOCK_BYTES)
    codes = value[pages[..., :4096].int()]  # [pages, hkv, per, 4096], in their places
    exps = pages[..., 4096:4098].int() - 127
    slot = s["slots"].long()
    page, blk, off = slot // s["page"], slot % s["page"] // BLOCK, slot % BLOCK
    key = page * per + blk
    for kind in (0, 1):
        x = new[kind]
        top = torch.full((pages.shape[0] * per, hkv), -1.0, dtype=torch.float64, device=dev)
        top.index_reduce_(0, key, x.abs().amax(-1), "amax")
        need = torch.ceil(torch.log2(top.clamp(min=2.0 ** -200) / 448)).int()
        need = need + (top > 448 * torch.exp2(need.double())).int()  # log2 next to a border
        need = need - (top <= 448 * torch.exp2(need.double() - 1)).int()
        need = need.clamp(E_MIN, E_MAX).view(-1, per, hkv).transpose(1, 2)
        hit = (top >= 0).view(-1, per, hkv).transpose(1, 2)
        anew = torch.zeros(pages.shape[0] * per, dtype=torch.bool, device=dev)
        anew[key[off == 0]] = True
        anew = anew.view(-1, 1, per).expand(-1, hkv, per)
        was = exps[..., kind].clone()
        now = torch.where(hit, torch.where(anew, need, torch.maximum(was, need)), was)
        exps[..., kind] = now
        part = codes[..., 2048 * kind:2048 * kind + 2048]
        grown = (now > was) & ~anew
        part[grown] = _round_e4m3(part[grown] * torch.exp2((was - now)[grown].double())[:, None])
        rows = _round_e4m3(x * torch.exp2(-now[page, :, blk].double())[..., None])  # [n, hkv, 128]
        at = places[kind][off] - 2048 * kind  # [n, 128]
        h = torch.arange(hkv, device=dev)
        part[page[:, None, None], h[None, :, None], blk[:, None, None], at[:, None]] = rows
    return _exact_turn(s["q"], s["wq"], s), codes, torch.exp2(exps.double())


def _exact_attend(s, case):
    dev, q, hkv = s["q"].device, s["q"], s["hkv"]
    value, places = _e4m3_values(dev), _places(dev)
    b, t, hq = q.shape[:3]
    g = hq // hkv
    out = torch.zeros(q.shape, dtype=torch.float64, device=dev)
    pages = s["pages"].view(-1, hkv, s["page"] // BLOCK, BLOCK_BYTES)
    for i, length in enumerate(s["lens"].tolist()):
        used = s["table"][i, :(length + s["page"] - 1) // s["page"]].long()
        for h in range(hkv):
            raw = pages[used, h].reshape(-1, BLOCK_BYTES)
            scale = torch.exp2(raw[:, 4096:4098].double() - 127)
            k, v = ((value[raw[:, places[c].reshape(-1)].int()] * scale[:, c, None]).view(-1, D)[:length] for c in (0, 1))
            rows = q[i, :, h * g:(h + 1) * g].double().reshape(t * g, D)
            z = rows @ k.T / math.sqrt(D)
            last = length - t + torch.arange(t, device=dev).repeat_interleave(g)
            z[torch.arange(length, device=dev)[None] > last[:, None]] = -math.inf
            out[i, :, h * g:(h + 1) * g] = (torch.softmax(z, -1) @ v).view(t, g, D)
    return out


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "norm_rope":
        return _exact_turn(s["q"], s["wq"], s), _exact_turn(s["k"], s["wk"], s)
    return _exact_append(s) if case["op"] == "append" else _exact_attend(s, case)
