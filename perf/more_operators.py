"""Measured cases of latent attention: the append to a paged cache that holds one latent vector a token
(8 bits) and one position part that all heads share (16 bits), attention over that cache in its absorbed
form (decode, chain and tree verify), reading the cache back, and attention of a prompt in its expanded form.

`run` computes each operator in elementary torch operations, or, with `own`, through the framework's
entry points; `exact` gives the same from the definition in 64 bits.

The cache: a page of P tokens is P * 641 bytes.  Dim d (of 512) of token r is the e4m3 code at byte
d/128 * P*128 + r * 128 + (d%128/16 ^ r%8) * 16 + d%16, dim i (of 64) of its position part the 16-bit value at
512 P + r * 128 + (i/8 ^ r%8) * 16 + i%8 * 2, both times 2^E with the exponent byte E + 127 at 640 P + r.  E is
the smallest in [-60, 60] with which the codes stay within 448 and the position part within 2^15.
"""
import math
import random

import torch

own = False

LATENT, PE, NOPE, VALUE = 512, 64, 128, 128
TOKEN_BYTES = 641
E_MIN, E_MAX = -60, 60
BASE = 10000.0
EPS = 1e-6
SCALE = (NOPE + PE) ** -0.5


# ------------------------------------------------------------------------------------- cases

def listed():
    return [
        # the newest token of 64 sequences and its queries' position parts: a decode step, latency
        dict(name="append step 64", op="append", batch=64, new=1, start=4097, heads=128, page=64, dtype="bfloat16",
             interleaved=True, norm=True),
        # a prompt of one sequence that starts inside a page, the heads of one of several GPUs
        dict(name="append prompt 32768", op="append", batch=1, new=32768, start=1000, heads=16, page=16,
             dtype="bfloat16", interleaved=False, norm=True),
        # one short sequence, few heads: latency
        dict(name="decode 1x1024", op="attend", batch=1, least=1024, most=1024, t=1, heads=16, page=16,
             dtype="float16", tree=False),
        # a server's batch of ragged lengths, the heads of one of several GPUs
        dict(name="decode 32x1K-32K", op="attend", batch=32, least=1024, most=32768, t=1, heads=16, page=64,
             dtype="bfloat16", tree=False),
        # many sequences of equal length, all heads on one GPU
        dict(name="decode 64x16K", op="attend", batch=64, least=16384, most=16384, t=1, heads=128, page=64,
             dtype="bfloat16", tree=False),
        # a chain of 4 drafted tokens to be verified
        dict(name="verify 8x16K+4", op="attend", batch=8, least=16388, most=16388, t=4, heads=32, page=16,
             dtype="float16", tree=False),
        # a tree of drafted tokens over ragged sequences, an odd number of heads
        dict(name="tree 5x500-9K+13", op="attend", batch=5, least=500, most=9001, t=13, heads=20, page=32,
             dtype="bfloat16", tree=True),
        # the cached prefix of one sequence, read back to be expanded
        dict(name="read 1x1500", op="read", batch=1, least=1500, most=1500, page=16, dtype="float16"),
        # the prefixes of a batch, ragged
        dict(name="read 16x1K-16K", op="read", batch=16, least=1024, most=16384, page=64, dtype="bfloat16"),
        # a long prompt of one sequence
        dict(name="prompt 1x16384", op="prompt", batch=1, least_new=16384, new=16384, least_old=0, old=0, heads=16,
             dtype="bfloat16"),
        # a chunk of 512 tokens each over 8K cached ones
        dict(name="prompt 4x512 of 8K", op="prompt", batch=4, least_new=512, new=512, least_old=7680, old=7680,
             heads=64, dtype="bfloat16"),
        # short ragged prompts of odd sizes, some over a prefix
        dict(name="prompt 6x1-400", op="prompt", batch=6, least_new=1, new=400, least_old=0, old=300, heads=5,
             dtype="float16"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["append", "attend", "attend", "read", "prompt", "prompt"])
    heads = rng.choice([1, 2, 4, 5, 8, 16, 16, 20, 32, 40, 64, 128])
    dtype = rng.choice(["float16", "bfloat16"])
    page = rng.choice([16, 32, 48, 64, 128, 256])
    if op == "append":
        if rng.random() < 0.5:
            batch, new = _log(rng, 1, 256), rng.choice([1, 1, 2, 5, 8])
        else:
            batch = rng.randint(1, 4)
            new = _log(rng, 16, 32768 // batch)
        heads = min(heads, max(1, 32768 * 16 // (batch * new)))
        return dict(op=op, batch=batch, new=new, start=_log(rng, 1, 8192) - 1, heads=heads, page=page, dtype=dtype,
                    interleaved=rng.random() < 0.5, norm=rng.random() < 0.7)
    if op == "read":
        batch = _log(rng, 1, 64)
        most = _log(rng, 16, 131072 // batch)
        return dict(op=op, batch=batch, least=max(1, most // rng.choice([1, 4, 16])), most=most, page=page, dtype=dtype)
    if op == "attend":
        tree = rng.random() < 0.25
        t = rng.choice([3, 7, 13, 16]) if tree else rng.choice([1, 1, 1, 2, 4, 6])
        batch = _log(rng, 1, 64)
        room = 64 * 16384 * 128 // (batch * max(t * heads, 64))
        most = _log(rng, 64, min(65536, 64 * 16384 // batch, room))
        return dict(op=op, batch=batch, least=max(t, most // rng.choice([1, 4, 32])), most=max(t, most), t=t,
                    heads=heads, page=page, dtype=dtype, tree=tree)
    batch = rng.randint(1, 8)
    new = _log(rng, 8, 8192)
    old = rng.choice([0, 0, _log(rng, 1, 16384)])
    while batch * new * (old + new / 2) * heads > 16384 * 8192 * 16 or batch * (old + new) * heads > 4 * 8192 * 64:
        new, old = max(1, new // 2), old // 2
    part = rng.choice([1, 2, 8])
    return dict(op=op, batch=batch, least_new=max(1, new // part), new=new, least_old=old // part, old=old, heads=heads,
                dtype=dtype)


# ------------------------------------------------------------------------------------ inputs

def _lengths(lo, hi, n):
    """n whole numbers of [lo, hi], the first one hi: the same for every seed, so that outputs keep their shapes."""
    rng = random.Random(31 * hi + n)
    return [hi] + [rng.randint(lo, hi) for _ in range(n - 1)]


def _exponent(top_c, top_pe):
    """The smallest E in [E_MIN, E_MAX] with top_c <= 448 * 2^E (448 = 0.875 * 2^9) and top_pe <= 2^(15 + E)."""
    m, e = torch.frexp(top_c)
    for_c = torch.where(top_c > 0, torch.where(m <= 0.875, e - 9, e - 8), E_MIN)
    m, e = torch.frexp(top_pe)
    for_pe = torch.where(top_pe > 0, torch.where(m == 0.5, e - 16, e - 15), E_MIN)
    return torch.maximum(for_c, for_pe).clamp(E_MIN, E_MAX)


def _turned_chunks(x):
    """x [..., tokens, 8, bytes]: the 16-byte chunks of token r in the order j ^ r%8 (its own inverse)."""
    r = torch.arange(8, device=x.device)
    x = x.unflatten(-3, (-1, 8))
    return x[..., r[:, None], r[:, None] ^ r, :].flatten(-4, -3)


def _parts(pages, page):
    """The three parts of pages uint8 [n, P * 641]: codes [n, 4, P, 128], position parts [n, P, 128], exponents [n, P]."""
    return (pages[:, :512 * page].unflatten(1, (4, page, 128)), pages[:, 512 * page:640 * page].unflatten(1, (page, 128)),
            pages[:, 640 * page:])


def _pool(num_pages, page, dtype, gen, device):
    """A cache in use: latents as a norm leaves them, some dims larger, and position parts of a larger size."""
    pages = torch.zeros((num_pages, page * TOKEN_BYTES), dtype=torch.uint8, device=device)
    gain = torch.ones(LATENT, device=device)
    gain[torch.randperm(LATENT, generator=gen, device=device)[:8]] = 6.0
    step = max(1, (1 << 25) // (page * LATENT))
    for lo in range(0, num_pages, step):
        codes, pe, exps = _parts(pages[lo:lo + step], page)
        c = torch.randn((codes.shape[0], page, LATENT), generator=gen, device=device) * gain
        p = 2 * torch.randn((codes.shape[0], page, PE), generator=gen, device=device)
        e = _exponent(c.abs().amax(-1), p.abs().amax(-1))
        c = torch.ldexp(c, -e[..., None]).to(torch.float8_e4m3fn).view(torch.uint8)
        c = c.unflatten(-1, (4, 8, 16)).permute(0, 2, 1, 3, 4)  # [n, 4, P, 8, 16]
        codes.copy_(_turned_chunks(c).flatten(-2))
        p = torch.ldexp(p, -e[..., None]).to(dtype).view(torch.uint8).unflatten(-1, (8, 16))
        pe.copy_(_turned_chunks(p).flatten(-2))
        exps.copy_((e + 127).to(torch.uint8))
    return pages


def _table(lens, page, gen, device):
    """Pages of all sequences in a random order: block table [batch, most pages], pages in all."""
    need = (lens.cpu() + page - 1) // page
    width, total = int(need.max()), int(need.sum())
    table = torch.zeros((len(lens), width), dtype=torch.int32, device=device)
    mask = torch.arange(width, device=device)[None] < need.to(device)[:, None]
    table[mask] = torch.randperm(total, generator=gen, device=device).to(torch.int32)
    return table, total


def _offsets(lens):
    return torch.cat((torch.zeros(1, dtype=torch.int32, device=lens.device), lens.cumsum(0).to(torch.int32)))


def _tree(batch, t, gen, device):
    """Draft trees: draft j's parent is a draft before it, or none; a draft sees its ancestors and itself."""
    parent = (torch.rand((batch, t), generator=gen, device=device) * torch.arange(1, t + 1, device=device)).long() - 1
    see = torch.zeros((batch, t, t), dtype=torch.bool, device=device)
    rows = torch.arange(batch, device=device)
    for j in range(t):
        up = parent[:, j]
        see[:, j] = see[rows, up.clamp(min=0)] & (up >= 0)[:, None]
        see[:, j, j] = True
    return (see.long() << torch.arange(t, device=device)).sum(-1)


def _handles(case, state, device):
    """What a program of the framework keeps: the cache and the rotation."""
    from rotation_quantized_kv_rq_gb300 import rq
    if case["op"] == "prompt":
        state["status"] = torch.zeros(1, dtype=torch.int32, device=device)
        return
    state["cache"] = rq.LatentCache(case.get("heads", 1), case["page"], state["pages"].shape[0], max_batch=case["batch"],
                                    max_query_tokens=case.get("t", 1), max_pages_per_seq=state["table"].shape[1],
                                    sm_scale=SCALE, device=device, dtype=getattr(torch, case["dtype"]),
                                    pages=state["pages"])
    if case["op"] == "append":
        state["rope"] = rq.Rope(PE, base=BASE, interleaved=case["interleaved"], device=device)


def prepare(case, seed):
    device = torch.device("cuda", torch.cuda.current_device())
    gen = torch.Generator(device=device)
    gen.manual_seed(seed)
    dtype = getattr(torch, case["dtype"])
    op, batch, page = case["op"], case["batch"], case.get("page")
    state = dict(op=op, page=page, dtype=dtype)

    def randn(*shape):
        return torch.randn(shape, generator=gen, device=device)

    if op == "append":
        new, start, n = case["new"], case["start"], batch * case["new"]
        first = start + torch.arange(batch, device=device) % 32
        state["table"], pages = _table(first + new, page, gen, device)
        pos = first[:, None] + torch.arange(new, device=device)
        seq = torch.arange(batch, device=device)[:, None]
        state["slots"] = (state["table"][seq, pos // page] * page + pos % page).reshape(-1).to(torch.int32)
        state["positions"] = pos.reshape(-1).to(torch.int32)
        state["pages"] = _pool(pages, page, dtype, gen, device)
        down = randn(n, LATENT + PE)  # the down projection's output: the latent and the shared position part
        down[:, :4] *= 8.0
        down = down.to(dtype)
        state.update(c=down[:, :LATENT], k_pe=down[:, LATENT:])
        state["q_pe"] = randn(n, case["heads"], NOPE + PE).to(dtype)[..., NOPE:]  # a slice of the query projection
        state["weight"] = 1 + 0.1 * randn(LATENT) if case["norm"] else None
        state["interleaved"] = case["interleaved"]
    elif op in ("attend", "read"):
        lens = torch.tensor(_lengths(case["least"], case["most"], batch), device=device)
        state["lens"] = lens.to(torch.int32)
        state["table"], pages = _table(lens, page, gen, device)
        state["pages"] = _pool(pages, page, dtype, gen, device)
        if op == "read":
            state["offsets"], state["rows"] = _offsets(lens), int(lens.sum())
        else:
            t, heads = case["t"], case["heads"]
            # the queries in the latents' space as a product for each head gives them, [heads][tokens][512]
            state["q_c"] = randn(heads, batch * t, LATENT).to(dtype).transpose(0, 1).unflatten(0, (batch, t))
            state["q_pe"] = randn(batch, t, heads, NOPE + PE).to(dtype)[..., NOPE:]
            state["tree"] = _tree(batch, t, gen, device) if case["tree"] else None
    else:
        heads = case["heads"]
        new, old = (torch.tensor(_lengths(case["least_" + k], case[k], batch), device=device) for k in ("new", "old"))
        state["q_offsets"], state["k_offsets"] = _offsets(new), _offsets(new + old)
        state["max_new"] = int(new.max())
        nk = int((new + old).sum())
        state["q"] = randn(int(new.sum()), heads, NOPE + PE).to(dtype)
        kv = randn(nk, heads, NOPE + VALUE).to(dtype)  # the up projection's output: keys and values of each head
        state.update(k=kv[..., :NOPE], v=kv[..., NOPE:], k_pe=(2 * randn(nk, PE)).to(dtype))
    if own:
        _handles(case, state, device)
    return state


# ----------------------------------------------------------------------------------- plain forms

def _turned(x, positions, interleaved):
    """The position rotation of x [n, heads, 64], in 32 bits; angles in 64."""
    i = torch.arange(PE // 2, device=x.device, dtype=torch.float64)
    angle = positions.double()[:, None] * torch.pow(BASE, -2.0 * i / PE)
    cos, sin = angle.cos().float()[:, None], angle.sin().float()[:, None]
    if interleaved:
        a, b = x[..., 0::2], x[..., 1::2]
        return torch.stack((a * cos - b * sin, a * sin + b * cos), -1).flatten(-2)
    a, b = x[..., :PE // 2], x[..., PE // 2:]
    return torch.cat((a * cos - b * sin, a * sin + b * cos), -1)


def _views(pages, page, dtype):
    """The pool's codes, position parts and scales as the values that they are."""
    codes, pe, exps = _parts(pages, page)
    return codes.view(torch.float8_e4m3fn), pe.view(dtype), exps.view(torch.float8_e8m0fnu)


def _plain_append(s):
    page = s["page"]
    c = s["c"].float()
    if s["weight"] is not None:
        c = c * torch.rsqrt(c.square().mean(-1, keepdim=True) + EPS) * s["weight"]
    pe = _turned(s["k_pe"].float()[:, None], s["positions"], s["interleaved"])[:, 0]
    q_pe = _turned(s["q_pe"].float(), s["positions"], s["interleaved"]).to(s["dtype"])
    e = _exponent(c.abs().amax(-1), pe.abs().amax(-1))
    c = torch.ldexp(c, -e[:, None]).to(torch.float8_e4m3fn).view(torch.uint8).unflatten(-1, (4, 8, 16))
    pe = torch.ldexp(pe, -e[:, None]).to(s["dtype"]).view(torch.uint8).unflatten(-1, (8, 16))
    slot = s["slots"].long()
    where, r = slot // page, slot % page
    order = (torch.arange(8, device=c.device) ^ r[:, None] % 8)[:, :, None]  # chunk j stands at j ^ r%8
    c = c.gather(2, order[:, None].expand(-1, 4, 8, 16)).flatten(-2)
    pe = pe.gather(1, order.expand(-1, 8, 16)).flatten(-2)
    codes, pes, exps = _parts(s["pages"], page)
    codes[where, :, r], pes[where, r], exps[where, r] = c, pe, (e + 127).to(torch.uint8)
    return (q_pe,) + _views(s["pages"], page, s["dtype"])


def _tokens(pages, page, dtype):
    """Latents [n, P, 512] and position parts [n, P, 64] of pages, in 32 bits."""
    codes, pe, exps = _parts(pages, page)
    scale = torch.where(exps == 255, math.nan, torch.exp2(exps.float().clamp(127 + E_MIN, 127 + E_MAX) - 127))[..., None]
    c = _turned_chunks(codes.unflatten(-1, (8, 16)))  # [n, 4, P, 8, 16]
    c = c.permute(0, 2, 1, 3, 4).flatten(2).view(torch.float8_e4m3fn).float()
    p = _turned_chunks(pe.unflatten(-1, (8, 16))).flatten(-2).view(dtype).float()
    return c * scale, p * scale


def _plain_attend(s):
    c, pe = _tokens(s["pages"][s["table"].long().flatten()], s["page"], s["dtype"])
    b, t, heads = s["q_c"].shape[:3]
    k = torch.cat((c, pe), -1).view(b, -1, LATENT + PE)
    q = torch.cat((s["q_c"].float(), s["q_pe"].float()), -1).view(b, t * heads, LATENT + PE)
    score = q @ k.transpose(-1, -2) * SCALE
    at = torch.arange(k.shape[1], device=q.device)
    before = (s["lens"].long()[:, None] - t).expand(b, t)  # what every draft sees
    draft = at - before[..., None]  # [b, t, length]
    if s["tree"] is None:
        see = draft <= torch.arange(t, device=q.device)[:, None]
    else:
        see = (draft < 0) | ((s["tree"][..., None] >> draft.clamp(0, 63) & 1).bool() & (draft < t))
    score = score.masked_fill_(~see.repeat_interleave(heads, 1), -math.inf)
    score = torch.exp(score - score.amax(-1, keepdim=True))
    out = score @ k[..., :LATENT] / score.sum(-1, keepdim=True)
    return out.view(b, t, heads, LATENT).to(s["dtype"])


def _plain_read(s):
    n, page = s["rows"], s["page"]
    row = torch.arange(n, device=s["pages"].device)
    seq = torch.searchsorted(s["offsets"][1:].long(), row, right=True)
    at = row - s["offsets"].long()[seq]
    where, r = s["table"].long()[seq, at // page], at % page
    c, pe = _tokens(s["pages"], page, s["dtype"])
    return c[where, r].to(s["dtype"]), pe[where, r].to(s["dtype"])


def _plain_prompt(s):
    q, k, v = s["q"], s["k"], s["v"]
    out = torch.zeros((q.shape[0], q.shape[1], VALUE), dtype=q.dtype, device=q.device)
    qo, ko = s["q_offsets"].tolist(), s["k_offsets"].tolist()
    for i in range(len(qo) - 1):
        keys, ahead = slice(ko[i], ko[i + 1]), ko[i + 1] - ko[i] - (qo[i + 1] - qo[i])
        kk = torch.cat((k[keys], s["k_pe"][keys, None].expand(-1, k.shape[1], -1)), -1).float().permute(1, 2, 0)
        vv = v[keys].float().transpose(0, 1)
        for lo in range(qo[i], qo[i + 1], 1024):
            hi = min(lo + 1024, qo[i + 1])
            end = ahead + hi - qo[i]
            score = q[lo:hi].float().transpose(0, 1) @ kk[..., :end] * SCALE
            last = ahead + torch.arange(lo, hi, device=q.device) - qo[i]
            score = score.masked_fill_(torch.arange(end, device=q.device) > last[:, None], -math.inf)
            score = torch.exp(score - score.amax(-1, keepdim=True))
            out[lo:hi] = (score @ vv[:, :end] / score.sum(-1, keepdim=True)).transpose(0, 1).to(q.dtype)
    return out


# ------------------------------------------------------------------------------------ the pass

def run(state):
    s = state
    if not own:
        return dict(append=_plain_append, attend=_plain_attend, read=_plain_read, prompt=_plain_prompt)[s["op"]](s)
    if s["op"] == "prompt":
        from rotation_quantized_kv_rq_gb300 import rq
        return rq.prompt_attention(s["q"], s["k"], s["k_pe"], s["v"], s["q_offsets"], s["k_offsets"], s["max_new"],
                                   sm_scale=SCALE, status=s["status"])
    cache = s["cache"]
    if s["op"] == "append":
        q_pe = cache.append(s["c"], s["k_pe"], s["slots"], rope=s["rope"], positions=s["positions"],
                            weight=s["weight"], eps=EPS, q_pe=s["q_pe"])
        return q_pe, cache.codes(), cache.position_parts(), cache.scales()
    if s["op"] == "read":
        return cache.read(s["table"], s["offsets"], s["rows"])
    if s["tree"] is not None:
        return cache.tree_verify(s["q_c"], s["q_pe"], s["tree"], s["table"], s["lens"])
    if s["q_c"].shape[1] == 1:
        return cache.decode(s["q_c"][:, 0], s["q_pe"][:, 0], s["table"], s["lens"])[:, None]
    return cache.verify(s["q_c"], s["q_pe"], s["table"], s["lens"])


# ------------------------------------------------------------------------------------- the work

def work(case):
    batch = case["batch"]
    if case["op"] == "append":
        n, heads = batch * case["new"], case["heads"]
        return dict(bytes=n * (2 * (LATENT + PE) + TOKEN_BYTES + 4 * PE * heads + 8) + (4 * LATENT if case["norm"] else 0),
                    flops=n * (4 * LATENT + 3 * PE * (1 + heads)))

    if case["op"] == "prompt":
        heads = case["heads"]
        news, olds = (_lengths(case["least_" + k], case[k], batch) for k in ("new", "old"))
        new, old, pairs = sum(news), sum(olds), sum(a * b + a * (a + 1) / 2 for a, b in zip(news, olds))
        return dict(bytes=2 * (new * heads * (NOPE + PE + VALUE) + (new + old) * (heads * (NOPE + VALUE) + PE)),
                    flops=2 * (NOPE + PE + VALUE) * heads * pairs)
    tokens = sum(_lengths(case["least"], case["most"], batch))
    cached = tokens * TOKEN_BYTES + 4 * tokens / case["page"]
    if case["op"] == "read":
        return dict(bytes=cached + tokens * 2 * (LATENT + PE), flops=tokens * (LATENT + PE))
    t, heads = case["t"], case["heads"]
    seen = tokens * t - batch * t * (t - 1) / 2  # visible (query token, cached token) pairs of a chain
    return dict(bytes=cached + 2 * batch * t * heads * (2 * LATENT + PE), flops=2 * (2 * LATENT + PE) * heads * seen)


# ------------------------------------------------------------------------------- 64-bit definition

def _e4m3_values(device):
    """The value of each e4m3 byte, from the format: sign, 4 exponent bits (bias 7), 3 mantissa bits."""
    v = []
    for byte in range(256):
        e, m = byte >> 3 & 15, byte & 7
        x = math.nan if e == 15 and m == 7 else m / 8 * 2.0 ** -6 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7)
        v.append(-x if byte >> 7 else x)
    return torch.tensor(v, dtype=torch.float64, device=device)


def _round(x, bits, least):
    """x to `bits` significant bits (ties to even), with the spacing of values near 2^least below that."""
    _, e = torch.frexp(x)
    step = torch.ldexp(torch.ones_like(x), (e - 1).clamp(min=least) - (bits - 1))
    return torch.round(x / step) * step


def _exact_turn(x, s):
    out = x.double().clone()
    for i in range(PE // 2):
        angle = s["positions"].double() * BASE ** (-2.0 * i / PE)
        a, b = (2 * i, 2 * i + 1) if s["interleaved"] else (i, i + PE // 2)
        z = torch.complex(out[..., a], out[..., b]) * torch.polar(torch.ones_like(angle), angle)[:, None]
        out[..., a], out[..., b] = z.real, z.imag
    return out


def _exact_append(s):
    dev, page, half = s["c"].device, s["page"], s["dtype"] == torch.float16
    c = s["c"].double()
    if s["weight"] is not None:
        c = c / torch.sqrt((c * c).sum(-1, keepdim=True) / LATENT + EPS) * s["weight"].double()
    pe = _exact_turn(s["k_pe"][:, None], s)[:, 0]
    e = torch.full((len(c),), E_MIN, device=dev)
    for _ in range(E_MAX - E_MIN):
        grow = (c.abs().amax(-1) > 448 * torch.exp2(e.double())) | (pe.abs().amax(-1) > torch.exp2(15.0 + e.double()))
        e += (grow & (e < E_MAX)).int()
    down = torch.exp2(-e.double())[:, None]
    c, pe = _round(c * down, 4, -6), _round(pe * down, *((11, -14) if half else (8, -126)))
    n = s["pages"].shape[0]
    codes = _e4m3_values(dev)[s["pages"][:, :512 * page].int()]
    pes = s["pages"][:, 512 * page:640 * page].view(s["dtype"]).double()
    exps = s["pages"][:, 640 * page:].int() - 127
    where, r = s["slots"].long() // page, s["slots"].long() % page
    d, i = torch.arange(LATENT, device=dev), torch.arange(PE, device=dev)
    r_ = r[:, None]
    codes[where[:, None], d // 128 * page * 128 + r_ * 128 + (d % 128 // 16 ^ r_ % 8) * 16 + d % 16] = c
    pes[where[:, None], r_ * 64 + (i // 8 ^ r_ % 8) * 8 + i % 8] = pe
    exps[where, r] = e.int()
    return _exact_turn(s["q_pe"], s), codes.view(n, 4, page, 128), pes.view(n, page, 64), torch.exp2(exps.double())


def _exact_tokens(s, seq, length):
    """Latents [length, 512] and position parts [length, 64] of a sequence."""
    dev, page = s["pages"].device, s["page"]
    value = _e4m3_values(dev)
    d, i = torch.arange(LATENT, device=dev), torch.arange(PE, device=dev)
    latents, parts = [], []
    for lo in range(0, length, 1024):
        at = torch.arange(lo, min(lo + 1024, length), device=dev)
        raw, r = s["pages"][s["table"][seq, at // page].long()], (at % page)[:, None]
        c = value[raw.gather(1, d // 128 * page * 128 + r * 128 + (d % 128 // 16 ^ r % 8) * 16 + d % 16).int()]
        place = 512 * page + r * 128 + (i // 8 ^ r % 8) * 16 + i % 8 * 2
        pe = raw.gather(1, place).int() | raw.gather(1, place + 1).int() << 8
        scale = torch.exp2(raw.gather(1, 640 * page + r).double() - 127)
        latents.append(c * scale)
        parts.append(pe.to(torch.int16).view(s["dtype"]).double() * scale)
    return torch.cat(latents), torch.cat(parts)


def _exact_attend(s):
    b, t, heads = s["q_c"].shape[:3]
    out = torch.zeros((b, t, heads, LATENT), dtype=torch.float64, device=s["q_c"].device)
    for i, length in enumerate(s["lens"].tolist()):
        c, pe = _exact_tokens(s, i, length)
        at = torch.arange(length, device=c.device)
        for j in range(t):
            z = (s["q_c"][i, j].double() @ c.T + s["q_pe"][i, j].double() @ pe.T) / math.sqrt(NOPE + PE)
            if s["tree"] is None:
                hide = at > length - t + j
            else:
                bits = torch.tensor([int(s["tree"][i, j]) >> k & 1 for k in range(t)], device=c.device)
                hide = torch.zeros_like(at, dtype=torch.bool)
                hide[length - t:] = bits == 0
            z[:, hide] = -math.inf
            out[i, j] = torch.softmax(z, -1) @ c
    return out


def _exact_read(s):
    c, pe = zip(*(_exact_tokens(s, i, length) for i, length in enumerate(s["lens"].tolist())))
    return torch.cat(c), torch.cat(pe)


def _exact_prompt(s):
    q, k, v, pe = (s[x].double() for x in ("q", "k", "v", "k_pe"))
    out = torch.zeros((q.shape[0], q.shape[1], VALUE), dtype=torch.float64, device=q.device)
    qo, ko = s["q_offsets"].tolist(), s["k_offsets"].tolist()
    for i in range(len(qo) - 1):
        nq, nk = qo[i + 1] - qo[i], ko[i + 1] - ko[i]
        for h in range(q.shape[1]):
            for lo in range(0, nq, 4096):
                rows = q[qo[i] + lo:qo[i] + min(lo + 4096, nq), h]
                end = nk - nq + lo + len(rows)
                z = (rows[:, :NOPE] @ k[ko[i]:ko[i] + end, h].T + rows[:, NOPE:] @ pe[ko[i]:ko[i] + end].T) * SCALE
                z += torch.full_like(z, -math.inf).triu(nk - nq + lo + 1)
                out[qo[i] + lo:qo[i] + lo + len(rows), h] = torch.softmax(z, -1) @ v[ko[i]:ko[i] + end, h]
    return out


def exact(case, seed):
    s = prepare(case, seed)
    return dict(append=_exact_append, attend=_exact_attend, read=_exact_read, prompt=_exact_prompt)[case["op"]](s)
