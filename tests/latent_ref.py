"""The cache of latents and attention over it, from their definitions in float64.  Test infrastructure: shares no code with
the library."""
from __future__ import annotations

import math

import numpy as np
import torch

from tests import block_ref as R

LATENT, PE = 512, 64
DIM, PART = np.arange(LATENT), np.arange(PE)


def code_place(P, r, d):
    return d // 128 * 128 * P + 128 * r + ((d % 128 // 16) ^ (r % 8)) * 16 + d % 16


def part_place(P, r, i):
    return 512 * P + 128 * r + ((i // 8) ^ (r % 8)) * 16 + 2 * (i % 8)


def exponent(top_c, top_pe):
    e = R.E_MIN
    while e < R.E_MAX and (top_c > 448 * 2.0 ** e or top_pe > 2.0 ** (15 + e)):
        e += 1
    return e


def coded(c, pe, dtype):
    """A token's codes (values), position part (before the scale) and exponent; None where it is stored as NaN."""
    if not (np.isfinite(c).all() and np.isfinite(pe).all()):
        return None
    e = exponent(np.abs(c).max(), np.abs(pe).max())
    part = np.clip(pe * 2.0 ** -e, -2.0 ** 15, 2.0 ** 15)
    return R.round_e4m3(c * 2.0 ** -e), torch.from_numpy(part).to(dtype).double().numpy(), e


def unpack(pages, P, dtype):
    """uint8 [n][641 P] -> codes (values) [n * P][512], position parts [n * P][64] before the scale, exponent bytes [n * P]."""
    pages = np.asarray(pages)
    n = len(pages)
    r = np.arange(P)[:, None]
    codes = R.VALUES[pages[:, code_place(P, r, DIM)]].reshape(n * P, LATENT)
    at = part_place(P, r, PART)
    raw = np.stack((pages[:, at], pages[:, at + 1]), -1).copy().view(np.int16)[..., 0]
    part = torch.from_numpy(raw).view(dtype).double().numpy().reshape(n * P, PE)
    return codes, part, pages[:, 640 * P:].reshape(n * P).astype(int)


def scale(byte):
    """2^E of exponent bytes; NaN for 255."""
    e = np.clip(np.asarray(byte) - 127, R.E_MIN, R.E_MAX)
    return np.where(np.asarray(byte) == 255, np.nan, 2.0 ** e)


def fill(P, num_pages, dtype, rng, spread=1.0, garbage=False):
    """A pool [num_pages][641 P] of coded random tokens of differing magnitudes (2^+-spread); garbage: bytes of any value."""
    if garbage:
        return rng.integers(0, 256, (num_pages, 641 * P)).astype(np.uint8)
    pages = np.zeros((num_pages, 641 * P), np.uint8)
    for n in range(num_pages):
        put(pages, P, np.arange(n * P, (n + 1) * P), rng.standard_normal((P, LATENT)) * 2.0 ** rng.uniform(-spread, spread, (P, 1)),
            2 * rng.standard_normal((P, PE)), dtype)
    return pages


CODE_OF = {float(v): i for i, v in reversed(list(enumerate(R.VALUES))) if not math.isnan(v)}


def put(pages, P, slots, c, pe, dtype):
    """Codes tokens into a host pool, by the definition."""
    c, pe = np.asarray(c, np.float64), np.asarray(pe, np.float64)
    top = np.abs(c).max(-1), np.abs(pe).max(-1)
    e = np.array([exponent(a, b) for a, b in zip(*top)])
    down = 2.0 ** -e.astype(float)
    codes = torch.from_numpy(c * down[:, None]).float().to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    part = torch.from_numpy(pe * down[:, None]).to(dtype).view(torch.int16).numpy().astype(np.uint16)
    for i, s in enumerate(slots):
        n, r = divmod(int(s), P)
        pages[n, code_place(P, r, DIM)] = codes[i]
        at = part_place(P, r, PART)
        pages[n, at], pages[n, at + 1] = part[i] & 255, part[i] >> 8
        pages[n, 640 * P + r] = e[i] + 127


def chain(T):
    return lambda b, j, pos, length: pos <= length - T + j


def tree(mask, T):
    def see(b, j, pos, length):
        draft = pos - (length - T)
        bits = np.array([int(mask[b, j]) >> i & 1 for i in range(64)], bool)
        return (draft < 0) | bits[np.clip(draft, 0, 63)]
    return see


def attention(q_c, q_pe, pages, block_table, lens, P, visible, sm_scale, dtype):
    """softmax(sm_scale (q_c . c + q_pe . p)) c in float64 on the GPU, q [B][T][H][512 and 64] (float64 arrays); and how far from
    it a kernel may be that feeds 8-bit multiplications exactly summed pieces, without the output's own rounding:
      a query row is 2^Eq (the least with |q_c| <= 448 2^Eq and |q_pe| <= 2^15 2^Eq) times e4m3 numbers that sum up to it, two for
      bf16 (4 + 4 of its 8 bits), three for fp16: off by half of e4m3's smallest step, 2^-10, where its low bits are below that,
      and an fp16 position part by 2^-25;
      a score is summed in f32 over at most 52 multiply steps, truncated each: 2^-17 of its products' magnitudes, and 2^-17 more
      for its scaling and the exponential's argument;
      a weight times its token's scale, in units of which the row's largest is at least 2^10, is rounded to fp16 (2^-11) and to an
      e5m2 number and one (bf16) or two (fp16) e4m3 numbers: off by 2^-8 (2^-12) of it, or where that is less by min(2^-10,
      an eighth of it), e4m3's and e5m2's steps, or 2^-17, half of e5m2's smallest;
      2^-20 for the exponential and the joins."""
    dev = "cuda"
    B, T, H = q_c.shape[:3]
    codes, part, byte = unpack(pages, P, dtype)
    out = np.zeros((B, T, H, LATENT))
    tol = np.zeros_like(out)
    eps = (2.0 ** -8 if dtype == torch.bfloat16 else 2.0 ** -12) + 2.0 ** -11
    for b in range(B):
        L = int(lens[b])
        if L <= 0:
            continue
        pos = np.arange(L)
        slot = block_table[b, pos // P].astype(np.int64) * P + pos % P
        s_tok = torch.from_numpy(scale(byte[slot])).to(dev)[:, None]
        code = torch.from_numpy(codes[slot]).to(dev)
        p = torch.from_numpy(part[slot]).to(dev) * s_tok
        for j in range(T):
            see = torch.from_numpy(visible(b, j, pos, L)).to(dev)
            if not see.any():
                continue
            cc, pp, sc = code[see], p[see], s_tok[see]
            c = cc * sc
            qc, qp = (torch.from_numpy(x[b, j]).to(dev) for x in (q_c, q_pe))
            score = sm_scale * (qc @ c.T + qp @ pp.T)
            mag = sm_scale * (qc.abs() @ c.abs().T + qp.abs() @ pp.abs().T)
            e = torch.tensor([exponent(a, d) for a, d in zip(qc.abs().amax(-1).tolist(), qp.abs().amax(-1).tolist())],
                             dtype=torch.float64, device=dev)
            off = sm_scale * torch.exp2(e)[:, None] * (2.0 ** -10 * c.abs().sum(-1) + 2.0 ** -25 * pp.abs().sum(-1))
            w = torch.softmax(score, -1)
            moved = (off + mag * 2.0 ** -16).amax(-1, keepdim=True)
            o, spread = w @ c, w @ c.abs()
            ws = w * sc.T
            unit = ws.amax(-1, keepdim=True) * 2.0 ** -10
            u = ws / unit
            lost = torch.maximum(eps * u, torch.minimum(torch.full_like(u, 2.0 ** -10), u / 8).clamp(min=2.0 ** -17))
            out[b, j] = o.cpu()
            tol[b, j] = ((2 * moved + 2.0 ** -20) * spread + (lost * unit) @ cc.abs() * (1 + 2 * moved)).cpu()
    return out, tol


def prompt(q, k, pe, v, qo, ko, sm_scale, dtype):
    """The expanded form in float64 on the GPU from host float64 arrays, and how far a kernel may be off before the output's
    rounding: a score is summed in f32 over 12 steps, truncated (2^-19 of its products' magnitudes, and 2^-17 for its scaling and the
    exponential's argument); a weight is rounded to the type (2^-8, or 2^-11 and 2^-32 of the row's largest); 2^-20 for the rest."""
    dev = "cuda"
    out = np.zeros((len(q), q.shape[1], 128))
    tol = np.zeros_like(out)
    eps = 2.0 ** -8 if dtype == torch.bfloat16 else 2.0 ** -11
    tq, tk, tp, tv = (torch.from_numpy(x).to(dev) for x in (q, k, pe, v))
    for b in range(len(qo) - 1):
        nq, nk = qo[b + 1] - qo[b], ko[b + 1] - ko[b]
        for j in range(nq):
            end = nk - nq + j + 1
            if end <= 0:
                continue
            row = tq[qo[b] + j]
            kk, pp, vv = (x[ko[b]:ko[b] + end] for x in (tk, tp, tv))
            s = sm_scale * (torch.einsum("hd,nhd->hn", row[:, :128], kk) + row[:, 128:] @ pp.T)
            mag = sm_scale * (torch.einsum("hd,nhd->hn", row[:, :128].abs(), kk.abs()) + row[:, 128:].abs() @ pp.abs().T)
            w = torch.softmax(s, -1)
            o = torch.einsum("hn,nhd->hd", w, vv)
            spread = torch.einsum("hn,nhd->hd", w, vv.abs())
            moved = (mag * (2.0 ** -19 + 2.0 ** -17)).amax(-1, keepdim=True)
            low = 2.0 ** -32 * w.amax(-1)[:, None] * vv.abs().sum(0) if dtype == torch.float16 else 0.0
            out[qo[b] + j] = o.cpu()
            tol[qo[b] + j] = ((eps + 2 * moved + 2.0 ** -20) * spread + low).cpu()
    return out, tol
