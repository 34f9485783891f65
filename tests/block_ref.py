"""The 8-bit block-scaled cache, the norms and position rotation, and attention over the cache, from
their definitions in float64, token by token.  Test infrastructure: shares no code with the library."""
from __future__ import annotations

import math

import numpy as np
import torch

D = 128
E_MIN, E_MAX = -60, 60


def e4m3_value(byte: int) -> float:
    e, m = byte >> 3 & 15, byte & 7
    x = math.nan if (e, m) == (15, 7) else m * 2.0 ** -9 if e == 0 else (8 + m) * 2.0 ** (e - 10)
    return -x if byte >> 7 else x


VALUES = np.array([e4m3_value(b) for b in range(256)])


def step_of(x):
    """The spacing of e4m3 values around |x| (the spacing below 2^-6 is that of subnormals)."""
    with np.errstate(divide="ignore"):
        e = np.floor(np.log2(np.abs(x), out=np.full(np.shape(x), -99.0), where=np.asarray(x) != 0))
    return 2.0 ** (np.maximum(e, -6) - 3)


def round_e4m3(x):
    """Nearest e4m3 value, ties to even; infinities to 448, NaN to NaN."""
    x = np.asarray(x, np.float64)
    with np.errstate(invalid="ignore"):
        s = step_of(np.where(np.isfinite(x), x, 1.0))
        y = np.rint(np.where(np.isfinite(x), x, 0.0) / s) * s
    y = np.clip(y, -448, 448)
    return np.where(np.isnan(x), np.nan, np.where(np.isinf(x), np.sign(x) * 448.0, y))


def exponent(amax: float) -> int:
    e = E_MIN
    while e < E_MAX and amax > 448 * 2.0 ** e:
        e += 1
    return e


def key_place(r, d):
    return ((r // 8 * 2 + d // 64) * 32 + r % 8 * 4 + d % 64 // 16) * 16 + d % 16


def value_place(r, d):
    return 2048 + (d // 32 * 32 + d // 4 % 8 * 4 + r % 8 // 2) * 16 + d % 4 * 4 + r // 8 * 2 + r % 2


R, DIM = np.arange(16)[:, None], np.arange(128)[None]
PLACES = (key_place(R, DIM), value_place(R, DIM))


def unpack(pages: np.ndarray, P: int):
    """uint8 [np][H][page bytes] -> codes [2][np][H][P][128] (their values), exponents [2][np][H][P / 16]."""
    n, H = pages.shape[:2]
    blk = pages.reshape(n, H, P // 16, 4112)
    codes = [VALUES[blk[..., p.reshape(-1)]].reshape(n, H, P, D) for p in PLACES]
    exps = [np.clip(blk[..., 4096 + i].astype(int) - 127, E_MIN, E_MAX) for i in (0, 1)]
    return codes, exps


class Cache:
    """What the pool holds, as values: codes and the exponent of each block's scales."""

    def __init__(self, num_pages, H, P):
        self.P = P
        self.codes = [np.zeros((num_pages * P // 16, H, 16, D)) for _ in range(2)]
        self.exps = [np.full((num_pages * P // 16, H), E_MIN) for _ in range(2)]

    def append(self, k, v, slots):
        """k, v: float64 [n][H][128]; tokens of a block stand together."""
        i, n = 0, len(slots)
        while i < n:
            if slots[i] < 0:
                i += 1
                continue
            blk, off, cnt = slots[i] // 16, slots[i] % 16, 1
            while i + cnt < n and slots[i + cnt] == slots[i] + cnt and (slots[i] + cnt) // 16 == blk:
                cnt += 1
            for kind, x in ((0, k), (1, v)):
                for h in range(x.shape[1]):
                    rows = x[i:i + cnt, h]
                    fin = np.abs(rows[np.isfinite(rows)])
                    e = exponent(fin.max() if fin.size else 0.0)
                    old = self.exps[kind][blk, h]
                    if off > 0:
                        e = max(e, old)
                        if e > old:
                            self.codes[kind][blk, h] = round_e4m3(self.codes[kind][blk, h] * 2.0 ** (old - e))
                    self.exps[kind][blk, h] = e
                    self.codes[kind][blk, h, off:off + cnt] = round_e4m3(rows * 2.0 ** -float(e))
            i += cnt


def turn(x, weight, eps, positions, inv_freq, axis=None, interleaved=False, scale=1.0):
    """Norm and rotation of x [n][heads][128] in float64; positions [axes][n].  Also the size that
    rounding errors scale with: |a| + |b| of each pair (|x| past rotary_dim)."""
    x = np.asarray(x, np.float64)
    if weight is not None:
        x = x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * np.asarray(weight, np.float64)
    out, size = x.copy(), np.abs(x)
    half = len(inv_freq)
    for i in range(half):
        # the angle reduced exactly: position times frequency in extended precision
        pos = positions[0 if axis is None else axis[i]].astype(np.int64)
        t = np.array([int(p) * _Turn.of(inv_freq[i]) % (1 << 128) / (1 << 128) for p in pos]) * (2 * math.pi)
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
        c, s = (np.cos(t) * scale)[:, None], (np.sin(t) * scale)[:, None]
        out[..., a], out[..., b] = x[..., a] * c - x[..., b] * s, x[..., a] * s + x[..., b] * c
        size[..., a] = size[..., b] = scale * (np.abs(x[..., a]) + np.abs(x[..., b]))
    return out, size


class _Turn:
    """Frequencies as fractions of a turn times 2^128, in whole numbers."""
    # 1 / (2 pi) * 2^256, from pi's digits
    PI = 31415926535897932384626433832795028841971693993751058209749445923078164062862089986280348253421170679
    INV = (1 << 256) * 10 ** (len(str(PI)) - 1) // (2 * PI)
    seen: dict = {}

    @classmethod
    def of(cls, f):
        if f not in cls.seen:
            num, den = float(f).as_integer_ratio()
            cls.seen[f] = (num * cls.INV // den >> 128) % (1 << 128)
        return cls.seen[f]


def attention(q, cache_codes, cache_exps, block_table, lens, P, visible, sm_scale=None):
    """softmax(sm_scale q K^T) V in float64 on the GPU.  q [B][T][Hq][128]; visible(b, j, positions)
    -> truth values.  Returns the result and how far a kernel with f32 sums and fp16 weights may be
    from it (without the output's own rounding):
      a weight is rounded to fp16: 2^-11 of it, or 2^-25 (of the row's largest weighted scale) where it is subnormal;
      a score is a sum of 128 exact products in f32: 2^-22 of their magnitudes' sum bounds its
      error (128 additions of 2^-24, halved again for the tensor cores' truncation), and a weight
      moves by as much relative to itself; 2^-20 covers the exponentials and the joins."""
    dev = "cuda"
    B, T, Hq = q.shape[:3]
    H = cache_codes[0].shape[1]
    G = Hq // H
    scale = D ** -0.5 if sm_scale is None else sm_scale
    out = torch.zeros((B, T, Hq, D), dtype=torch.float64, device=dev)
    tol = torch.zeros_like(out)
    codes = [torch.from_numpy(c).to(dev) for c in cache_codes]
    exps = [torch.from_numpy(np.asarray(e, np.float64)).to(dev) for e in cache_exps]
    for b in range(B):
        L = int(lens[b])
        if L <= 0:
            continue
        pos = np.arange(L)
        slot = torch.from_numpy(block_table[b, pos // P].astype(np.int64) * P + pos % P).to(dev)
        see = torch.from_numpy(np.stack([visible(b, j, pos) for j in range(T)])).to(dev).repeat_interleave(G, 0)
        for h in range(H):
            ck, cv = (c[slot // 16, h, slot % 16] for c in codes)
            ek, ev = (e[slot // 16, h] for e in exps)
            k, v = ck * torch.exp2(ek)[:, None], cv * torch.exp2(ev)[:, None]
            rows = q[b, :, h * G:(h + 1) * G].to(dev).double().reshape(T * G, D)
            s = rows @ k.T * scale
            mag = (rows.abs() @ k.abs().T * scale).masked_fill(~see, 0).amax(-1, keepdim=True)
            s = s.masked_fill(~see, -math.inf)
            some = see.any(-1, keepdim=True)
            p = torch.where(some, torch.softmax(torch.where(some, s, 0.0), -1), 0.0)
            p = torch.where(see, p, 0.0)
            vv = torch.where(see.any(0)[:, None], v, 0.0)
            o = p @ vv
            spread = p @ vv.abs()
            top = (p * torch.exp2(ev)).amax(-1, keepdim=True)  # the largest weighted scale of the row
            low = 2.0 ** -25 * top * (see.double() @ torch.where(see.any(0)[:, None], cv, 0.0).abs())
            t = (2.0 ** -11 + 2 * mag * 2.0 ** -22 + 2.0 ** -20) * spread + low
            out[b, :, h * G:(h + 1) * G] = o.reshape(T, G, D)
            tol[b, :, h * G:(h + 1) * G] = t.reshape(T, G, D)
    return out.cpu().numpy(), tol.cpu().numpy()


def half_step(dtype, ref):
    """Half a step of the output type at ref: eps / 2 of it, and half the smallest subnormal."""
    return torch.finfo(dtype).eps / 2 * np.abs(ref) + (2.0 ** -25 if dtype == torch.float16 else 0.0)
