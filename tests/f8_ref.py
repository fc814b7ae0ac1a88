"""64-bit definitions of the block-scaled E4M3 operators, written from their
formulas (numpy / torch double, no code of the product package), and the
error bounds that their tests hold the kernels to."""
import math

import numpy as np
import torch


def e4m3_table():
    """Value of every code byte: sign, 4 exponent bits (bias 7), 3 fraction bits; 0x7F / 0xFF are NaN."""
    v = np.empty(256)
    for b in range(256):
        ex, f = (b >> 3) & 15, b & 7
        m = f * 2.0 ** -9 if ex == 0 else (1 + f / 8) * 2.0 ** (ex - 7)
        v[b] = (-m if b & 128 else m) if b & 127 != 127 else math.nan
    return v


TABLE = e4m3_table()


def _round_code(y):
    """Code byte of a finite |y| <= 448: the nearest magnitude, ties to the even fraction."""
    mags = TABLE[:127]                       # 0 .. 448, ascending
    a = np.abs(y)
    hi = np.clip(np.searchsorted(mags, a), 1, 126)
    lo = hi - 1
    dl, dh = a - mags[lo], mags[hi] - a
    pick = np.where(dl < dh, lo, np.where(dh < dl, hi, np.where(lo % 2 == 0, lo, hi)))
    return (pick | np.where(np.signbit(y), 128, 0)).astype(np.uint8)


def scale_byte(amax):
    """The smallest byte b >= 0 with amax <= 448 * 2^(b - 127)."""
    if amax == 0:
        return 0
    b = 0
    while amax > math.ldexp(448.0, b - 127):
        b += 1
    return b


def quantize(x, block):
    """x [n, w] float64 -> codes uint8, scale bytes uint8 [n, blocks]."""
    n, w = x.shape
    block = block or w
    nb = -(-w // block)
    codes, scales = np.zeros((n, w), np.uint8), np.zeros((n, nb), np.uint8)
    for r in range(n):
        for b in range(nb):
            part = x[r, b * block:(b + 1) * block]
            fin = np.isfinite(part)
            s = scale_byte(np.abs(part[fin]).max() if fin.any() else 0.0)
            c = np.full(part.shape, 0x7F, np.uint8)
            c[fin] = _round_code(np.ldexp(part[fin], 127 - s))
            codes[r, b * block:(b + 1) * block], scales[r, b] = c, s
    return codes, scales


def quantize_squares(x):
    """x [N, K] -> codes, scale bytes of 128 x 128 squares."""
    N, K = x.shape
    codes = np.zeros((N, K), np.uint8)
    scales = np.zeros((-(-N // 128), -(-K // 128)), np.uint8)
    for i in range(scales.shape[0]):
        for j in range(scales.shape[1]):
            part = x[128 * i:128 * i + 128, 128 * j:128 * j + 128]
            s = scale_byte(np.abs(part).max())
            codes[128 * i:128 * i + 128, 128 * j:128 * j + 128] = _round_code(np.ldexp(part, 127 - s))
            scales[i, j] = s
    return codes, scales


def decode(codes, scales, block):
    """Codes [n, w] (uint8 tensor) under scale bytes [n, blocks] as a float64 tensor."""
    table = torch.as_tensor(TABLE, device=codes.device)
    col = torch.arange(codes.shape[1], device=codes.device) // (block or codes.shape[1])
    return table[codes.long()] * torch.exp2(scales.double() - 127)[:, col]


def decode_squares(codes, scales):
    table = torch.as_tensor(TABLE, device=codes.device)
    i = torch.arange(codes.shape[0], device=codes.device) // 128
    j = torch.arange(codes.shape[1], device=codes.device) // 128
    return table[codes.long()] * torch.exp2(scales.double() - 127)[i][:, j]


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


def gemm(a, b, dtype):
    """A . B^T in 64 bits and the bound on a kernel that accumulates in fp32 (any order, truncating adders: one
    step 2^-23 of the running magnitudes per addition) and rounds once to dtype.  Where the magnitudes add up to
    2^127 or more, a running sum may leave the range of fp32 (2^128) although the result does not: no bound there."""
    d = a @ b.t()
    mag = a.abs() @ b.abs().t()
    bound = (a.shape[1] + 2) * 2.0 ** -23 * mag + half_step(dtype) * d.abs() + 1e-37
    return d, torch.where(mag < 2.0 ** 127, bound, math.inf)


def mqa(q, codes, scales, sel, dtype):
    """One query row: q [nh, c] float64, entries codes [*, c] / scales [*], sel = the valid entry rows.
    -> output [nh, c] and its bound for a kernel with
      q: hi + lo, both E4M3, of the row scaled to a maximum in [128, 256): 8 significant bits are kept unless lo is
        subnormal (half of its step: 2^-10, that is 2^-17 of the row's maximum);
      scores: sums in fp32, one step 2^-23 per addition;
      weight times scale w = hi + lo, hi E4M3, lo E5M2, of a value rounded to fp16 (2^-11): hi is within 2^-4 of w
        (2^-10 where it is subnormal), lo within 2^-3 of the rest, so w is within 2^-7 + 2^-11 relative and 2^-13, or
        2^-17 where lo is subnormal: at most 2^-13 in all, of a largest weight of 2^3.5 or more: 2^-16.5 of it;
      and one rounding to dtype."""
    nh, c = q.shape
    if sel.numel() == 0:
        z = torch.zeros(nh, c, dtype=torch.float64, device=q.device)
        return z, z
    table = torch.as_tensor(TABLE, device=q.device)
    raw = table[codes[sel].long()]
    sc = torch.exp2(scales[sel].double() - 127)
    e = raw * sc[:, None]
    s = q @ e.t() / math.sqrt(c)
    p = torch.softmax(s, 1)
    o = p @ e
    ds = ((c + 4) * 2.0 ** -23 * (q.abs() @ e.abs().t())
          + 2.0 ** -17 * q.abs().amax(1, keepdim=True) * e.abs().sum(1)[None]) / math.sqrt(c) + 2.0 ** -20 * (1 + s.abs())
    dp = p * torch.expm1(2 * ds)                     # numerator and normaliser both move by exp(ds)
    floor = 2.0 ** -16 * (p * sc).amax(1, keepdim=True)
    bound = ((2.0 ** -7 + 2.0 ** -10) * p + dp) @ e.abs() + dp.sum(1, keepdim=True) * o.abs() + floor * raw.abs().sum(0)[None]
    return o, bound + half_step(dtype) * (o.abs() + bound) + 1e-37
