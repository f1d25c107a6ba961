"""The 4-bit cache's format in numpy, 64 bits, from its definition; test infrastructure only.

Rows are bf16 bit patterns (uint16) [..., d] in groups of 32 values.
"""
from __future__ import annotations

import numpy as np

import nosa_synth as syn

NAN_SCALE = 0x7FFF


def values(bits):
    """bf16 bit patterns as float64."""
    with np.errstate(invalid="ignore"):  # signalling NaN patterns
        return (bits.astype(np.uint32) << 16).view(np.float32).astype(np.float64)


def quantise(bits):
    """(codes uint8 [..., d/32, 32], scales as bf16 bits [..., d/32]) of rows [..., d]."""
    x = values(bits).reshape(*bits.shape[:-1], -1, 32)
    finite = np.isfinite(x).all(-1)
    a = np.where(finite[..., None], np.abs(x), 0).max(-1)
    s = syn.round_bf16(np.ascontiguousarray(a / 7)).reshape(a.shape)
    s = np.where(values(s) < 2.0**-126, 0, s).astype(np.uint16)
    sv = np.where(s == 0, 1.0, values(s))[..., None]
    xf = np.where(finite[..., None], x, 0)
    c = np.sign(xf) * np.floor(np.abs(xf) / sv + 0.5)
    c = np.where((s == 0)[..., None], 0, c)
    assert np.abs(c).max(initial=0) <= 7
    return (c + 8).astype(np.uint8), np.where(finite, s, NAN_SCALE).astype(np.uint16)


def dequantise(codes, scales):
    """float64 values [..., d]."""
    y = (codes.astype(np.float64) - 8) * values(scales)[..., None]
    return y.reshape(*codes.shape[:-2], -1)


def round_to_bf16(y):
    """bf16 bits of float64 values, nearest even, NaN kept (for values of at most 12 significant
    bits, exact in float32)."""
    f = y.astype(np.float32).view(np.uint32).astype(np.uint64)
    r = ((f + 0x7FFF + ((f >> 16) & 1)) >> 16).astype(np.uint16)
    return np.where(np.isnan(y), np.uint16(0x7FC0), r)


def pack(codes, scales, keys):
    """Pages [..., bytes] (uint8) of blocks codes [..., bs, d/32, 32], scales [..., bs, d/32]."""
    *lead, bs, ng, _ = codes.shape
    d, n = 32 * ng, 8 if keys else 4
    page = np.zeros((*lead, bs * d * 9 // 16), np.uint8)
    row = np.arange(bs)
    for g in range(ng):
        for x in range(32):
            c, i = divmod(x, n)
            at = row * (d // 2) + c * (d * n // 64) + g * n // 2 + i // 2
            page[..., at] |= codes[..., g, x] << (4 * (i % 2))
        s = scales[..., g]
        page[..., bs * d // 2 + row * (d // 16) + 2 * g] = s & 0xFF
        page[..., bs * d // 2 + row * (d // 16) + 2 * g + 1] = s >> 8
    return page


def unpack(page, bs, d, keys):
    """(codes, scales) of pages [..., bytes]."""
    n, row = 8 if keys else 4, np.arange(bs)
    codes = np.zeros((*page.shape[:-1], bs, d // 32, 32), np.uint8)
    scales = np.zeros((*page.shape[:-1], bs, d // 32), np.uint16)
    for g in range(d // 32):
        for x in range(32):
            c, i = divmod(x, n)
            b = page[..., row * (d // 2) + c * (d * n // 64) + g * n // 2 + i // 2]
            codes[..., g, x] = (b >> (4 * (i % 2))) & 15
        at = bs * d // 2 + row * (d // 16) + 2 * g
        scales[..., g] = page[..., at].astype(np.uint16) | (page[..., at + 1].astype(np.uint16) << 8)
    return codes, scales


def snap(bits):
    """Rows moved to values that the format holds exactly: multiples c * 2^e, |c| <= 7, with a 7 in
    every group that is not zero (so that the scale is 2^e and the codes are c)."""
    x = values(bits).reshape(*bits.shape[:-1], -1, 32)
    a = np.abs(x).max(-1, keepdims=True)
    e = np.exp2(np.ceil(np.log2(np.where(a == 0, 7, a) / 7)))
    c = np.clip(np.round(x / e), -7, 7)
    top = np.abs(x) == a
    c = np.where(top, np.where(x < 0, -7, 7), c) * e
    c = np.where(a == 0, 0, c)
    return syn.round_bf16(np.ascontiguousarray(c.reshape(bits.shape))).reshape(bits.shape).astype(np.uint16)


def attend(q, K, V, scale):
    """float64 attention of q [G, d] over rows K, V [n, d]; zeros where there is no row."""
    if not len(K):
        return np.zeros((len(q), K.shape[1]))
    x = q @ K.T * scale
    p = np.exp(x - x.max(-1, keepdims=True))
    return p @ V / p.sum(-1, keepdims=True)


def attend_bound(q, K, V, scale):
    """What an fp32 computation of attend() may be off by, per query row.

    Score: each of the d products' partial sums and the scale product carry at most 2^-23 of
    sum |q||k| (truncating accumulation), so the exponent is off by ex = (d + 4) 2^-23 scale
    max_t sum|q||k|. exp2 adds 2^-21 and splitting the weight in two 11-bit parts 2^-22, so each weight is off by
    w = ex + 2^-20 relative (first order, doubled below for the second). Numerator and denominator sum n terms: n 2^-23 more
    each. The output is a weighted mean of V: |error| <= 2 * 2 (w + n 2^-23) max|V|.
    """
    n, d = K.shape
    if not n:
        return np.zeros(len(q))
    ex = (d + 4) * 2.0**-23 * scale * (np.abs(q) @ np.abs(K).T).max(-1)
    return 4 * (ex + 2.0**-20 + n * 2.0**-23) * np.abs(V).max()
