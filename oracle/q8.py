"""Plain float64 definition of the 8-bit KV pool: quantising a row, and the
values a row stands for.  A pool is codes [num_blocks, Hkv, B, 128] and scale
bytes [num_blocks, Hkv, B]; a row's values are code * 2^(byte - 127), NaN for
byte 255.  fmt is "e4m3" or "int8"; codes are kept as uint8 bit patterns."""
from __future__ import annotations

import numpy as np

LIMIT = {"e4m3": 448.0, "int8": 127.0}


def e4m3_values() -> np.ndarray:
    """The 256 values of OCP FP8 E4M3 (bias 7, no infinities, 0x7f/0xff NaN)."""
    out = np.empty(256)
    for b in range(256):
        s, e, m = b >> 7, (b >> 3) & 15, b & 7
        v = m / 8.0 * 2.0 ** -6 if e == 0 else (1 + m / 8.0) * 2.0 ** (e - 7)
        out[b] = np.nan if (b & 0x7F) == 0x7F else (-v if s else v)
    return out


_E4M3 = e4m3_values()


def code_values(codes: np.ndarray, fmt: str) -> np.ndarray:
    return _E4M3[codes] if fmt == "e4m3" else codes.view(np.int8).astype(np.float64)


def quantise(x: np.ndarray, fmt: str):
    """Codes and scale bytes of rows x [..., 128] (float64 values of bf16).  A
    code is the nearest whose value is below 2^128, the first number that bf16
    does not hold."""
    x = np.asarray(x, np.float64)
    finite = np.all(np.isfinite(x), axis=-1)
    y = np.where(finite[..., None], x, 0.0)
    a = np.abs(y).max(-1)
    e = np.full(a.shape, -126.0)
    for k in range(-126, 128):  # the smallest power of two that fits (at least 2^-126)
        e = np.where((a > LIMIT[fmt] * 2.0 ** (k - 1)) & (k > e), float(k), e)
    y = y * np.exp2(-e)[..., None]
    held = _E4M3[:127] if fmt == "e4m3" else np.arange(128.0)
    for k in np.unique(e):
        top = held[held * 2.0 ** k < 2.0 ** 128].max()
        y[e == k] = np.clip(y[e == k], -top, top)
    if fmt == "int8":
        codes = np.rint(y).astype(np.int8).view(np.uint8)
    else:
        # Nearest of the non-negative values; between two neighbours the even
        # code (neighbours are consecutive codes).
        grid = _E4M3[:127]
        mag = np.abs(y)
        hi = np.minimum(np.searchsorted(grid, mag, side="left"), 126)
        lo = np.maximum(hi - 1, 0)
        dl, dh = mag - grid[lo], grid[hi] - mag
        pick = np.where(dl < dh, lo, np.where(dh < dl, hi, np.where(lo % 2 == 0, lo, hi)))
        codes = (pick + np.where(np.signbit(y), 128, 0)).astype(np.uint8)
        codes = np.where(finite[..., None], codes, 0).astype(np.uint8)
    return codes, np.where(finite, e + 127, 255).astype(np.uint8)


def values(codes: np.ndarray, scales: np.ndarray, fmt: str) -> np.ndarray:
    s = scales.astype(np.float64)
    s = np.where(s == 255, np.nan, np.exp2(s - 127))
    return code_values(codes, fmt) * s[..., None]


def store(x, codes, scales, slots, fmt):
    """Quantise rows x [N, Hkv, 128] into the pool (in place); negative slots skipped."""
    B = codes.shape[2]
    c, s = quantise(x, fmt)
    for i, slot in enumerate(slots):
        if slot >= 0:
            codes[slot // B, :, slot % B] = c[i]
            scales[slot // B, :, slot % B] = s[i]


def decode(q, kc, ks, vc, vs, fmt, block_tables, context_lens, scale):
    """float64 decode attention over the pool; beside it, per output, the error
    that the kernel's arithmetic may have (NaN where the output is).

    The result's bf16 rounding: 2^-8 of it.  The softmax weights, each times its
    value row's scale, are rounded to fp16: 2^-11 of each, so 2^-11 sum_p p|v|;
    below fp16's normal range the rounding is absolute, at most 2^-25 with the
    largest weight at 2^7 or more, so 2^-32 max_p(p * scale_p) * sum_p |code_p|.
    The scores are fp32 (|x| < 64 in base 2, sums of 128 products), and so are
    the exponentials and the weights' sum: each under 2^-14 of a weight, so
    3 * 2^-14 sum_p p|v|.
    Outputs below bf16's normal range are rounded to multiples of 2^-133 (from
    fp32 numbers that are multiples of 2^-149): under 2^-133."""
    batch, hq, d = q.shape
    hkv, B = kc.shape[1:3]
    G = hq // hkv
    out, tol = np.zeros((batch, hq, d)), np.zeros((batch, hq, d))
    for b in range(batch):
        n = int(context_lens[b])
        if n == 0:
            continue
        pos = np.arange(n)
        blk, off = np.asarray(block_tables[b])[pos // B], pos % B
        for g in range(hkv):
            k = values(kc[blk, g, off], ks[blk, g, off], fmt)
            v = values(vc[blk, g, off], vs[blk, g, off], fmt)
            x = q[b, g * G:(g + 1) * G] @ k.T * scale
            p = np.exp(x - x.max(-1, keepdims=True))
            p /= p.sum(-1, keepdims=True)
            h = slice(g * G, (g + 1) * G)
            out[b, h] = p @ v
            sv = np.exp2(vs[blk, g, off].astype(np.float64) - 127)
            codes = np.abs(code_values(vc[blk, g, off], fmt)).sum(0)
            tol[b, h] = (2.0 ** -8 * np.abs(out[b, h]) + (2.0 ** -11 + 3 * 2.0 ** -14) * (p @ np.abs(v))
                         + 2.0 ** -32 * (p * sv).max(-1, keepdims=True) * codes + 2.0 ** -133)
    return out, tol
