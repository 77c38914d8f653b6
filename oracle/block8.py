"""Oracle of the block-scaled 8-bit KV cache (numpy, fp64).

TEST INFRASTRUCTURE ONLY, like the rest of this package.

A code is an INT8 integer (TOP 127) or an E4M3 number (TOP 448) and stands for code * scale,
one fp32 scale per (block, KV head).  Codes [N, Hkv, bs, d] uint8, scales [N, Hkv] fp32.
An append to a block, with a the largest magnitude of the rows R that it writes there:
base = 0 if row 0 is in R, else the scale; s = max(base, fl32(a / TOP)); rows in R become
code(fl32(x / s)) (0 where s = 0), the others, if 0 < base < s, code(fl32(c fl32(base / s))).
"""
from __future__ import annotations

import numpy as np

from .cache4 import softmax_attention

TOP = {"int8": np.float32(127), "fp8": np.float32(448)}


def _e4m3_table() -> np.ndarray:
    """fp64 numbers of the 256 E4M3 bytes: sign, 4 exponent bits (bias 7), 3 mantissa bits;
    exponent 0 is subnormal, 0x7F and 0xFF are NaN."""
    out = np.empty(256)
    for b in range(256):
        e, m = b >> 3 & 15, b & 7
        v = np.nan if b & 127 == 127 else m * 2.0 ** -9 if e == 0 else (8 + m) * 2.0 ** (e - 10)
        out[b] = -v if b & 128 else v
    return out


E4M3 = _e4m3_table()


def numbers(codes, fmt: str) -> np.ndarray:
    codes = np.asarray(codes, np.uint8)
    return codes.view(np.int8).astype(np.float64) if fmt == "int8" else E4M3[codes]


def encode(x, fmt: str) -> np.ndarray:
    """Nearest codes of finite numbers, ties to the even code, saturating."""
    x = np.asarray(x, np.float64)
    if fmt == "int8":
        return np.clip(np.rint(x), -127, 127).astype(np.int8).view(np.uint8)
    mag = E4M3[:127]                                  # ascending
    a = np.abs(x)
    hi = np.clip(np.searchsorted(mag, a), 1, 126)     # mag[hi - 1] < a <= mag[hi], or the ends
    down, up = a - mag[hi - 1], mag[hi] - a
    low = (down < up) | ((down == up) & (hi % 2 == 1))
    code = np.where(low, hi - 1, hi).astype(np.uint8)
    return code | (np.signbit(x).astype(np.uint8) << 7)


def append(new, slots, codes, scale, fmt: str) -> None:
    """One tensor's append, in place: new [T, Hkv, d] fp32, slots [T]; the tokens of a block
    are taken together wherever they stand in the call."""
    new = np.asarray(new, np.float32)
    N, _, bs, _ = codes.shape
    of = {}
    for t, s in enumerate(np.asarray(slots, np.int64)):
        if 0 <= s < N * bs:
            of.setdefault(int(s) // bs, []).append((t, int(s) % bs))
    for b, rows in of.items():
        t, r = (np.array(v) for v in zip(*rows))
        base = np.zeros_like(scale[b]) if (r == 0).any() else scale[b].copy()
        s = np.maximum(base, (np.abs(new[t]).max((0, 2)) / TOP[fmt]).astype(np.float32))
        div = np.where(s > 0, s, np.float32(1))
        grows = (base > 0) & (base < s)
        ratio = (base / div).astype(np.float32)[:, None, None]
        with np.errstate(invalid="ignore"):           # E4M3 NaN bytes of rows that nothing wrote
            c = (numbers(codes[b], fmt).astype(np.float32) * ratio).astype(np.float32)
        again = np.where(np.isnan(c), codes[b], encode(np.nan_to_num(c), fmt))
        codes[b] = np.where(grows[:, None, None], again, codes[b])
        y = (new[t] / div[:, None]).astype(np.float32)
        codes[b][:, r] = np.where(s[:, None] > 0, encode(y, fmt), 0).astype(np.uint8).transpose(1, 0, 2)
        scale[b] = s


def values(codes, scale, fmt: str) -> np.ndarray:
    return numbers(codes, fmt) * np.asarray(scale, np.float64)[..., None, None]


def gather(codes, scale, slots, fmt: str) -> np.ndarray:
    """fp64 values [T, Hkv, d] of the slots (all >= 0)."""
    bs = codes.shape[2]
    s = np.asarray(slots, np.int64)
    return numbers(codes[s // bs, :, s % bs], fmt) * scale[s // bs].astype(np.float64)[..., None]


def context(k_codes, v_codes, k_scale, v_scale, table, n: int, fmt: str):
    """fp64 K and V [n, Hkv, d] of one sequence; an entry outside the pool stands for zeros."""
    N, _, bs, _ = k_codes.shape
    pos = np.arange(int(n))
    blk = np.asarray(table, np.int64)[pos // bs]
    ok = (blk >= 0) & (blk < N)
    slots = np.where(ok, blk, 0) * bs + pos % bs
    return [np.where(ok[:, None, None], gather(c, s, slots, fmt), 0.0)
            for c, s in ((k_codes, k_scale), (v_codes, v_scale))]


def decode(q, k_codes, v_codes, k_scale, v_scale, block_tables, context_lens, scale: float,
           fmt: str) -> np.ndarray:
    """fp64 paged decode; q [B, H, d] fp64."""
    out = np.zeros(q.shape)
    for i in range(q.shape[0]):
        k, v = context(k_codes, v_codes, k_scale, v_scale, block_tables[i], context_lens[i], fmt)
        out[i] = softmax_attention(q[i], k, v, scale)
    return out
