"""Shared inputs and bounds of the block-scaled 8-bit cache's GPU tests."""
from __future__ import annotations

import numpy as np
import torch

from oracle import block8 as o

FMTS = ("int8", "fp8")


def cache(N, Hkv, bs, d, fmt, seed, mag=1.0, shift=0.0, spread=0):
    """Random K/V, blocks coded whole by the oracle: k_codes, v_codes, k_scale, v_scale (numpy);
    each block's magnitude times 2^(-spread .. spread)."""
    rng = np.random.default_rng(seed)
    out = []
    for _ in "kv":
        x = (rng.standard_normal((N, Hkv, bs, d)) * mag + shift).astype(np.float32)
        if spread:
            x *= 2.0 ** rng.integers(-spread, spread + 1, (N, Hkv, 1, 1)).astype(np.float32)
        s = (np.abs(x).max((2, 3)) / o.TOP[fmt]).astype(np.float32)
        y = (x / np.where(s > 0, s, np.float32(1))[..., None, None]).astype(np.float32)
        out.append((o.encode(y, fmt), s))
    return [out[0][0], out[1][0], out[0][1], out[1][1]]


def behind(c, lens, tbl, bs, byte=0x7F):
    """Rows behind each context's end hold ``byte`` (E4M3: NaN)."""
    for i, n in enumerate(lens):
        for pos in range(int(n), -(-int(n) // bs) * bs):
            for x in c[:2]:
                x[tbl[i, pos // bs], :, pos % bs] = byte


def decode_bound(q, c, tbl, lens, scale, dtype, ref, fmt):
    """Largest |gpu - ref| per output element.

    * the output is rounded once: eps / 2 of |ref| (2^-25 near fp16's subnormals);
    * P times the block's V scale is two bf16 numbers, off by 2^-16 of itself: at most
      2^-16 of sum_j w_j |v_j|;
    * a logit error of D moves the output by at most 2 D max |v|.  A logit is a sum of d
      products in fp32, in MMA steps of 16 (each rounding 2^-22 of the largest partial sum, at most 16 of
      them) and a handful of fp32 operations; INT8 codes are multiplied from 128 on, so the
      partial sums are those of |c| + 256: D <= 2^-17 scale s sum |q| (|c| + 256);
    * the sums over the keys run in fp32, two products per 16 keys and some 64 steps of
      joining, each rounded by 2^-22 of a partial sum, which is at most max |v| (INT8: of
      |c| + 128); exp2 is good to 2^-22.
    """
    kc, vc, ks, vs = c
    N, Hkv, bs, _ = kc.shape
    B, H, d = q.shape
    G = H // Hkv
    more_k, more_v = (256.0, 128.0) if fmt == "int8" else (0.0, 0.0)
    bound = torch.finfo(dtype).eps / 2 * np.abs(ref) + 2.0 ** -24
    for i in range(B):
        n = int(lens[i])
        if n == 0:
            continue
        k, v = o.context(kc, vc, ks, vs, tbl[i], n, fmt)
        blk = np.clip(np.asarray(tbl[i], np.int64)[np.arange(n) // bs], 0, N - 1)
        sk, sv = ks[blk].astype(np.float64), vs[blk].astype(np.float64)
        for h in range(H):
            g = h // G
            s = (k[:, g] @ q[i, h]) * scale
            w = np.exp(s - s.max())
            w /= w.sum()
            D = 2.0 ** -17 * abs(scale) * ((np.abs(k[:, g]) + more_k * sk[:, g: g + 1]) @ np.abs(q[i, h])).max()
            vmax = (np.abs(v[:, g]).max(-1) + more_v * sv[:, g]).max()
            bound[i, h] += (2.0 ** -16 * (w @ np.abs(v[:, g]))
                            + (2 * D + (n / 8 + 64) * 2.0 ** -22) * vmax)
    return bound
