"""Shared inputs and bounds of the 4-bit-cache and block-sparse GPU tests."""
from __future__ import annotations

import math

import numpy as np
import torch

from oracle import cache4 as o
from paged_kv_cache_103_gb300 import binding

NAN16 = float("nan")


def rand_tables(lens, bs, seed, slack=3):
    """(tables int32 [B, W] with -1 in unused entries, N): blocks scattered over a pool."""
    rng = np.random.default_rng(seed)
    nb = [-(-int(n) // bs) for n in lens]
    N = sum(nb) + slack
    order = rng.permutation(N)
    tbl = np.full((len(nb), max(max(nb, default=0), 1)), -1, np.int32)
    at = 0
    for i, k in enumerate(nb):
        tbl[i, :k] = order[at: at + k]
        at += k
    return tbl, N


def int4_cache(N, Hkv, bs, d, seed, mag=1.0, shift=0.0):
    """Random K/V quantised by the oracle: k_codes, v_codes, k_scale, v_scale (numpy)."""
    rng = np.random.default_rng(seed)
    out = [o.quantize_rows_int4((rng.standard_normal((N, Hkv, bs, d)) * mag + shift).astype(np.float32))
           for _ in "kv"]
    return [out[0][0], out[1][0], out[0][1], out[1][1]]


def behind(lens, tbl, bs):
    """(block, row) of every slot of a used block behind its sequence's last token."""
    for i, n in enumerate(lens):
        for pos in range(int(n), -(-int(n) // bs) * bs):
            yield tbl[i, pos // bs], pos % bs


def nan_behind(cache, lens, tbl, bs):
    for b, r in behind(lens, tbl, bs):
        for codes, scale in ((cache[0], cache[2]), (cache[1], cache[3])):
            codes[b, :, r] = 0xA5
            scale[b, :, r] = NAN16


def dev(*arrays):
    return [torch.from_numpy(np.ascontiguousarray(a)).cuda() for a in arrays]


def workspace(B, H, d):
    ws = torch.empty(max(binding.pa_decode_workspace_size(B, H, d), 1), dtype=torch.uint8, device="cuda")
    binding.pa_decode_workspace_init(ws)
    return ws


def decode_bound(q, cache, tbl, lens, scale, dtype, ref):
    """Largest |gpu - ref| per output element.

    * the output is rounded once: eps / 2 of |ref|;
    * P (a probability times the step s) is rounded to f16 once, 2^-11 of it, and multiplies
      c - 8 (the value of code 8 stays fp32): at most 2^-11 of sum_j w_j s |c - 8|;
    * a logit error of D moves the output by at most 2 D max |v|.  A logit is a sum of at most
      2 d products in fp32, in MMA steps of 16 (each step's rounding 2^-22 of the largest partial
      sum, at most 16 of them) and a handful of fp32 operations: D <= 2^-17 scale sum |q| (s c + |m|);
    * exp2 is good to 2^-22 and sums over the keys to 2^-20: below 2^-19 of max |v|.
    """
    codes_k, codes_v, ks, vs = cache
    N, Hkv, bs, _ = codes_k.shape
    B, H, d = q.shape
    G = H // Hkv
    eps = torch.finfo(dtype).eps / 2
    bound = eps * np.abs(ref) + 2.0 ** -24
    for i in range(B):
        n = int(lens[i])
        if n == 0:
            continue
        t = np.arange(n)
        blk = tbl[i][t // bs].astype(np.int64)
        ok = (blk >= 0) & (blk < N)
        at = np.where(ok, blk, 0) * bs + t % bs
        k = np.where(ok[:, None, None], o.gather_int4(codes_k, ks, at), 0)
        v = np.where(ok[:, None, None], o.gather_int4(codes_v, vs, at), 0)
        mk = np.repeat(np.abs(ks[at // bs, :, at % bs, :, 1].astype(np.float64)), 64, -1)
        mv = np.repeat(vs[at // bs, :, at % bs, :, 1].astype(np.float64), 64, -1)
        sv = np.repeat(vs[at // bs, :, at % bs, :, 0].astype(np.float64), 64, -1)
        off_v = np.where(ok[:, None, None], np.abs(v - mv - 8 * sv), 0)     # s |c - 8|
        mag_k = np.where(ok[:, None, None], np.abs(k) + 2 * mk, 0)
        for h in range(H):
            g = h // G
            s = (k[:, g] @ q[i, h]) * scale
            w = np.exp(s - s.max())
            w /= w.sum()
            D = 2.0 ** -17 * abs(scale) * (mag_k[:, g] @ np.abs(q[i, h])).max()
            vmax = np.abs(v[:, g]).max()
            bound[i, h] += 2.0 ** -11 * (w @ off_v[:, g]) + (2 * D + 2.0 ** -19) * vmax
    return bound


def max_blocks_of(lens, bs):
    return max(1, max((math.ceil(int(n) / bs) for n in lens), default=1))
