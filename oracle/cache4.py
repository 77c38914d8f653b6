"""Oracle of the 4-bit KV cache and of block-sparse decode (numpy, fp64).

TEST INFRASTRUCTURE ONLY, like the rest of this package.

4-bit cache (a reading: "LLM推理优化技术地图：从KV Cache到量化与投机解码", section 4.3
quantises the cache and fixes no format).  A row of d values is cut into groups of
64; a group x has m = f16(min x), s = f16(fl32(fl32(max x - min x) / 15)), both
saturating at +-65504, and codes c = rint(fl32(fl32(x - m) / s)) clamped to 0 .. 15
(ties to even, 0 where s = 0).  A code stands for s c + m.  Byte i of a row holds
values 2i (low nibble) and 2i + 1.  Codes [N, Hkv, bs, d / 2], scales
[N, Hkv, bs, d / 64, 2] f16 (s, m).

Block summaries: lo and hi are the smallest and largest key of each channel over
the rows in use, S = fl32(max(|lo|, |hi|) / 127), codes rint(fl32(x / S)) clamped to
+-127 (0 where S = 0).  Scores: the query is coded the same way (sq per head), dot =
sum_c c (c > 0 ? hi : lo), score = max over the group's heads of
fl32(fl32(dot sq) S).
"""
from __future__ import annotations

import numpy as np

GROUP = 64
_F16_MAX = np.float32(65504)


def quantize_rows_int4(x_fp32):
    """Rows (last axis) of fp32 values -> (codes uint8 [..., d / 2], scales f16 [..., d / 64, 2])."""
    x = np.asarray(x_fp32, dtype=np.float32)
    g = x.reshape(x.shape[:-1] + (x.shape[-1] // GROUP, GROUP))
    lo, hi = g.min(-1), g.max(-1)
    m = np.clip(lo, -_F16_MAX, _F16_MAX).astype(np.float16)
    with np.errstate(over="ignore"):
        s = np.minimum(((hi - lo) / np.float32(15)).astype(np.float32), _F16_MAX).astype(np.float16)
        sf, mf = s.astype(np.float32)[..., None], m.astype(np.float32)[..., None]
        y = (g - mf) / np.where(sf > 0, sf, np.float32(1))
    c = np.where(sf > 0, np.clip(np.rint(y.astype(np.float64)), 0, 15), 0).astype(np.uint8)
    c = c.reshape(x.shape)
    return c[..., 0::2] | (c[..., 1::2] << 4), np.stack([s, m], axis=-1)


def int4_values(codes, scale) -> np.ndarray:
    """The fp64 values that packed codes [..., d / 2] and scales [..., d / 64, 2] stand for."""
    codes = np.asarray(codes, dtype=np.uint8)
    c = np.empty(codes.shape[:-1] + (2 * codes.shape[-1],), np.float64)
    c[..., 0::2], c[..., 1::2] = codes & 15, codes >> 4
    sm = np.repeat(np.asarray(scale, np.float64), GROUP, axis=-2)
    return c * sm[..., 0] + sm[..., 1]


def reshape_and_cache_int4(k_new, v_new, slot_mapping, k_codes, v_codes, k_scale, v_scale) -> None:
    """The 4-bit KV append: token t's rows go to slot s (block s // bs, row s % bs)."""
    bs = k_codes.shape[2]
    for new, codes, scale in ((k_new, k_codes, k_scale), (v_new, v_codes, v_scale)):
        c, sm = quantize_rows_int4(new.float().numpy())
        for t in range(new.shape[0]):
            s = int(slot_mapping[t])
            if s >= 0:
                codes[s // bs, :, s % bs] = c[t]
                scale[s // bs, :, s % bs] = sm[t]


def gather_int4(codes, scale, slot_mapping) -> np.ndarray:
    """fp64 values [T, Hkv, d] of the slots (all >= 0)."""
    bs = codes.shape[2]
    s = np.asarray(slot_mapping, np.int64)
    return int4_values(codes[s // bs, :, s % bs], scale[s // bs, :, s % bs])


def softmax_attention(q, k, v, scale: float) -> np.ndarray:
    """q [H, d], k / v [n, Hkv, d] fp64 -> [H, d]; zeros for n = 0."""
    H, d = q.shape
    out = np.zeros((H, d))
    if k.shape[0] == 0:
        return out
    G = H // k.shape[1]
    for h in range(H):
        s = (k[:, h // G] @ q[h]) * scale
        w = np.exp(s - s.max())
        out[h] = (w @ v[:, h // G]) / w.sum()
    return out


def decode_int4(q, k_codes, v_codes, k_scale, v_scale, block_tables, context_lens,
                scale: float) -> np.ndarray:
    """fp64 paged decode over a 4-bit cache; q [B, H, d] fp64.  A table entry outside the pool
    stands for rows of zeros."""
    N, Hkv, bs, _ = k_codes.shape
    B, H, d = q.shape
    out = np.zeros((B, H, d))
    for i in range(B):
        pos = np.arange(int(context_lens[i]))
        blk = np.asarray(block_tables[i], np.int64)[pos // bs]
        ok = (blk >= 0) & (blk < N)
        slots = np.where(ok, blk, 0) * bs + pos % bs
        k, v = (np.where(ok[:, None, None], gather_int4(c, s, slots), 0.0)
                for c, s in ((k_codes, k_scale), (v_codes, v_scale)))
        out[i] = softmax_attention(q[i], k, v, scale)
    return out


def _code8(x, s):
    """INT8 codes of fp32 values x for the step s (0 where s = 0)."""
    s = np.asarray(s, np.float32)
    y = (np.asarray(x, np.float32) / np.where(s > 0, s, np.float32(1))).astype(np.float32)
    return np.where(s > 0, np.clip(np.rint(y.astype(np.float64)), -127, 127), 0).astype(np.int8)


def summarize_blocks(k, block_ids, fills, boxes, box_scale) -> None:
    """k [N, bs, Hkv, d] fp32 -> boxes [N, Hkv, 2, d] int8, box_scale [N, Hkv] fp32, in place."""
    for b, f in zip(block_ids, fills):
        b, f = int(b), int(f)
        rows = np.asarray(k[b, :f], np.float32)
        zero = np.zeros(k.shape[2:], np.float32)
        box = np.stack([rows.min(0), rows.max(0)], 1) if f else np.stack([zero, zero], 1)
        s = (np.abs(box).max((1, 2)) / np.float32(127)).astype(np.float32)
        boxes[b] = _code8(box, s[:, None, None])
        box_scale[b] = s


def block_scores(q, boxes, box_scale, ids) -> np.ndarray:
    """fp32 scores [Hkv, len(ids)] of the blocks ids for one sequence's q [H, d] (fp32)."""
    Hkv = boxes.shape[1]
    q = np.asarray(q, np.float32)
    sq = (np.abs(q).max(-1) / np.float32(127)).astype(np.float32)
    c = _code8(q, sq[:, None]).astype(np.int64)
    G = q.shape[0] // Hkv
    out = np.empty((Hkv, len(ids)), np.float32)
    for g in range(Hkv):
        lo, hi = boxes[ids, g, 0].astype(np.int64), boxes[ids, g, 1].astype(np.int64)
        each = []
        for h in range(g * G, g * G + G):
            dot = np.where(c[h] > 0, hi * c[h], lo * c[h]).sum(-1)
            each.append(((dot.astype(np.float32) * sq[h]).astype(np.float32)
                         * box_scale[ids, g]).astype(np.float32))
        out[g] = np.max(each, axis=0)
    return out


def select_blocks(q, boxes, box_scale, block_tables, context_lens, bs: int, keep: int, first: int,
                  last: int):
    """(sel_blocks [B, Hkv, keep], sel_lens [B, Hkv]) int32; q [B, H, d] fp32."""
    B, Hkv = q.shape[0], boxes.shape[1]
    sel = np.full((B, Hkv, keep), -1, np.int32)
    lens = np.zeros((B, Hkv), np.int32)
    for i in range(B):
        n = int(context_lens[i])
        nb = -(-n // bs)
        if nb == 0:
            continue
        ids = np.asarray(block_tables[i][:nb], np.int64)
        tail = n - (nb - 1) * bs
        score = block_scores(q[i], boxes, box_scale, ids) if nb > keep else None
        for g in range(Hkv):
            if nb <= keep:
                pick = np.arange(nb)
            else:
                mid = np.arange(first, nb - last)
                order = mid[np.argsort(-score[g, mid].astype(np.float64), kind="stable")]
                pick = np.sort(np.concatenate([np.arange(first), order[: keep - first - last],
                                               np.arange(nb - last, nb)]))
            sel[i, g, : len(pick)] = ids[pick]
            lens[i, g] = (len(pick) - 1) * bs + tail
    return sel, lens


def decode_selected(q, k, v, sel_blocks, sel_lens, scale: float) -> np.ndarray:
    """fp64 attention of q [B, H, d] over the first sel_lens[i][g] tokens of the blocks
    sel_blocks[i][g]; k / v [N, bs, Hkv, d] fp64."""
    B, H, d = q.shape
    _, bs, Hkv, _ = k.shape
    G = H // Hkv
    out = np.zeros((B, H, d))
    for i in range(B):
        for g in range(Hkv):
            t = np.arange(int(sel_lens[i, g]))
            blk = np.asarray(sel_blocks[i, g], np.int64)[t // bs]
            out[i, g * G: g * G + G] = softmax_attention(
                q[i, g * G: g * G + G], k[blk, t % bs, g][:, None], v[blk, t % bs, g][:, None], scale)
    return out
