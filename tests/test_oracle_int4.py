"""Pins of the 4-bit and block-sparse oracle (no GPU): closed forms, format bounds, torch."""
import numpy as np
import pytest
import torch

from oracle import cache4 as o


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
def test_rows_come_back_within_half_a_step(d, dtype):
    g = torch.Generator().manual_seed(d)
    x = (torch.randn(200, d, generator=g) * torch.logspace(-3, 3, 200)[:, None]
         + torch.randn(200, 1, generator=g)).to(dtype).float().numpy()
    codes, sm = o.quantize_rows_int4(x)
    back = o.int4_values(codes, sm)
    s = np.repeat(sm[..., 0].astype(np.float64), 64, axis=-1)
    m = np.repeat(np.abs(sm[..., 1].astype(np.float64)), 64, axis=-1)
    # half a step; the ends clip by what m (2^-11 |m|) and 15 s (15 s 2^-11) were rounded by, and
    # by half the smallest f16 (2^-25) where they are subnormal
    assert (np.abs(back - x) <= s / 2 * (1 + 2.0 ** -22) + (m + 15 * s) * 2.0 ** -11 + 16 * 2.0 ** -25).all()


def test_codes_of_hand_made_rows():
    x = np.zeros((5, 64), np.float32)
    x[0] = np.arange(64) % 16                     # the codes themselves: m = 0, s = 1
    x[1] = 3.0                                    # constant: s = 0, codes 0, value m
    x[2, :4] = [0.5, 1.5, 2.5, 15.0]              # ties go to even: 0, 2, 2
    x[3, 0], x[3, 1] = -1e5, 1e5                  # beyond f16: m saturates, s is f16(2e5 / 15)
    x[4, 0] = 15 * 2.0 ** -26                     # s = f16(2^-26) = 0 (half the smallest, to even)
    codes, sm = o.quantize_rows_int4(x)
    c = np.stack([codes & 15, codes >> 4], -1).reshape(5, 64)
    assert (c[0] == np.arange(64) % 16).all() and (sm[0, 0] == [1, 0]).all()
    assert (c[1] == 0).all() and (sm[1, 0] == [0, 3]).all() and (o.int4_values(codes, sm)[1] == 3).all()
    assert c[2, :4].tolist() == [0, 2, 2, 15]
    assert sm[3, 0, 1] == -65504 and sm[3, 0, 0] == np.float16(2e5 / 15) and c[3, 1] == 12
    assert (c[4] == 0).all() and (sm[4] == 0).all()


def test_groups_are_independent_and_nibbles_in_order():
    x = np.zeros((1, 128), np.float32)
    x[0, :64] = np.arange(64) % 16
    x[0, 64:] = 100 + 2 * (np.arange(64) % 16)[::-1]
    codes, sm = o.quantize_rows_int4(x)
    assert codes[0, 0] == 0x10 and codes[0, 1] == 0x32 and codes[0, 32] == 0xEF
    assert sm[0].tolist() == [[1, 0], [2, 100]]
    assert (o.int4_values(codes, sm) == x).all()


@pytest.mark.parametrize("bs,Hkv,G,d", [(16, 2, 3, 64), (8, 1, 1, 128)])
def test_int4_decode_equals_sdpa_on_the_values(bs, Hkv, G, d):
    rng = np.random.default_rng(bs)
    lens, N = [0, 1, 37], 12
    tbl = rng.permutation(N)[: 3 * 3].reshape(3, 3) if bs == 16 else rng.permutation(15)[:15].reshape(3, 5)
    N = int(tbl.max()) + 1
    ks, vs = (o.quantize_rows_int4(rng.standard_normal((N, Hkv, bs, d)).astype(np.float32)) for _ in "kv")
    q = rng.standard_normal((3, Hkv * G, d))
    got = o.decode_int4(q, ks[0], vs[0], ks[1], vs[1], tbl, lens, d ** -0.5)
    assert (got[0] == 0).all()
    for i in (1, 2):
        slots = tbl[i][np.arange(lens[i]) // bs] * bs + np.arange(lens[i]) % bs
        k, v = (torch.from_numpy(o.gather_int4(c, s, slots)).permute(1, 0, 2).repeat_interleave(G, 0)
                for c, s in (ks, vs))
        ref = torch.nn.functional.scaled_dot_product_attention(torch.from_numpy(q[i])[:, None], k, v)
        assert np.abs(ref[:, 0].numpy() - got[i]).max() < 1e-12


def test_boxes_bound_every_score():
    """The box's bound is at least the score of every key in the block, up to the half steps of
    the codes: per channel (|q| S + sq |box| + sq S / 2) / 2 at most."""
    rng = np.random.default_rng(3)
    k = rng.standard_normal((6, 8, 2, 64)).astype(np.float32)
    boxes, S = np.zeros((6, 2, 2, 64), np.int8), np.zeros((6, 2), np.float32)
    o.summarize_blocks(k, range(6), [8, 8, 8, 8, 8, 5], boxes, S)
    assert (np.abs(boxes.astype(int)).max((2, 3)) == 127).all()
    assert (boxes[:, :, 0] <= boxes[:, :, 1]).all()
    q = rng.standard_normal((4, 64)).astype(np.float32)
    sc = o.block_scores(q, boxes, S, np.arange(6))
    sq = np.abs(q).max(-1) / 127
    for b in range(6):
        for g in range(2):
            rows = k[b, : (5 if b == 5 else 8), g]
            best = (q[2 * g: 2 * g + 2] @ rows.T).max()
            slack = max(((np.abs(q[h]) + sq[h] / 2) * S[b, g] / 2 + sq[h] / 2 * 127 * S[b, g]).sum()
                        for h in (2 * g, 2 * g + 1))
            assert sc[g, b] >= best - slack


def test_selection_of_hand_made_scores():
    """One channel carries the score: block b's box is [0, b'], the query is 1 there."""
    N, d, bs = 10, 64, 8
    boxes, S = np.zeros((N, 1, 2, d), np.int8), np.ones((N, 1), np.float32)
    worth = [3, 9, 9, 1, 7, 9, 0, 2, 8, 0]
    boxes[:, 0, 1, 5] = worth
    q = np.zeros((3, 1, d), np.float32)
    q[:, 0, 5] = 1
    tbl = np.tile(np.arange(N), (3, 1))
    sel, n = o.select_blocks(q, boxes, S, tbl, [79, 0, 32], bs, 5, 1, 1)
    assert sel[0, 0].tolist() == [0, 1, 2, 5, 9] and n[0, 0] == 4 * 8 + 7   # three nines, in order
    assert sel[1, 0].tolist() == [-1] * 5 and n[1, 0] == 0
    assert sel[2, 0].tolist() == [0, 1, 2, 3, -1] and n[2, 0] == 32
    sel, _ = o.select_blocks(q, boxes, S, tbl, [80, 0, 0], bs, 4, 1, 1)
    assert sel[0, 0].tolist() == [0, 1, 2, 9]                                # ties: the lower position


def test_selecting_everything_is_the_dense_decode():
    rng = np.random.default_rng(8)
    N, bs, Hkv, d = 9, 8, 2, 64
    k, v = rng.standard_normal((2, N, bs, Hkv, d))
    q = rng.standard_normal((2, 4, d))
    tbl, lens = rng.permutation(8).reshape(2, 4), [30, 9]
    boxes, S = np.zeros((N, Hkv, 2, d), np.int8), np.zeros((N, Hkv), np.float32)
    sel, n = o.select_blocks(q.astype(np.float32), boxes, S, tbl, lens, bs, 4, 0, 1)
    got = o.decode_selected(q, k, v, sel, n, 0.2)
    for i in range(2):
        t = np.arange(lens[i])
        ref = o.softmax_attention(q[i], k[tbl[i][t // bs], t % bs], v[tbl[i][t // bs], t % bs], 0.2)
        assert np.abs(ref - got[i]).max() < 1e-13
