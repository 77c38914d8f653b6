"""The block-scaled 8-bit oracle and the eviction oracle: pins without a GPU."""
import numpy as np
import pytest
import torch

from oracle import block8 as o
from oracle import evict as ev


def test_e4m3_codes_equal_torch():
    b = torch.arange(256, dtype=torch.uint8)
    want = b.view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(o.numbers(b.numpy(), "fp8"), want, equal_nan=True)
    rng = np.random.default_rng(0)
    x = np.concatenate([rng.standard_normal(4000) * 60, rng.standard_normal(4000) * 2.0 ** -7,
                        o.E4M3[:127], (o.E4M3[:126] + o.E4M3[1:127]) / 2, [448.0, -448.0, 0.0]])
    x = np.clip(x, -448, 448).astype(np.float32)
    want = torch.from_numpy(x).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert np.array_equal(o.encode(x, "fp8"), want)


@pytest.mark.parametrize("fmt", ["int8", "fp8"])
def test_append_by_hand(fmt):
    """One head, one block of 8: scale and codes of three calls, from the definition."""
    top = float(o.TOP[fmt])
    codes, scale = np.full((2, 1, 8, 64), 5, np.uint8), np.array([[9.0], [7.0]], np.float32)
    x = np.zeros((2, 1, 64), np.float32)
    x[0, 0, 0], x[1, 0, 1] = top, -top / 2
    o.append(x, [0, 1], codes, scale, fmt)                      # begins anew: the old 9 is gone
    assert scale[0, 0] == 1 and scale[1, 0] == 7
    assert o.values(codes, scale, fmt)[0, 0, 0, 0] == top and (codes[0, 0, 2:] == 5).all() and (codes[1] == 5).all()
    y = np.zeros((1, 1, 64), np.float32)
    y[0, 0, 3] = 2 * top
    codes[0, 0, 3:] = 0
    o.append(y, [2], codes, scale, fmt)                         # grows: earlier codes are halved
    assert scale[0, 0] == 2
    v = o.values(codes, scale, fmt)[0, 0]
    assert v[2, 3] == 2 * top and abs(v[0, 0] - top) <= 1 and v[1, 1] <= -top / 2 + 1
    before = codes.copy()
    o.append(y / 4, [-1], codes, scale, fmt)                    # padding
    assert np.array_equal(before, codes)
    o.append(y / 4, [3], codes, scale, fmt)                     # smaller: the scale stays
    assert scale[0, 0] == 2 and np.array_equal(codes[0, 0, :3], before[0, 0, :3])


@pytest.mark.parametrize("fmt", ["int8", "fp8"])
def test_token_by_token_and_at_once_have_the_same_scale(fmt):
    rng = np.random.default_rng(1)
    x = rng.standard_normal((16, 3, 64)).astype(np.float32)
    a, b = ((np.zeros((1, 3, 16, 64), np.uint8), np.zeros((1, 3), np.float32)) for _ in "ab")
    o.append(x, np.arange(16), *a, fmt)
    for t in range(16):
        o.append(x[t: t + 1], [t], *b, fmt)
    assert np.array_equal(a[1], b[1])
    # each rescaling is off by half a step of that time's scale at most, each step is at most the last
    step = a[1][..., None, None] * (1 if fmt == "int8" else 32)
    assert (np.abs(o.values(*a, fmt) - x.transpose(1, 0, 2)[None]) <= step / 2 * (1 + 1e-6)).all()
    assert (np.abs(o.values(*b, fmt) - x.transpose(1, 0, 2)[None]) <= 8 * step).all()


def test_decode_equals_torch():
    rng = np.random.default_rng(2)
    N, Hkv, bs, d, H, n = 5, 2, 8, 64, 6, 37
    x = rng.standard_normal((2, N, Hkv, bs, d)).astype(np.float32)
    s = np.abs(x).max((3, 4)).astype(np.float32) / np.float32(127)
    codes = o.encode(x / s[..., None, None], "int8")
    q = rng.standard_normal((1, H, d))
    tbl = np.array([[3, 0, 4, 1, 2]], np.int32)
    got = o.decode(q, codes[0], codes[1], s[0], s[1], tbl, [n], 0.125, "int8")
    k, v = (torch.from_numpy(o.values(codes[i], s[i], "int8")[tbl[0]].transpose(0, 2, 1, 3).reshape(-1, Hkv, d)[:n])
            for i in range(2))
    want = torch.nn.functional.scaled_dot_product_attention(
        torch.from_numpy(q).transpose(0, 1), k.repeat_interleave(3, 1).transpose(0, 1),
        v.repeat_interleave(3, 1).transpose(0, 1), scale=0.125)
    np.testing.assert_allclose(got[0], want[:, 0].numpy(), rtol=1e-12, atol=1e-13)


def test_selection_by_hand():
    w = np.zeros((2, 1, 12), np.float32)
    w[1, 0, :9] = [0, 5, 1, np.nan, -0.0, 0.0, 3, 1, 9]
    new = np.full_like(w, 7)
    kept, n = ev.select_tokens(w, [1, -1, 2], [9, 9, 9], keep=6, first=1, last=1, new_weights=new)
    # between: positions 1 .. 7, four of them; 5, 3, 1 (lower position), 1
    assert kept[0, 0].tolist() == [0, 1, 2, 6, 7, 8] and n.tolist() == [6, 0, 0]
    assert (kept[1:] == -1).all()
    assert new[1, 0].tolist() == [0, 5, 1, 3, 1, 9] + [0] * 6 and (new[0] == 7).all()
    kept, n = ev.select_tokens(w, [1], [9], keep=7, first=0, last=0)
    assert kept[0, 0].tolist() == [0, 1, 2, 4, 6, 7, 8]          # of three zeros the last goes, and the NaN
    kept, n = ev.select_tokens(w, [1], [4], keep=7, first=0, last=0)
    assert kept[0, 0].tolist() == [0, 1, 2, 3, -1, -1, -1] and n.tolist() == [4]


def test_weights_sum_to_the_query_heads():
    rng = np.random.default_rng(3)
    q, k, v = rng.standard_normal((2, 6, 8)), *rng.standard_normal((2, 4, 8, 2, 8))
    out, w = ev.decode_weights(q, k, v, np.array([[1, 3], [2, 9]]), [11, 3], 0.3)
    for x, n in zip(w, (11, 3)):
        assert x.shape == (2, n)
        np.testing.assert_allclose(x.sum(1), 3.0, rtol=1e-12)


def test_compaction_reads_what_was_there():
    c = np.arange(4 * 2 * 1).reshape(4, 2, 1).copy()
    kept = np.array([[[1, 2, 5]]], np.int32)
    ev.compact_tokens(c, kept, [3], np.array([[3, 0, 2]]), np.array([[3, 1]]))
    # old positions 0 .. 5 hold 6 7 0 1 4 5
    assert c[3, :, 0].tolist() == [7, 0] and c[1, 0, 0] == 5 and c[1, 1, 0] == 3
