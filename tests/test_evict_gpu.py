"""Decode with accumulated weights, the choice of tokens and their compaction on the GPU."""
import numpy as np
import pytest
import torch

from oracle import evict as o
from paged_kv_cache_103_gb300 import binding
from paged_kv_cache_103_gb300 import workloads as wl

from _cache4 import dev, rand_tables

pytestmark = pytest.mark.gpu
F16, BF16 = torch.float16, torch.bfloat16
E = binding.DEVERR


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from paged_kv_cache_103_gb300 import build
    build.build()
    binding.load()


def weights_workspace(B, H, Hkv, d, tokens):
    ws = torch.empty(binding.pa_decode_weights_workspace_size(B, H, Hkv, d, tokens), dtype=torch.uint8, device="cuda")
    binding.pa_decode_workspace_init(ws)
    return ws


def bounds(q, k, v, tbl, lens, scale, dtype, ref, w):
    """(of out, of the step's weights).

    * A logit is a sum of d products of 16-bit values in fp32, in MMA steps of 16 (each rounding
      2^-22 of the largest partial sum, 8 of them at most) and two fp32 operations:
      D = 2^-19 scale sum |q| |k|.  A softmax weight is off by 2 D of itself, exp2 and its sum
      (n / 16 fp32 additions a lane, 2^-24 each, and some 40 to join) by 2^-20 + n 2^-28, the sum over the
      query heads by 2^-20: relative to the weight.
    * out: rounded once; P is two 16-bit numbers, off by 2^-16 of itself; the logits as above;
      sums over the keys in fp32, two products per 16 keys and some 64 steps of joining, each
      2^-22 of at most max |v|.
    """
    N, bs, Hkv, _ = k.shape
    B, H, d = q.shape
    G = H // Hkv
    ob = torch.finfo(dtype).eps / 2 * np.abs(ref) + 2.0 ** -24
    wb = []
    for i in range(B):
        n = int(lens[i])
        rel = np.zeros((Hkv, 1))
        if n:
            pos = np.arange(n)
            blk = np.clip(np.asarray(tbl[i], np.int64)[pos // bs], 0, N - 1)
            kk, vv = np.abs(k[blk, pos % bs]), np.abs(v[blk, pos % bs])
            for h in range(H):
                D = 2.0 ** -19 * abs(scale) * (kk[:, h // G] @ np.abs(q[i, h])).max()
                rel[h // G] = max(rel[h // G], 2 * D + 2.0 ** -19 + n * 2.0 ** -28)
                ob[i, h] += (2.0 ** -16 + 2 * D + (n / 8 + 64) * 2.0 ** -22) * vv[:, h // G].max()
        wb.append(w[i] * rel + 1e-30)
    return ob, wb


def check_weights(lens, H, Hkv, d, bs, dtype, width=None, scale=None, steps=2, seed=0, mag=1.0):
    B = len(lens)
    tbl, N = rand_tables(lens, bs, seed)
    width = width or max(max(lens), 1) + 5
    rng = np.random.default_rng(seed)
    k, v = (wl.normal_tensor((N, bs, Hkv, d), dtype, seed + x) * mag for x in (1, 2))
    for i, n in enumerate(lens):                        # nothing was written behind a context's end
        for pos in range(n, -(-n // bs) * bs):
            k[tbl[i, pos // bs], pos % bs] = float("nan")
            v[tbl[i, pos // bs], pos % bs] = float("nan")
    q = wl.normal_tensor((B, H, d), dtype, seed + 3)
    R = B + 2
    rows = rng.permutation(R)[:B].astype(np.int32)
    w0 = np.zeros((R, Hkv, width), np.float32)
    w0[:, :, ::3] = rng.random((R, Hkv, len(range(0, width, 3))))
    weights = torch.from_numpy(w0.copy()).cuda()
    out = torch.full((B, H, d), 7.0, dtype=dtype, device="cuda")
    scale = d ** -0.5 if scale is None else scale
    ws = weights_workspace(B, H, Hkv, d, sum(lens))
    dt, dl, dr = dev(tbl, np.asarray(lens, np.int32), rows)
    for _ in range(steps):
        binding.pa_decode_weights(q.cuda(), k.cuda(), v.cuda(), dt, dl, max([*lens, 1]), scale, out, weights, dr, ws)
    assert binding.pa_check_device_errors() == (E["TABLE_WIDTH"] if max(lens) > width else 0)
    qn, kn, vn = (x.double().numpy() for x in (q, k, v))
    ref, w = o.decode_weights(qn, kn, vn, tbl, lens, scale)
    ob, wb = bounds(qn, kn, vn, tbl, lens, scale, dtype, ref, w)
    assert (np.abs(out.double().cpu().numpy() - ref) <= ob).all()
    got = weights.double().cpu().numpy()
    want, bound = w0.astype(np.float64), np.zeros_like(w0, dtype=np.float64)
    for i in range(B):
        n = min(lens[i], width)
        want[rows[i], :, :n] += steps * w[i][:, :n]
        # each addition rounds the accumulator by half a step
        bound[rows[i], :, :n] = steps * wb[i][:, :n] + steps * 2.0 ** -24 * want[rows[i], :, :n]
    bad = ~(np.abs(got - want) <= bound)
    assert not bad.any(), (bad.sum(), got[bad][:4], want[bad][:4], bound[bad][:4])


@pytest.mark.parametrize("lens,H,Hkv,d,bs,dtype", [
    ([1], 1, 1, 64, 8, F16), ([1, 0], 2, 1, 128, 32, BF16), ([0, 0], 4, 2, 64, 16, F16), ([5, 0, 33], 4, 2, 64, 16, F16),
    ([32, 31, 64, 65], 3, 3, 128, 8, F16), ([100, 7, 300], 14, 2, 128, 16, BF16), ([257, 1], 8, 1, 64, 32, F16),
    ([513], 16, 1, 128, 16, F16), ([130, 300, 2, 511], 24, 2, 64, 8, BF16), ([777, 12], 32, 2, 128, 32, F16),
    ([400], 96, 2, 64, 16, BF16), ([40] * 60, 5, 5, 128, 16, F16), ([3, 200] * 9, 6, 2, 128, 16, BF16)])
def test_decode_weights(lens, H, Hkv, d, bs, dtype):
    check_weights(lens, H, Hkv, d, bs, dtype)


@pytest.mark.parametrize("d,bs,G,dtype", [(128, 16, 1, F16), (128, 16, 4, BF16), (64, 8, 7, F16), (128, 32, 16, BF16)])
def test_decode_weights_long(d, bs, G, dtype):
    check_weights([5003, 9000, 1, 2048], 2 * G, 2, d, bs, dtype)


def test_decode_weights_flat_and_sharp():
    check_weights([700, 90], 8, 2, 128, 16, F16, scale=0.0)
    check_weights([700, 90], 8, 2, 128, 16, BF16, scale=2.0)
    check_weights([700, 90], 8, 2, 64, 16, F16, scale=-0.3)


def test_decode_weights_of_contexts_wider_than_a_row():
    check_weights([100, 40, 64], 4, 2, 64, 16, F16, width=64)
    check_weights([100, 1], 2, 2, 128, 8, BF16, width=1)


def test_rows_that_take_no_part():
    """Negative rows (padding) and rows outside the accumulators: out is computed, nothing is added."""
    lens, H, Hkv, d, bs = [20, 50, 33, 0], 4, 2, 64, 16
    tbl, N = rand_tables(lens, bs, 1)
    k, v, q = (wl.normal_tensor(s, F16, x) for x, s in enumerate(((N, bs, Hkv, d), (N, bs, Hkv, d), (4, H, d))))
    weights = torch.zeros(3, Hkv, 64, device="cuda")
    out = torch.empty(4, H, d, dtype=F16, device="cuda")
    ws = weights_workspace(4, H, Hkv, d, sum(lens))
    dt, dl = dev(tbl, np.asarray(lens, np.int32))
    for rows, flag in (([-1, 2, -5, -1], 0), ([3, 2, -1, 1], E["SLOT"]), ([2 ** 31 - 1, 2, -2 ** 31, 0], E["SLOT"])):
        weights.zero_()
        binding.pa_decode_weights(q.cuda(), k.cuda(), v.cuda(), dt, dl, 50, 0.125, out, weights,
                                  torch.tensor(rows, dtype=torch.int32).cuda(), ws)
        assert binding.pa_check_device_errors() == flag
        qn, kn, vn = (x.double().numpy() for x in (q, k, v))
        ref, w = o.decode_weights(qn, kn, vn, tbl, lens, 0.125)
        ob, wb = bounds(qn, kn, vn, tbl, lens, 0.125, F16, ref, w)
        assert (np.abs(out.double().cpu().numpy() - ref) <= ob).all()
        got = weights.double().cpu().numpy()
        assert (got[:2] == 0).all() and (got[2, :, 50:] == 0).all()
        assert (np.abs(got[2, :, :50] - w[1]) <= wb[1] + 2.0 ** -24 * w[1]).all()


def test_a_workspace_for_fewer_tokens_adds_nothing():
    lens, H, Hkv, d, bs = [300, 200], 4, 2, 64, 16
    tbl, N = rand_tables(lens, bs, 1)
    k, v, q = (wl.normal_tensor(s, BF16, x) for x, s in enumerate(((N, bs, Hkv, d), (N, bs, Hkv, d), (2, H, d))))
    weights = torch.zeros(2, Hkv, 300, device="cuda")
    out = torch.empty(2, H, d, dtype=BF16, device="cuda")
    dt, dl, dr = dev(tbl, np.asarray(lens, np.int32), np.arange(2, dtype=np.int32))
    for tokens, flag in ((100, E["CONTEXT"]), (500, 0)):
        binding.pa_decode_weights(q.cuda(), k.cuda(), v.cuda(), dt, dl, 300, 0.125, out, weights, dr,
                                  weights_workspace(2, H, Hkv, d, tokens))
        assert binding.pa_check_device_errors() == flag
        ref, w = o.decode_weights(*(x.double().numpy() for x in (q, k, v)), tbl, lens, 0.125)
        ob, _ = bounds(*(x.double().numpy() for x in (q, k, v)), tbl, lens, 0.125, BF16, ref, w)
        assert (np.abs(out.double().cpu().numpy() - ref) <= ob).all()
        assert (weights.sum().item() == 0) == bool(flag)


def test_equal_calls_give_equal_weights():
    lens, H, Hkv, d, bs = [3000, 1, 777, 2900], 8, 2, 128, 16
    tbl, N = rand_tables(lens, bs, 4)
    k, v, q = (wl.normal_tensor(s, F16, x).cuda() for x, s in enumerate(((N, bs, Hkv, d), (N, bs, Hkv, d), (4, H, d))))
    dt, dl, dr = dev(tbl, np.asarray(lens, np.int32), np.arange(4, dtype=np.int32))
    ws, got = weights_workspace(4, H, Hkv, d, sum(lens)), []
    for _ in range(5):
        weights, out = torch.zeros(4, Hkv, 3000, device="cuda"), torch.empty(4, H, d, dtype=F16, device="cuda")
        binding.pa_decode_weights(q, k, v, dt, dl, 3000, 0.1, out, weights, dr, ws)
        got.append(weights)
    assert all(torch.equal(got[0], w) for w in got)


# ------------------------------------------------------------------------------- selection
def check_select(weights, rows, lens, keep, first, last, in_place=False, flag=0):
    R, Hkv, W = weights.shape
    B = len(rows)
    want_new = np.full_like(weights, 5.0) if not in_place else weights.copy()
    kept = torch.full((B, Hkv, keep), 77, dtype=torch.int32, device="cuda")
    n = torch.full((B,), 77, dtype=torch.int32, device="cuda")
    w = torch.from_numpy(weights.copy()).cuda()
    new = w if in_place else torch.full_like(w, 5.0)
    binding.pa_select_tokens(w, *dev(np.asarray(rows, np.int32), np.asarray(lens, np.int32)), first, last, kept, n, new)
    assert binding.pa_check_device_errors() == flag
    want, want_n = o.select_tokens(weights, rows, lens, keep, first, last, want_new)
    assert np.array_equal(n.cpu().numpy(), want_n)
    assert np.array_equal(kept.cpu().numpy(), want)
    assert np.array_equal(new.cpu().numpy(), want_new, equal_nan=True)
    if not in_place:
        assert np.array_equal(w.cpu().numpy(), weights, equal_nan=True)


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("Hkv,W,keep,first,last", [
    (1, 1, 1, 0, 0), (2, 40, 1, 0, 0), (2, 40, 1, 1, 0), (3, 100, 37, 4, 9), (1, 100, 20, 20, 0), (2, 100, 20, 0, 20),
    (2, 1000, 999, 1, 1), (2, 1000, 256, 0, 0), (8, 5000, 1234, 4, 100), (1, 9000, 33, 1, 1), (2, 40000, 20000, 4, 512),
    (1, 70000, 4096, 4, 64), (1, 800, 700, 5, 400), (1, 9000, 5000, 4, 3000), (1, 5000, 2048, 0, 2048),
    (1, 30000, 9000, 2000, 3000), (1, 60000, 9000, 2000, 3000), (40, 12000, 5000, 10, 2000)])
def test_select(in_place, Hkv, W, keep, first, last):
    rng = np.random.default_rng(W + keep)
    lens = sorted({W, max(1, W - 1), keep, min(W, keep + 1), max(keep - 1, 0), 0, W // 2})
    rows = rng.permutation(len(lens) + 1)[: len(lens)]
    w = rng.exponential(size=(len(lens) + 1, Hkv, W)).astype(np.float32)
    check_select(w, rows, lens, keep, first, last, in_place)


def test_select_ties_signs_and_values_that_are_no_numbers():
    rng = np.random.default_rng(0)
    for n, keep in ((500, 200), (500, 499), (2000, 37)):
        w = rng.integers(0, 3, (6, 2, n)).astype(np.float32)          # many ties
        w[1] = 1.0                                                    # nothing but ties
        w[2] = rng.standard_normal((2, n))                            # both signs
        w[3] = np.where(rng.random((2, n)) < 0.5, np.float32(-0.0), np.float32(0.0))
        w[4, :, ::3] = np.nan
        w[4, :, 1::7] = np.inf
        w[4, :, 2::11] = -np.inf
        w[5] = np.nan
        w[5, 0, 7] = 2.0 ** -149
        check_select(w, np.arange(6), [n] * 6, keep, 3, 5)
        check_select(w, np.arange(6), [n] * 6, keep, 0, 0, in_place=True)
    # keys in two far groups, the border inside each
    w = np.where(np.arange(3000) % 2 == 0, 1.0 + np.arange(3000) * 2.0 ** -23, 1e-30).astype(np.float32)[None, None]
    for keep in (100, 1500, 1501, 2900):
        check_select(w, [0], [3000], keep, 0, 0)


def test_select_reports_and_leaves_out():
    w = np.random.default_rng(1).random((4, 2, 50)).astype(np.float32)
    check_select(w, [2, -1, 0], [50, 50, 30], 20, 2, 3)
    check_select(w, [2, 4, 0], [50, 50, 30], 20, 2, 3, flag=E["SLOT"])
    check_select(w, [2, 3, 0], [50, -4, 30], 20, 2, 3, flag=E["CONTEXT"])
    check_select(w, [2, 3, 0], [50, 51, 2 ** 31 - 1], 20, 2, 3, flag=E["TABLE_WIDTH"])


@pytest.mark.parametrize("pairs_each", [2, 100, 130])
@pytest.mark.parametrize("W", [20000, 100000])
def test_select_short_contexts_of_wide_rows(W, pairs_each):
    """What one launch's rows may hold is far more than its contexts do; one of them does hold it."""
    rng = np.random.default_rng(W)
    lens = [700, 8200, 2100, 30, W, 8300]
    w = rng.standard_normal((6, pairs_each, W)).astype(np.float32)
    w[1] = rng.integers(0, 4, (pairs_each, W))
    for in_place in (False, True):
        check_select(w, [3, 1, 0, 4, 2, 5], lens, 600, 3, 50, in_place)


def test_select_without_new_weights():
    w = torch.rand(2, 3, 64, device="cuda")
    kept, n = torch.empty(2, 3, 10, dtype=torch.int32, device="cuda"), torch.empty(2, dtype=torch.int32, device="cuda")
    binding.pa_select_tokens(w, *dev(np.array([1, 0], np.int32), np.array([64, 9], np.int32)), 1, 1, kept, n)
    want, want_n = o.select_tokens(w.cpu().numpy(), [1, 0], [64, 9], 10, 1, 1)
    assert np.array_equal(kept.cpu().numpy(), want) and np.array_equal(n.cpu().numpy(), want_n)


# ------------------------------------------------------------------------------ compaction
def pick(lens, Hkv, keep, seed):
    rng = np.random.default_rng(seed)
    kept, n = np.full((len(lens), Hkv, keep), -1, np.int32), np.minimum(lens, keep).astype(np.int32)
    for i, m in enumerate(n):
        for g in range(Hkv):
            kept[i, g, :m] = np.sort(rng.choice(lens[i], m, replace=False))
    return kept, n


@pytest.mark.parametrize("fresh", [0, 2, 1000])
@pytest.mark.parametrize("lens,Hkv,keep,d,bs,dtype", [
    ([1], 1, 1, 64, 8, F16), ([10, 0, 3], 2, 4, 128, 16, BF16), ([100, 64, 7], 3, 33, 64, 8, F16),
    ([500, 501, 16, 15, 17], 2, 250, 128, 32, BF16), ([3000, 2000], 1, 1999, 128, 16, F16),
    ([5000], 5, 4990, 64, 16, BF16), ([700] * 20, 8, 77, 128, 16, F16)])
def test_compact(fresh, lens, Hkv, keep, d, bs, dtype):
    tbl, N = rand_tables(lens, bs, 1)
    width = (keep + bs - 1) // bs
    new = np.full((len(lens), width), -1, np.int32)
    new[:, : tbl.shape[1]] = tbl[:, :width]
    nb = [-(-min(n, keep) // bs) for n in lens]
    for i, m in enumerate(nb):                           # the first `fresh` blocks are replaced
        f = min(fresh, m)
        new[i, :f] = np.arange(N, N + f)
        N += f
        new[i, m:] = -1
    rng = np.random.default_rng(2)
    host = [rng.integers(-2 ** 15, 2 ** 15, (N, bs, Hkv, d)).astype(np.int16) for _ in "kv"]
    kept, n = pick(lens, Hkv, keep, 3)
    kc, vc = (x.view(dtype) for x in dev(*host))
    binding.pa_compact_tokens(kc, vc, *dev(kept, n, tbl, new))
    assert binding.pa_check_device_errors() == 0
    for got, want in zip((kc, vc), host):
        o.compact_tokens(want, kept, n, tbl, new)
        assert np.array_equal(got.view(torch.int16).cpu().numpy(), want)


def test_compact_reports_bad_entries_and_moves_the_rest():
    bs, Hkv, d, N = 8, 1, 64, 6
    host = np.random.default_rng(2).integers(-2 ** 15, 2 ** 15, (N, bs, Hkv, d)).astype(np.int16)
    kept = np.array([[[1, 9, 20, 30]], [[0, 2, 9, 17]], [[-3, 5, 6, 7]]], np.int32)
    tbl = np.array([[0, 1, -1], [2, 77, 3], [4, -1, -1]], np.int32)       # 30 lies behind a table of 24
    kc, vc = (x.view(F16) for x in dev(host, host))
    binding.pa_compact_tokens(kc, vc, *dev(kept, np.array([4, 4, 3], np.int32), tbl, tbl))
    assert binding.pa_check_device_errors() == E["TABLE_WIDTH"] | E["BLOCK_ID"]
    want = host.copy()
    want[0, :2, 0] = host[0, 1, 0], host[1, 1, 0]
    want[2, 1, 0], want[2, 3, 0] = host[2, 2, 0], host[3, 1, 0]
    want[4, 1, 0], want[4, 2, 0] = host[4, 5, 0], host[4, 6, 0]
    for got in (kc, vc):
        assert np.array_equal(got.view(torch.int16).cpu().numpy(), want)
    for bad in (-1, 5):
        binding.pa_compact_tokens(kc, vc, *dev(kept[:1] * 0, np.array([bad], np.int32), tbl[:1], tbl[:1, :1]))
        assert binding.pa_check_device_errors() & E["CONTEXT"]


# -------------------------------------------------------------------------- as they are used
@pytest.mark.parametrize("dtype,G", [(F16, 1), (BF16, 4)])
def test_a_run_of_steps_with_evictions(dtype, G):
    """Three sequences, two of them forked from one, decode under a budget: append, decode with
    weights, and at 96 tokens cut to 64; every step against a host model that follows the same choices."""
    Hkv, d, bs, budget, keep, first, last, width = 2, 64, 8, 96, 64, 2, 16, 128
    H, N, B = Hkv * G, 80, 3
    alloc = binding.Allocator(N, bs)
    alloc.alloc(0, 90)
    alloc.fork(0, 1)
    alloc.alloc(2, 30)
    ids = [0, 1, 2]
    k, v = (torch.zeros(N, bs, Hkv, d, dtype=dtype, device="cuda") for _ in "kv")
    model = {i: [np.zeros((0, Hkv, d)) for _ in "kv"] for i in ids}
    for s, n in ((0, 90), (2, 30)):
        kn, vn = (wl.normal_tensor((n, Hkv, d), dtype, 50 + s + x) for x in (0, 1))
        binding.pa_reshape_and_cache(kn.cuda(), vn.cuda(), torch.from_numpy(alloc.seq_slots(s, 0, n)).cuda(), k, v)
        for i in ([0, 1] if s == 0 else [2]):
            model[i] = [kn.double().numpy(), vn.double().numpy()]
    rows = np.array([4, 0, 2], np.int32)
    weights = torch.zeros(5, Hkv, width, device="cuda")
    ws = weights_workspace(B, H, Hkv, d, B * width)
    evictions = 0
    for step in range(90):
        kn, vn = (wl.normal_tensor((B, Hkv, d), dtype, 1000 + 2 * step + x) for x in (0, 1))
        q = wl.normal_tensor((B, H, d), dtype, 5000 + step)
        slots, cow = alloc.append_batch(ids)
        if len(cow):
            binding.pa_copy_blocks([k], [v], torch.from_numpy(np.asarray(cow, np.int32)).cuda())
        binding.pa_reshape_and_cache(kn.cuda(), vn.cuda(), torch.from_numpy(slots).cuda(), k, v)
        tbl, lens = alloc.export(ids, 16)
        out = torch.empty(B, H, d, dtype=dtype, device="cuda")
        before = weights.double().cpu().numpy()
        binding.pa_decode_weights(q.cuda(), k, v, *dev(tbl, lens), int(lens.max()), 0.125, out, weights,
                                  torch.from_numpy(rows).cuda(), ws)
        got, after = out.double().cpu().numpy(), weights.double().cpu().numpy()
        for b, i in enumerate(ids):
            model[i] = [np.concatenate([m, x[b: b + 1].double().numpy()]) for m, x in zip(model[i], (kn, vn))]
            n = len(model[i][0])
            assert n == lens[b]
            one = np.arange(1)[None]
            kk, vv = (m[None] for m in model[i])         # one block of n tokens
            ref, w = o.decode_weights(q[b: b + 1].double().numpy(), kk, vv, one, [n], 0.125)
            ob, wb = bounds(q[b: b + 1].double().numpy(), kk, vv, one, [n], 0.125, dtype, ref, w)
            assert (np.abs(got[b] - ref[0]) <= ob[0]).all(), (step, i)
            sum_ = before[rows[b], :, :n] + w[0]
            assert (np.abs(after[rows[b], :, :n] - sum_) <= wb[0] + 2.0 ** -24 * sum_).all(), (step, i)
        full = [b for b in range(B) if lens[b] == budget]
        if not full:
            continue
        evictions += len(full)
        kept = torch.empty(len(full), Hkv, keep, dtype=torch.int32, device="cuda")
        n = torch.empty(len(full), dtype=torch.int32, device="cuda")
        binding.pa_select_tokens(weights, *dev(rows[full], lens[full]), first, last, kept, n, weights)
        for b in full:
            alloc.evict(ids[b], keep)
        new, new_lens = alloc.export([ids[b] for b in full], 16)
        assert (new_lens == keep).all()
        binding.pa_compact_tokens(k, v, kept, n, *dev(tbl[full], new))
        for x, b in enumerate(full):
            p = kept[x].cpu().numpy()
            assert (p[:, :first] == np.arange(first)).all() and (p[:, -last:] == np.arange(budget - last, budget)).all()
            model[ids[b]] = [np.stack([m[p[g], g] for g in range(Hkv)], 1) for m in model[ids[b]]]
            assert (weights[rows[b], :, keep:] == 0).all()
    # the two that begin at 90 tokens at steps 6, 38 and 70, the one that begins at 30 at step 66
    assert evictions == 7 and binding.pa_check_device_errors() == 0
