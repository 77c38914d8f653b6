"""Block-sparse decode on the GPU: boxes and selections exactly as the oracle's, the decode of the
selected blocks within the 16-bit decode's bound of it."""
import numpy as np
import pytest
import torch

from oracle import cache4 as o
from paged_kv_cache_103_gb300 import binding
from paged_kv_cache_103_gb300 import workloads as wl

from _cache4 import behind, dev, rand_tables, workspace
from _harness import assert_close

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from paged_kv_cache_103_gb300 import build
    build.build()
    binding.load()


def _boxes(N, Hkv, d):
    return (torch.full((N, Hkv, 2, d), 99, dtype=torch.int8, device="cuda"),
            torch.full((N, Hkv), -1.0, device="cuda"))


@pytest.mark.parametrize("N,bs,Hkv,d,dtype,n", [(1, 8, 1, 64, torch.float16, 1), (9, 16, 3, 128, torch.bfloat16, 5),
                                                (40, 32, 4, 64, torch.bfloat16, 33), (300, 8, 5, 128, torch.float16, 257)])
def test_summaries_are_exact(N, bs, Hkv, d, dtype, n):
    rng = np.random.default_rng(N)
    k = wl.normal_tensor((N, bs, Hkv, d), dtype, N) * 3
    k[0, :, 0] = 0                                     # S = 0
    k[N // 2, 0, :, 1] = 60000.0
    ids = rng.permutation(N)[:n].astype(np.int32)
    fills = rng.integers(0, bs + 1, n).astype(np.int32)
    fills[: n // 2] = bs
    kn = k.clone()
    for b, f in zip(ids, fills):
        kn[int(b), int(f):] = float("nan")             # rows behind the fill are not read
    boxes, S = _boxes(N, Hkv, d)
    binding.pa_summarize_blocks(kn.cuda(), *dev(ids), boxes, S, dev(fills)[0])
    assert binding.pa_check_device_errors() == 0
    hb, hs = np.full((N, Hkv, 2, d), 99, np.int8), np.full((N, Hkv), -1, np.float32)
    o.summarize_blocks(k.float().numpy(), ids, fills, hb, hs)
    assert np.array_equal(boxes.cpu().numpy(), hb) and np.array_equal(S.cpu().numpy(), hs)
    # without fills every row counts; an id twice is written twice alike
    twice = np.concatenate([ids[:1], ids[:1]])
    binding.pa_summarize_blocks(k.cuda(), *dev(twice), boxes, S)
    o.summarize_blocks(k.float().numpy(), twice, [bs, bs], hb, hs)
    assert np.array_equal(boxes.cpu().numpy(), hb) and np.array_equal(S.cpu().numpy(), hs)


def test_bad_ids_and_fills_are_flagged():
    k = wl.normal_tensor((4, 8, 2, 64), torch.float16, 1)
    boxes, S = _boxes(4, 2, 64)
    binding.pa_summarize_blocks(k.cuda(), *dev(np.array([4, -1, 2], np.int32)), boxes, S)
    assert binding.pa_check_device_errors() == binding.DEVERR["BLOCK_ID"]
    assert (S[[0, 1, 3]] == -1).all() and (S[2] > 0).all()
    binding.pa_summarize_blocks(k.cuda(), *dev(np.array([0, 1], np.int32)), boxes, S,
                                dev(np.array([9, -2], np.int32))[0])
    assert binding.pa_check_device_errors() == binding.DEVERR["CONTEXT"]
    hb, hs = np.full((4, 2, 2, 64), 99, np.int8), np.full((4, 2), -1, np.float32)
    o.summarize_blocks(k.float().numpy(), [0, 1], [8, 0], hb, hs)
    assert np.array_equal(boxes.cpu().numpy()[:2], hb[:2])


def _case(lens, bs, H, Hkv, d, dtype, seed):
    tbl, N = rand_tables(lens, bs, seed)
    k, v = (wl.normal_tensor((N, bs, Hkv, d), dtype, seed * 7 + i) for i in (1, 2))
    q = wl.normal_tensor((len(lens), H, d), dtype, seed * 7 + 3)
    hb, hs = np.zeros((N, Hkv, 2, d), np.int8), np.zeros((N, Hkv), np.float32)
    o.summarize_blocks(k.float().numpy(), range(N), [bs] * N, hb, hs)
    for b, r in behind(lens, tbl, bs):
        k[b, r], v[b, r] = float("nan"), float("nan")
    return q, k, v, tbl, hb, hs


def _select(q, hb, hs, tbl, lens, bs, keep, first, last, ws=None):
    B, H, d = q.shape
    Hkv = hb.shape[1]
    sel = torch.full((B, Hkv, keep), 77, dtype=torch.int32, device="cuda")
    n = torch.full((B, Hkv), 77, dtype=torch.int32, device="cuda")
    if ws is None:
        ws = torch.empty(binding.pa_select_blocks_workspace_size(B, Hkv, tbl.shape[1]), dtype=torch.uint8,
                         device="cuda")
        binding.pa_decode_workspace_init(ws)
    binding.pa_select_blocks(q.cuda(), *dev(hb, hs, tbl, np.asarray(lens, np.int32)), bs, first, last, sel, n, ws)
    return sel, n


CASES = [  # lens, bs, H, Hkv, d, dtype, keep, first, last
    ([1], 8, 1, 1, 64, torch.float16, 1, 0, 1),
    ([0, 8, 9, 200], 8, 2, 1, 64, torch.bfloat16, 3, 1, 2),
    ([700, 0, 1000, 64], 16, 8, 2, 128, torch.bfloat16, 8, 1, 2),
    ([3000, 5, 1500], 16, 28, 4, 128, torch.bfloat16, 40, 1, 4),
    ([5000], 8, 3, 3, 128, torch.float16, 200, 2, 1),
    ([900, 901, 927, 928, 929], 32, 12, 1, 64, torch.float16, 7, 0, 1),
    ([600, 20], 16, 32, 1, 128, torch.float16, 20, 3, 3),          # two groups of 16 heads
    ([40000], 8, 4, 1, 64, torch.bfloat16, 333, 0, 1),
    ([300, 77], 16, 40, 40, 128, torch.float16, 6, 1, 1),          # more KV heads than lane groups
    ([260], 16, 70, 70, 64, torch.bfloat16, 5, 0, 2),
    ([100, 33], 8, 4, 2, 64, torch.float16, 40, 1, 1),             # everything is kept
    ([200, 90], 8, 4, 2, 64, torch.float16, 3, 1, 2),              # nothing but the ends is
]


@pytest.mark.parametrize("lens,bs,H,Hkv,d,dtype,keep,first,last", CASES)
def test_select_then_decode(lens, bs, H, Hkv, d, dtype, keep, first, last):
    q, k, v, tbl, hb, hs = _case(lens, bs, H, Hkv, d, dtype, len(lens) + bs)
    sel, n = _select(q, hb, hs, tbl, lens, bs, keep, first, last)
    want, wn = o.select_blocks(q.float().numpy(), hb, hs, tbl, lens, bs, keep, first, last)
    assert np.array_equal(n.cpu().numpy(), wn)
    assert np.array_equal(sel.cpu().numpy(), want)
    out = torch.full_like(q, float("nan"), device="cuda")
    binding.pa_decode_selected(q.cuda(), k.cuda(), v.cuda(), sel, n, keep * bs, d ** -0.5, out,
                               workspace(len(lens), H, d))
    assert binding.pa_check_device_errors() == 0
    ref = o.decode_selected(q.double().numpy(), k.double().numpy(), v.double().numpy(), want, wn, d ** -0.5)
    assert_close(out.cpu(), ref)


@pytest.mark.parametrize("scores", ["equal", "zero", "two"])
@pytest.mark.parametrize("nblk,keep", [(50, 7), (515, 300), (2052, 300), (5000, 64), (9001, 5000)])
def test_ties_go_to_the_lower_position(scores, nblk, keep):
    bs, d, Hkv = 8, 64, 2
    lens = [nblk * bs - 3]
    tbl, N = rand_tables(lens, bs, 4)
    rng = np.random.default_rng(5)
    hb, hs = np.zeros((N, Hkv, 2, d), np.int8), np.ones((N, Hkv), np.float32)
    if scores != "zero":
        hb[..., 0] = 3 if scores == "equal" else rng.integers(3, 5, (N, Hkv, 1))
    q = torch.zeros(1, 4, d, dtype=torch.float16)
    q[..., 0], q[0, 2:, 0] = 1, -1                     # negative scores for the second KV head
    sel, n = _select(q, hb, hs, tbl, lens, bs, keep, 2, 2)
    want, wn = o.select_blocks(q.float().numpy(), hb, hs, tbl, lens, bs, keep, 2, 2)
    assert np.array_equal(sel.cpu().numpy(), want) and np.array_equal(n.cpu().numpy(), wn)


@pytest.mark.parametrize("H,Hkv,d", [(128, 1, 128), (256, 2, 64)])
def test_selection_for_wide_groups(H, Hkv, d):
    """Up to 128 query heads a KV head (the decode takes them sixteen at a time)."""
    lens, bs = [900, 250], 16
    q, k, v, tbl, hb, hs = _case(lens, bs, H, Hkv, d, torch.bfloat16, 5)
    sel, n = _select(q, hb, hs, tbl, lens, bs, 9, 1, 1)
    want, wn = o.select_blocks(q.float().numpy(), hb, hs, tbl, lens, bs, 9, 1, 1)
    assert np.array_equal(sel.cpu().numpy(), want) and np.array_equal(n.cpu().numpy(), wn)


def test_scores_of_every_sign_zero_and_subnormal_order_alike():
    """Keys far below one, queries of both signs, boxes of zero scale among them."""
    lens, bs, Hkv, d = [1600], 8, 2, 64
    q, k, v, tbl, hb, hs = _case(lens, bs, 4, Hkv, d, torch.float16, 9)
    hs *= np.float32(2.0) ** np.random.default_rng(3).integers(-140, 20, hs.shape).astype(np.float32)
    hs[::7] = 0
    q[0, 1] = 0
    sel, n = _select(q, hb, hs, tbl, lens, bs, 60, 0, 1)
    want, wn = o.select_blocks(q.float().numpy(), hb, hs, tbl, lens, bs, 60, 0, 1)
    assert np.array_equal(sel.cpu().numpy(), want)


def test_selection_flags_bad_input():
    bs, d = 8, 64
    lens = [100, 50, 90]
    q, k, v, tbl, hb, hs = _case(lens, bs, 2, 1, d, torch.float16, 3)
    bad = tbl.copy()
    bad[0, 4] = tbl.max() + 100                        # ranks last, so it is not chosen
    sel, n = _select(q, hb, hs, bad, lens, bs, 4, 1, 1)
    assert binding.pa_check_device_errors() == binding.DEVERR["BLOCK_ID"]
    good = np.delete(np.arange(13), 4)
    want, _ = o.select_blocks(q.float().numpy(), hb, hs, np.pad(tbl[:, good], ((0, 0), (0, 1)), constant_values=-1),
                              [92, 50, 82], bs, 4, 1, 1)
    assert np.array_equal(sel[0].cpu().numpy(), want[0])
    sel, n = _select(q, hb, hs, tbl, [105, -1, 90], bs, 4, 1, 1)
    assert binding.pa_check_device_errors() == binding.DEVERR["CONTEXT"] | binding.DEVERR["TABLE_WIDTH"]
    assert (sel[1] == -1).all() and int(n[1, 0]) == 0 and int(n[0, 0]) == 4 * bs


def test_a_workspace_is_reused_and_repeats_agree():
    lens, bs, H, Hkv, d = [9000, 300, 4000], 16, 8, 4, 128
    q, k, v, tbl, hb, hs = _case(lens, bs, H, Hkv, d, torch.bfloat16, 2)
    ws = torch.zeros(binding.pa_select_blocks_workspace_size(3, Hkv, tbl.shape[1]), dtype=torch.uint8,
                     device="cuda")
    a = _select(q, hb, hs, tbl, lens, bs, 30, 1, 1, ws)
    _select(q[:1], hb, hs, tbl[:1, :200], lens[:1], bs, 5, 0, 1, ws)
    binding.pa_check_device_errors()
    for _ in range(5):
        b = _select(q, hb, hs, tbl, lens, bs, 30, 1, 1, ws)
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    assert binding.pa_check_device_errors() == 0


def test_lists_per_kv_head_need_not_come_from_the_selection():
    """Any block lists and lengths, the same block in several of them, an empty pair among them."""
    N, bs, H, Hkv, d = 9, 16, 6, 3, 128
    k, v = (wl.normal_tensor((N, bs, Hkv, d), torch.float16, s) for s in (1, 2))
    q = wl.normal_tensor((2, H, d), torch.float16, 3)
    sel = np.random.default_rng(2).integers(0, N, (2, Hkv, 5)).astype(np.int32)
    n = np.array([[80, 0, 33], [1, 16, 70]], np.int32)
    out = torch.full_like(q, float("nan"), device="cuda")
    binding.pa_decode_selected(q.cuda(), k.cuda(), v.cuda(), *dev(sel, n), 80, 0.1, out, workspace(2, H, d))
    assert binding.pa_check_device_errors() == 0
    ref = o.decode_selected(q.double().numpy(), k.double().numpy(), v.double().numpy(), sel, n, 0.1)
    assert_close(out.cpu(), ref)
    assert (out[0, 2:4] == 0).all()


def test_summaries_selection_and_decode_in_one_graph():
    """A decode step as a program replays it: the filled block summarised, blocks chosen, attended."""
    lens, bs, H, Hkv, d, keep = [1000, 640], 16, 8, 2, 128, 10
    q, k, v, tbl, hb, hs = _case(lens, bs, H, Hkv, d, torch.bfloat16, 6)
    fresh = np.array([tbl[0, 3], tbl[1, 20]], np.int32)
    stale_b, stale_s = hb.copy(), hs.copy()
    stale_b[fresh], stale_s[fresh] = 0, 0
    dq, dk, dv = q.cuda(), k.cuda(), v.cuda()
    db, ds, dt, dl, df = dev(stale_b, stale_s, tbl, np.asarray(lens, np.int32), fresh)
    sel = torch.empty(2, Hkv, keep, dtype=torch.int32, device="cuda")
    n = torch.empty(2, Hkv, dtype=torch.int32, device="cuda")
    out, ws = torch.empty_like(dq), workspace(2, H, d)
    sws = torch.zeros(binding.pa_select_blocks_workspace_size(2, Hkv, tbl.shape[1]), dtype=torch.uint8,
                      device="cuda")
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        binding.pa_summarize_blocks(dk, df, db, ds)
        binding.pa_select_blocks(dq, db, ds, dt, dl, bs, 1, 2, sel, n, sws)
        binding.pa_decode_selected(dq, dk, dv, sel, n, keep * bs, d ** -0.5, out, ws)
    for seed in (1, 2):
        x = wl.normal_tensor(q.shape, torch.bfloat16, seed)
        dq.copy_(x)
        graph.replay()
        torch.cuda.synchronize()
        assert binding.pa_check_device_errors() == 0
        want, wn = o.select_blocks(x.float().numpy(), hb, hs, tbl, lens, bs, keep, 1, 2)
        assert np.array_equal(sel.cpu().numpy(), want) and np.array_equal(n.cpu().numpy(), wn)
        ref = o.decode_selected(x.double().numpy(), k.double().numpy(), v.double().numpy(), want, wn, d ** -0.5)
        assert_close(out.cpu(), ref)
