"""Block-sparse decode at the sizes where its calls change form or meet their limits."""
import numpy as np
import pytest
import torch

from oracle import cache4 as o
from paged_kv_cache_103_gb300 import binding

from _cache4 import workspace
from _harness import assert_close
from test_sparse_gpu import _case, _select

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from paged_kv_cache_103_gb300 import build
    build.build()
    binding.load()


@pytest.mark.parametrize("B,H,Hkv,d", [(128, 40, 40, 128), (103, 80, 40, 64), (4096, 4, 2, 64)])
def test_what_is_selected_can_be_decoded(B, H, Hkv, d):
    """Batches of more than 4096 (sequence, KV head) pairs, ragged last part among them."""
    rng = np.random.default_rng(B)
    bs, keep = 8, 3
    lens = rng.integers(0, 60, B).tolist()
    q, k, v, tbl, hb, hs = _case(lens, bs, H, Hkv, d, torch.float16, 3)
    sel, n = _select(q, hb, hs, tbl, lens, bs, keep, 0, 1)
    want, wn = o.select_blocks(q.float().numpy(), hb, hs, tbl, lens, bs, keep, 0, 1)
    assert np.array_equal(sel.cpu().numpy(), want) and np.array_equal(n.cpu().numpy(), wn)
    out = torch.full_like(q, float("nan"), device="cuda")
    ws = workspace(B, H, d)
    for _ in range(2):
        binding.pa_decode_selected(q.cuda(), k.cuda(), v.cuda(), sel, n, keep * bs, d ** -0.5, out, ws)
    assert binding.pa_check_device_errors() == 0
    ref = o.decode_selected(q.double().numpy(), k.double().numpy(), v.double().numpy(), want, wn, d ** -0.5)
    assert_close(out.cpu(), ref)
    assert int(ws[: B * H * 4].view(torch.int32).abs().sum()) == 0


@pytest.mark.parametrize("at,keep,last", [(0, 4, 1), (12, 4, 1), (11, 4, 2), (5, 13, 1), (5, 40, 1)])
@pytest.mark.parametrize("bad_id", [-1, 1 << 20])
def test_a_bad_id_is_flagged_where_it_is_kept_unscored(at, keep, last, bad_id):
    """The first and last blocks, and all of them where nothing is left out, are listed without a
    score; an id outside the pool among them is passed on and flagged like any other."""
    lens, bs = [100, 30], 8
    q, k, v, tbl, hb, hs = _case(lens, bs, 6, 3, 64, torch.float16, 3)
    good = tbl.copy()
    tbl[0, at] = bad_id
    sel, n = _select(q, hb, hs, tbl, lens, bs, keep, 1, last)
    assert binding.pa_check_device_errors() == binding.DEVERR["BLOCK_ID"]
    want, wn = o.select_blocks(q.float().numpy(), hb, hs, good, lens, bs, keep, 1, last)
    assert np.array_equal(sel.cpu().numpy(), np.where(want == good[0, at], bad_id, want))
    assert np.array_equal(n.cpu().numpy(), wn)
    _select(q, hb, hs, good, lens, bs, keep, 1, last)
    assert binding.pa_check_device_errors() == 0


@pytest.mark.parametrize("bs,H,Hkv,d,W", [(8, 8, 2, 128, 3000), (16, 6, 3, 64, 700), (8, 40, 40, 128, 1200),
                                          (32, 4, 1, 64, 9000)])
def test_tables_much_wider_than_their_contexts(bs, H, Hkv, d, W):
    """The lists do not depend on a table's width, whatever form and shares it makes the call take."""
    lens = [0, 5, 40 * bs, 41 * bs - 3, 300 * bs + 1, 130 * bs, 1000]
    q, k, v, tbl, hb, hs = _case(lens, bs, H, Hkv, d, torch.bfloat16, 6)
    wide = np.full((len(lens), W), -1, np.int32)
    wide[:, : tbl.shape[1]] = tbl
    for keep, first, last in ((4, 1, 1), (40, 0, 2), (70, 3, 1)):
        want, wn = o.select_blocks(q.float().numpy(), hb, hs, tbl, lens, bs, keep, first, last)
        for t in (tbl, wide):
            sel, n = _select(q, hb, hs, t, lens, bs, keep, first, last)
            assert binding.pa_check_device_errors() == 0
            assert np.array_equal(n.cpu().numpy(), wn) and np.array_equal(sel.cpu().numpy(), want)


def test_a_wide_table_costs_little():
    """8 contexts of 512 blocks: in tables of 8192 the selection took 4 times as long as in tables
    of 512 while its shares were cut from the table (31.4 against 7.7 us), 1.7 times since."""
    B, Hkv, G, d, bs, nb, keep = 8, 8, 4, 128, 16, 512, 64
    gen = torch.Generator().manual_seed(1)
    boxes = torch.randint(-100, 100, (B * nb, Hkv, 2, d), dtype=torch.int8, generator=gen).cuda()
    S = torch.rand(B * nb, Hkv, generator=gen).cuda()
    ids = torch.randperm(B * nb, generator=gen).view(B, nb).int()
    lens = torch.full((B,), nb * bs, dtype=torch.int32).cuda()
    q = torch.randn(B, Hkv * G, d, generator=gen).bfloat16().cuda()
    sel = torch.empty(B, Hkv, keep, dtype=torch.int32).cuda()
    n = torch.empty(B, Hkv, dtype=torch.int32).cuda()
    times = []
    for W in (nb, 16 * nb):
        tbl = torch.full((B, W), -1, dtype=torch.int32)
        tbl[:, :nb] = ids
        tbl = tbl.cuda()
        ws = torch.empty(binding.pa_select_blocks_workspace_size(B, Hkv, W), dtype=torch.uint8).cuda()
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            for _ in range(20):
                binding.pa_select_blocks(q, boxes, S, tbl, lens, bs, 1, 2, sel, n, ws)
        best = 1e9
        for _ in range(10):
            a, b = (torch.cuda.Event(enable_timing=True) for _ in range(2))
            a.record()
            graph.replay()
            b.record()
            torch.cuda.synchronize()
            best = min(best, a.elapsed_time(b))
        times.append(best)
    assert times[1] < 3 * times[0], times


@pytest.mark.parametrize("H,Hkv,d", [(2, 2, 128), (12, 3, 64), (8, 1, 128), (16, 1, 128), (32, 1, 64)])
def test_an_f16_result_over_chosen_blocks_is_off_by_its_own_rounding(H, Hkv, d):
    """Root mean squares, r that of the output's rounding (known from the reference; some 2^-12.3 of
    the result): a probability in two f16 parts is off by 2^-22 of itself, or 2^-25 of the largest,
    and the fp32 steps by less than 2^-18 together (logits of a few units: 2^-21 each, exp2 2^-22, sums
    of at most 64 keys on the tensor cores 2^-21), 2% of r; a single f16 part gives 1.1 r and more."""
    B, bs, n = 24, 16, 60
    rng = np.random.default_rng(H)
    N = 40
    k, v = (torch.from_numpy(rng.standard_normal((N, bs, Hkv, d)).astype(np.float32)).half() for _ in "kv")
    q = torch.from_numpy(rng.standard_normal((B, H, d)).astype(np.float32)).half()
    sel = rng.integers(0, N, (B, Hkv, 4)).astype(np.int32)
    lens = np.full((B, Hkv), n, np.int32)
    out = torch.empty_like(q, device="cuda")
    binding.pa_decode_selected(q.cuda(), k.cuda(), v.cuda(), torch.from_numpy(sel).cuda(), torch.from_numpy(lens).cuda(),
                               64, d ** -0.5, out, workspace(B, H, d))
    assert binding.pa_check_device_errors() == 0
    ref = o.decode_selected(q.double().numpy(), k.double().numpy(), v.double().numpy(), sel, lens, d ** -0.5)
    rms = lambda x: float(np.sqrt(np.mean(np.square(x))))  # noqa: E731
    r = rms(ref.astype(np.float16).astype(np.float64) - ref)
    assert rms(out.cpu().double().numpy() - ref) <= 1.02 * r, rms(out.cpu().double().numpy() - ref) / r
