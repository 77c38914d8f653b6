"""pa_decode_int4 against the fp64 oracle over the same codes, with bounds derived in
_cache4.decode_bound."""
import numpy as np
import pytest
import torch

from oracle import cache4 as o
from paged_kv_cache_103_gb300 import binding
from paged_kv_cache_103_gb300 import workloads as wl

from _cache4 import decode_bound, dev, int4_cache, nan_behind, rand_tables, workspace
from _harness import assert_close

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from paged_kv_cache_103_gb300 import build
    build.build()
    binding.load()


def run(q, cache, tbl, lens, scale, ws=None, out=None, max_len=None):
    B, H, d = q.shape
    out = torch.full_like(q, float("nan"), device="cuda") if out is None else out
    ws = workspace(B, H, d) if ws is None else ws
    binding.pa_decode_int4(q.cuda(), *dev(*cache), *dev(np.asarray(tbl, np.int32), np.asarray(lens, np.int32)),
                           int(max(lens, default=0)) if max_len is None else max_len, scale, out, ws)
    return out


def check(q, cache, tbl, lens, scale, got):
    qd = q.double().numpy()
    ref = o.decode_int4(qd, *cache, tbl, lens, scale)
    err = np.abs(got.cpu().double().numpy() - ref)
    bound = decode_bound(qd, cache, tbl, lens, scale, q.dtype, ref)
    assert (err <= bound).all(), "worst %.3g of its bound" % (err / bound).max()
    return float((err / bound).max())


CASES = [  # H, Hkv, d, bs, dtype, lens
    (4, 2, 64, 16, torch.float16, [1, 64, 17, 33]),
    (1, 1, 64, 8, torch.bfloat16, [1]),
    (1, 1, 128, 32, torch.float16, [0]),
    (2, 1, 128, 8, torch.bfloat16, [0, 7, 8, 9, 0, 129]),
    (40, 40, 128, 16, torch.float16, [130, 1, 555]),
    (32, 8, 128, 16, torch.bfloat16, [1024]),
    (28, 4, 128, 32, torch.bfloat16, [31, 32, 33, 0, 700, 2000]),
    (28, 4, 64, 8, torch.float16, [63, 64, 65, 500]),
    (24, 3, 128, 16, torch.float16, [300, 15, 16, 17]),
    (12, 1, 128, 16, torch.bfloat16, [400, 3]),
    (16, 1, 64, 32, torch.bfloat16, [257, 1000]),
    (32, 1, 128, 8, torch.float16, [100, 65]),        # 32 heads a KV head: two groups of 16
    (96, 2, 128, 16, torch.bfloat16, [77]),
    (8, 8, 128, 16, torch.bfloat16, [5000, 1]),       # one long context over many CTAs
]


@pytest.mark.parametrize("H,Hkv,d,bs,dtype,lens", CASES)
def test_matches_the_oracle(H, Hkv, d, bs, dtype, lens):
    tbl, N = rand_tables(lens, bs, H + d)
    cache = int4_cache(N, Hkv, bs, d, H + bs)
    nan_behind(cache, lens, tbl, bs)
    q = wl.normal_tensor((len(lens), H, d), dtype, H * 3 + d)
    got = run(q, cache, tbl, lens, d ** -0.5)
    assert binding.pa_check_device_errors() == 0
    check(q, cache, tbl, lens, d ** -0.5, got)


@pytest.mark.parametrize("mag,shift,qmag", [(1e-4, 0.0, 1.0), (100.0, 0.0, 0.05), (0.01, 5.0, 1.0),
                                            (1.0, 0.0, 2.0 ** -12), (3e-7, 0.0, 1.0), (4000.0, 0.0, 1e-3)])
@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
def test_small_large_and_shifted_values(mag, shift, qmag, dtype):
    lens, bs, Hkv, d = [50, 200], 16, 2, 128
    tbl, N = rand_tables(lens, bs, 1)
    cache = int4_cache(N, Hkv, bs, d, 2, mag, shift)
    q = (wl.normal_tensor((2, 8, d), torch.float32, 4) * qmag).to(dtype)
    check(q, cache, tbl, lens, d ** -0.5, run(q, cache, tbl, lens, d ** -0.5))


def test_a_query_of_zeros_and_a_dominant_key():
    lens, bs, Hkv, d = [70, 70], 16, 1, 64
    tbl, N = rand_tables(lens, bs, 5)
    cache = int4_cache(N, Hkv, bs, d, 6)
    q = wl.normal_tensor((2, 3, d), torch.float16, 7)
    q[0] = 0
    q[1] *= 40
    check(q, cache, tbl, lens, 1.0, run(q, cache, tbl, lens, 1.0))


def test_rows_of_equal_values_are_their_value():
    """s = 0: every code is 0 and the row is its minimum; V constant gives the constant."""
    lens, bs, d = [37], 8, 128
    tbl, N = rand_tables(lens, bs, 3)
    cache = int4_cache(N, 1, bs, d, 1)
    cache[1][:], cache[3][..., 0], cache[3][..., 1] = 0, 0, 0.75
    q = wl.normal_tensor((1, 4, d), torch.float16, 2)
    got = run(q, cache, tbl, lens, d ** -0.5).cpu()
    # weights sum to 1 within 2^-20, then one rounding: 0.75 is a f16 value
    assert (got - 0.75).abs().max() <= 2.0 ** -11 * 0.75


def test_bad_tables_and_lengths_are_flagged_and_read_as_zeros():
    bs, Hkv, d = 16, 2, 64
    lens = [60, 40, 33]
    tbl, N = rand_tables(lens, bs, 9)
    cache = int4_cache(N, Hkv, bs, d, 4)
    q = wl.normal_tensor((3, 4, d), torch.bfloat16, 3)
    bad = tbl.copy()
    bad[0, 1], bad[2, 2] = N, -1
    got = run(q, cache, bad, lens, 0.125)
    assert binding.pa_check_device_errors() == binding.DEVERR["BLOCK_ID"]
    check(q, cache, bad, lens, 0.125, got)
    got = run(q, cache, tbl, [60, -3, 65], 0.125)
    assert binding.pa_check_device_errors() == binding.DEVERR["CONTEXT"] | binding.DEVERR["TABLE_WIDTH"] | (
        binding.DEVERR["BLOCK_ID"] if tbl[2, 3] < 0 else 0)
    check(q, cache, tbl, [60, 0, 64], 0.125, got)


def test_one_workspace_serves_calls_of_different_shapes_and_repeats_agree():
    """Same inputs, same bits; the tickets are back at zero after each call."""
    lens, bs, Hkv, d = [3000, 1, 0, 900], 16, 2, 128
    tbl, N = rand_tables(lens, bs, 2)
    cache = int4_cache(N, Hkv, bs, d, 8)
    q = wl.normal_tensor((4, 16, d), torch.float16, 1)
    ws = workspace(4, 16, d)
    first = run(q, cache, tbl, lens, 0.1, ws).clone()
    small = run(q[:2], cache, tbl[:2], [700, 1], 0.1, ws)
    check(q[:2], cache, tbl[:2], [700, 1], 0.1, small)
    for _ in range(3):
        assert torch.equal(run(q, cache, tbl, lens, 0.1, ws), first)
    check(q, cache, tbl, lens, 0.1, first)
    assert int(ws[: 4 * 16 * 4].view(torch.int32).abs().sum()) == 0


def test_an_understated_maximum_length_changes_nothing():
    """max_context_len only guides the split: a wrong hint may cost time, not results."""
    lens, bs, Hkv, d = [700, 64], 16, 2, 128
    tbl, N = rand_tables(lens, bs, 2)
    cache = int4_cache(N, Hkv, bs, d, 8)
    q = wl.normal_tensor((2, 8, d), torch.bfloat16, 1)
    a = run(q, cache, tbl, lens, 0.1)
    for hint in (0, 64, 1 << 20):
        assert torch.equal(run(q, cache, tbl, lens, 0.1, max_len=hint), a)


def test_two_streams_with_a_workspace_each_and_a_replayed_graph():
    lens, bs, Hkv, d = [900, 33], 16, 4, 128
    tbl, N = rand_tables(lens, bs, 2)
    cache = int4_cache(N, Hkv, bs, d, 8)
    dc, (dt, dl) = dev(*cache), dev(tbl, np.asarray(lens, np.int32))
    qs = [wl.normal_tensor((2, 16, d), torch.bfloat16, s) for s in (1, 2)]
    dq = [x.cuda() for x in qs]
    outs = [torch.empty_like(x) for x in dq]
    wss = [workspace(2, 16, d) for _ in dq]
    streams = [torch.cuda.Stream() for _ in dq]
    torch.cuda.synchronize()
    for _ in range(20):
        for s, x, out, ws in zip(streams, dq, outs, wss):
            binding.pa_decode_int4(x, *dc, dt, dl, 900, 0.1, out, ws, stream=s)
    torch.cuda.synchronize()
    for x, out in zip(qs, outs):
        check(x, cache, tbl, lens, 0.1, out)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        binding.pa_decode_int4(dq[0], *dc, dt, dl, 900, 0.1, outs[0], wss[0])
    dq[0].copy_(qs[1])
    dl.copy_(torch.tensor([33, 500], dtype=torch.int32))
    tbl2 = tbl[::-1].copy()
    dt.copy_(torch.from_numpy(tbl2))
    graph.replay()
    torch.cuda.synchronize()
    assert binding.pa_check_device_errors() == 0
    check(qs[1], cache, tbl2, [33, 500], 0.1, outs[0])


def test_many_short_sequences():
    rng = np.random.default_rng(1)
    lens, bs, Hkv, d = rng.integers(0, 40, 700).tolist(), 8, 1, 64
    tbl, N = rand_tables(lens, bs, 2)
    cache = int4_cache(N, Hkv, bs, d, 8)
    q = wl.normal_tensor((700, 2, d), torch.float16, 1)
    check(q, cache, tbl, lens, 0.125, run(q, cache, tbl, lens, 0.125))


def test_append_decode_and_read_back_into_multi_query():
    """The cache as it is used: a prompt appended, a step decoded over it, then the context read
    back into a 16-bit scratch cache that pa_multi_query reads: both see the same rows."""
    bs, H, Hkv, d, dtype = 16, 8, 2, 128, torch.bfloat16
    lens = [37, 100]
    alloc = binding.Allocator(20, bs)
    for i, n in enumerate(lens):
        alloc.alloc(i, n)
    slots = np.concatenate([alloc.seq_slots(i, 0, n) for i, n in enumerate(lens)])
    T = int(slots.size)
    kn, vn = (wl.normal_tensor((T, Hkv, d), dtype, s) for s in (1, 2))
    host = [np.zeros((20, Hkv, bs, d // 2), np.uint8) for _ in "kv"]
    host += [np.zeros((20, Hkv, bs, 2, 2), np.float16) for _ in "kv"]
    cache = dev(*host)
    binding.pa_reshape_and_cache_int4(kn.cuda(), vn.cuda(), torch.from_numpy(slots).cuda(), *cache)
    o.reshape_and_cache_int4(kn, vn, slots, *host)
    tbl, ln = alloc.export([0, 1], 8)
    q = wl.normal_tensor((2, H, d), dtype, 3)
    check(q, host, tbl, ln, d ** -0.5, run(q, host, tbl, ln, d ** -0.5))
    # the scratch pool: sequence i's blocks in a row
    nb = [-(-n // bs) for n in lens]
    back = np.full(sum(nb) * bs, -1, np.int64)
    at = 0
    stbl = np.zeros((2, max(nb)), np.int32)
    for i, n in enumerate(lens):
        back[at * bs: at * bs + n] = alloc.seq_slots(i, 0, n)
        stbl[i, : nb[i]] = np.arange(at, at + nb[i])
        at += nb[i]
    k16, v16 = (torch.full((sum(nb), bs, Hkv, d), float("nan"), dtype=dtype, device="cuda") for _ in "kv")
    binding.pa_gather_cache_int4(*cache, torch.from_numpy(back).cuda(), k16.view(-1, Hkv, d),
                                 v16.view(-1, Hkv, d))
    ws = torch.zeros(binding.pa_multi_query_workspace_size(2, H, Hkv, d, 1), dtype=torch.uint8, device="cuda")
    out = torch.empty_like(q, device="cuda")
    binding.pa_multi_query(q.cuda(), torch.tensor([0, 1, 2], dtype=torch.int32, device="cuda"), k16, v16,
                           torch.from_numpy(stbl).cuda(), torch.from_numpy(ln).cuda(), 1, d ** -0.5, out, ws)
    assert binding.pa_check_device_errors() == 0
    # the scratch holds the rows' values rounded to bf16: the attention over those
    for i, n in enumerate(lens):
        at = alloc.seq_slots(i, 0, n)
        k, v = (torch.from_numpy(o.gather_int4(c, sm, at)).float().bfloat16().double().numpy()
                for c, sm in ((host[0], host[2]), (host[1], host[3])))
        assert_close(out[i].cpu(), o.softmax_attention(q[i].double().numpy(), k, v, d ** -0.5))


@pytest.mark.parametrize("H,Hkv,d", [(8, 1, 128), (16, 1, 64)])
def test_the_largest_batch(H, Hkv, d):
    """4096 sequences: the list's prefix sums take shared memory from the rings."""
    rng = np.random.default_rng(2)
    lens = np.where(rng.random(4096) < 0.9, 0, rng.integers(1, 90, 4096))
    lens[[0, 4095]] = 130, 77
    bs = 16
    tbl, N = rand_tables(lens, bs, 2)
    cache = int4_cache(N, Hkv, bs, d, 8)
    q = wl.normal_tensor((4096, H, d), torch.bfloat16, 1)
    got = run(q, cache, tbl, lens, 0.1)
    assert binding.pa_check_device_errors() == 0
    check(q, cache, tbl, lens, 0.1, got)


def test_seeded_random_shapes():
    """Groupings, block sizes and length mixes beyond the listed ones."""
    rng = np.random.default_rng(77)
    for _ in range(12):
        G = int(rng.choice([1, 2, 3, 4, 5, 6, 7, 8, 9, 11, 13, 16, 48]))
        Hkv, d, bs = int(rng.integers(1, 5)), int(rng.choice([64, 128])), int(rng.choice([8, 16, 32]))
        B = int(rng.integers(1, 9))
        lens = [int(x) for x in np.exp(rng.uniform(0, np.log(1500), B))]
        lens[int(rng.integers(0, B))] = 0
        dtype = torch.float16 if rng.random() < 0.5 else torch.bfloat16
        tbl, N = rand_tables(lens, bs, G)
        cache = int4_cache(N, Hkv, bs, d, G + d)
        nan_behind(cache, lens, tbl, bs)
        q = wl.normal_tensor((B, Hkv * G, d), dtype, G)
        got = run(q, cache, tbl, lens, d ** -0.5)
        assert binding.pa_check_device_errors() == 0, (G, Hkv, d, bs, lens)
        check(q, cache, tbl, lens, d ** -0.5, got)


@pytest.mark.parametrize("H,Hkv,d,bs,dtype,lens", [
    (16, 1, 128, 16, torch.bfloat16, [9000]),             # more outputs than threads, over 8 CTAs a pair
    (16, 2, 64, 32, torch.float16, [12000, 40]),
    (7, 1, 128, 32, torch.bfloat16, [20000]),
    (4, 1, 64, 8, torch.float16, [30000, 1]),
    (2, 2, 128, 16, torch.float16, [1] * 37 + [6000] + [33] * 50),      # short pairs around a long one
    (12, 4, 128, 16, torch.bfloat16, [40] * 100 + [0] * 20 + [700] * 3),
])
def test_pairs_over_many_ctas_and_many_pairs_in_one(H, Hkv, d, bs, dtype, lens):
    """Shares are cut by cost: a pair's chunks meet every number of CTAs and of joins at the end."""
    tbl, N = rand_tables(lens, bs, 11)
    cache = int4_cache(N, Hkv, bs, d, 12)
    nan_behind(cache, lens, tbl, bs)
    q = wl.normal_tensor((len(lens), H, d), dtype, 13)
    got = run(q, cache, tbl, lens, d ** -0.5)
    assert binding.pa_check_device_errors() == 0
    check(q, cache, tbl, lens, d ** -0.5, got)
