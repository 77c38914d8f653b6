"""The forms that only large calls take: four pieces a thread in the read back, reads and writes cut
into launches, the scoring kernel's largest tile, addresses beyond 32 bits."""
import numpy as np
import pytest
import torch

import oracle
from oracle import cache4 as o
from paged_kv_cache_103_gb300 import binding
from paged_kv_cache_103_gb300 import workloads as wl

from _cache4 import decode_bound, dev, int4_cache, workspace

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from paged_kv_cache_103_gb300 import build
    build.build()
    binding.load()


def room(gigabytes):
    if torch.cuda.mem_get_info()[0] < gigabytes << 30:
        pytest.skip("needs %d GB" % gigabytes)


def pool(fmt, N, Hkv, bs, d, seed):
    """Host caches of random rows and the fp32 values [N * bs, Hkv, d] that they stand for."""
    if fmt == "int4":
        c = int4_cache(N, Hkv, bs, d, seed)
        at = np.arange(N * bs)
        return c, [o.gather_int4(c[i], c[i + 2], at).astype(np.float32) for i in range(2)]
    T = N * bs
    rng = np.random.default_rng(seed)
    codes = [rng.integers(0, 256, (N, bs, Hkv, d)).astype(np.uint8) for _ in "kv"]
    if fmt == "fp8":
        for c in codes:
            c[(c & 127) == 127] = 0                   # not a number
    scales = [rng.uniform(0.001, 2, (N, Hkv, bs)).astype(np.float32) for _ in "kv"]
    vals = []
    for c, s in zip(codes, scales):
        wide = c.view(np.int8).astype(np.float32) if fmt == "int8" else oracle.e4m3_to_double(c).astype(np.float32)
        vals.append((wide * s.transpose(0, 2, 1)[..., None]).reshape(T, Hkv, d))
    return codes + scales, vals


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("fmt,d", [("int4", 64), ("int4", 128), ("int8", 128), ("fp8", 128)])
@pytest.mark.parametrize("extra", [0, 1, 37])
def test_large_read_back(fmt, d, dtype, extra):
    """Four pieces of 8 values a thread: taken from 4 x 2048 pieces an SM on, 152 SMs at most; with
    extra tokens the last CTA is ragged.  Padding and slots outside the pool among them."""
    Hkv, bs, N = 5, 16, 300
    T = -(-4 * 2048 * 152 // (Hkv * d // 8)) + extra
    host, vals = pool(fmt, N, Hkv, bs, d, T)
    rng = np.random.default_rng(T)
    slots = rng.integers(0, N * bs, T)
    slots[rng.integers(0, T, T // 9)] = -1
    slots[-1] = 3
    bad = rng.integers(0, T - 1, 40)
    slots[bad[:20]], slots[bad[20:]] = N * bs, 1 << 40
    ko, vo = (torch.full((T, Hkv, d), 0.25, dtype=dtype, device="cuda") for _ in "kv")
    read = dict(int4=binding.pa_gather_cache_int4, int8=binding.pa_gather_cache_int8,
                fp8=binding.pa_gather_cache_fp8)[fmt]
    read(*dev(*host), torch.from_numpy(slots).cuda(), ko, vo)
    assert binding.pa_check_device_errors() == binding.DEVERR["SLOT"]
    live = torch.from_numpy((slots >= 0) & (slots < N * bs)).cuda()
    at = torch.from_numpy(np.where((slots >= 0) & (slots < N * bs), slots, 0)).cuda()
    for got, val in zip((ko, vo), vals):
        want = torch.from_numpy(val).to(dtype).cuda()[at]
        want[~live] = 0.25
        assert torch.equal(got.view(torch.int16), want.view(torch.int16))


def test_reads_and_writes_beyond_one_launch():
    """A launch takes 2^30 pieces of 8 values at most: here 2^30 and a few tokens more."""
    room(90)
    Hkv, bs, d, N, dtype = 4096, 8, 64, 20, torch.bfloat16
    per = (1 << 30) // (Hkv * d // 8)                  # tokens of a launch
    T = per + 3
    rng = np.random.default_rng(1)
    x = torch.randn(2, 64, Hkv, d, generator=torch.Generator().manual_seed(2)).to(dtype)
    new = [torch.zeros(T, Hkv, d, dtype=dtype, device="cuda") for _ in "kv"]
    slots = np.full(T, -1, np.int64)
    where = np.concatenate([rng.permutation(per - 2)[:60], [per - 2, per - 1, per, per + 2]])   # both sides
    slots[where] = rng.permutation(N * bs)[:64]
    for n, y in zip(new, x):
        n[torch.from_numpy(where).cuda()] = y.cuda()
    host = [np.zeros((N, Hkv, bs, d // 2), np.uint8) for _ in "kv"]
    host += [np.zeros((N, Hkv, bs, 1, 2), np.float16) for _ in "kv"]
    cache = dev(*host)
    ds = torch.from_numpy(slots).cuda()
    binding.pa_reshape_and_cache_int4(*new, ds, *cache)
    o.reshape_and_cache_int4(x[0], x[1], slots[where], *host)
    for got, want in zip(cache, host):
        assert np.array_equal(got.cpu().numpy().view(np.uint8), want.view(np.uint8))
    out = new                                          # read back into the rows themselves
    for n in out:
        n.fill_(0.5)
    binding.pa_gather_cache_int4(*cache, ds, *out)
    assert binding.pa_check_device_errors() == 0
    for got, c, s in zip(out, host[:2], host[2:]):
        want = torch.from_numpy(o.gather_int4(c, s, slots[where]).astype(np.float32)).to(dtype)
        assert torch.equal(got[torch.from_numpy(where).cuda()].cpu(), want)
        got[torch.from_numpy(where).cuda()] = 0.5
        assert all(bool((part == 0.5).all()) for part in got.split(1 << 10))


@pytest.mark.parametrize("Hkv,G,d", [(8, 4, 128), (40, 1, 128), (3, 2, 64), (1, 128, 128)])
def test_the_scoring_kernels_largest_tile(Hkv, G, d):
    """A table so wide that a scoring CTA takes as many blocks as it may, some 2048; contexts that end
    inside, at and behind a tile, with the scores' ties."""
    bs, B, W, keep = 8, 96, 8192, 6
    rng = np.random.default_rng(Hkv)
    N = 5000
    lens = np.minimum(rng.integers(0, W * bs, B), rng.integers(0, 40000, B)).astype(np.int64)
    lens[:6] = [0, 2048 * bs, 2048 * bs + bs * 2, 2050 * bs + 1, W * bs, 9]
    tbl = rng.integers(0, N, (B, W)).astype(np.int32)
    hb = rng.integers(-127, 128, (N, Hkv, 2, d)).astype(np.int8)
    hb[:, :, 0] = np.minimum(hb[:, :, 0], hb[:, :, 1])
    hs = rng.uniform(0, 1, (N, Hkv)).astype(np.float32)
    q = wl.normal_tensor((B, Hkv * G, d), torch.float16, 3)
    sel = torch.full((B, Hkv, keep), 77, dtype=torch.int32, device="cuda")
    n = torch.full((B, Hkv), 77, dtype=torch.int32, device="cuda")
    ws = torch.empty(binding.pa_select_blocks_workspace_size(B, Hkv, W), dtype=torch.uint8, device="cuda")
    binding.pa_select_blocks(q.cuda(), *dev(hb, hs, tbl, lens.astype(np.int32)), bs, 1, 2, sel, n, ws)
    assert binding.pa_check_device_errors() == 0
    some = [0, 1, 2, 3, 4, 5] + rng.integers(6, B, 4).tolist()
    want, wn = o.select_blocks(q[some].float().numpy(), hb, hs, tbl[some], lens[some], bs, keep, 1, 2)
    assert np.array_equal(n.cpu().numpy()[some], wn)
    assert np.array_equal(sel.cpu().numpy()[some], want)


def test_decode_beyond_32_bits_of_code_bytes():
    """Blocks at both ends of a pool whose codes pass 4 GiB."""
    room(14)
    Hkv, bs, d = 8, 32, 128
    N = (1 << 32) // (Hkv * bs * d // 2) + 2
    small = int4_cache(3, Hkv, bs, d, 4)
    cache = [torch.zeros(N, *a.shape[1:], dtype=t.dtype, device="cuda") for a, t in zip(small, dev(*small))]
    where = [N - 1, 2, N - 2]
    for c, a in zip(cache, small):
        c[torch.tensor(where).cuda()] = torch.from_numpy(a).cuda()
    lens = [90, 40]
    tbl, stbl = np.array([where, [N - 1, N - 2, -1]], np.int32), np.array([[0, 1, 2], [0, 2, -1]], np.int32)
    q = wl.normal_tensor((2, 32, d), torch.bfloat16, 3)
    out = torch.empty_like(q, device="cuda")
    binding.pa_decode_int4(q.cuda(), *cache, *dev(tbl, np.array(lens, np.int32)), 96, d ** -0.5, out, workspace(2, 32, d))
    assert binding.pa_check_device_errors() == 0
    ref = o.decode_int4(q.double().numpy(), *small, stbl, lens, d ** -0.5)
    err = np.abs(out.cpu().double().numpy() - ref)
    assert (err <= decode_bound(q.double().numpy(), small, stbl, lens, d ** -0.5, q.dtype, ref)).all()
