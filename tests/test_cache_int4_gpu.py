"""The 4-bit append and the read back of the quantised caches on the GPU, bit for bit against
the oracle."""
import numpy as np
import pytest
import torch

import oracle
from oracle import cache4 as o
from paged_kv_cache_103_gb300 import binding
from paged_kv_cache_103_gb300 import workloads as wl

from _cache4 import dev

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from paged_kv_cache_103_gb300 import build
    build.build()
    binding.load()


def _empty(N, Hkv, bs, d):
    c = [np.full((N, Hkv, bs, d // 2), 0x5A, np.uint8) for _ in "kv"]
    s = [np.full((N, Hkv, bs, d // 64, 2), 7, np.float16) for _ in "kv"]
    return c + s


def _rows(T, Hkv, d, dtype, seed):
    x = wl.normal_tensor((T, Hkv, d), torch.float32, seed)
    x = x * (1 + 9 * (torch.arange(d) % 17 == 3)) + 3 * (torch.arange(d) % 23 == 5)
    f = x.view(-1, d)
    specials = [0.0, 1.5, -65504.0, 2.0 ** -24, -2.0 ** -20]
    for r, v in enumerate(specials):                  # constant rows
        if r < f.shape[0]:
            f[r] = v
    if f.shape[0] > 7:
        f[5, 0], f[5, 1] = 65504.0, -65504.0          # the widest f16 row
        f[6] = torch.arange(d) % 16                   # codes 0 .. 15
        f[7] = (torch.arange(d) % 31) / 2             # ties
    if dtype == torch.bfloat16 and f.shape[0] > 9:
        f[8, 3] = 3e38                                # beyond f16: saturates
        f[9, 0], f[9, 1] = -1e6, 2e5
    return x.to(dtype)


@pytest.mark.parametrize("T,N,bs,Hkv,d,dtype", [
    (1, 1, 8, 1, 64, torch.float16), (1, 3, 32, 1, 128, torch.bfloat16),
    (4, 64, 16, 2, 64, torch.bfloat16), (5, 9, 16, 3, 128, torch.float16),
    (77, 50, 32, 40, 128, torch.float16), (256, 400, 16, 4, 128, torch.bfloat16),
    (1000, 3000, 8, 5, 64, torch.float16), (1023, 2050, 8, 8, 128, torch.bfloat16)])
def test_append_and_read_back_bit_exact(T, N, bs, Hkv, d, dtype):
    rng = np.random.default_rng(T)
    slots = rng.choice(N * bs, size=T, replace=False).astype(np.int64)
    slots[3::7] = -1
    kn, vn = _rows(T, Hkv, d, dtype, 5), _rows(T, Hkv, d, dtype, 6)
    host = _empty(N, Hkv, bs, d)
    cache = dev(*host)
    ds = torch.from_numpy(slots).cuda()
    binding.pa_reshape_and_cache_int4(kn.cuda(), vn.cuda(), ds, *cache)
    o.reshape_and_cache_int4(kn, vn, slots, *host)
    for got, want in zip(cache, host):
        assert np.array_equal(got.cpu().numpy().view(np.uint8), want.view(np.uint8))
    # read back, in another order, some slots twice
    order = rng.integers(0, T, size=T + 3)
    back = slots[order]
    for out_dtype in (torch.float16, torch.bfloat16):
        ko, vo = (torch.full((T + 3, Hkv, d), 0.5, dtype=out_dtype, device="cuda") for _ in "kv")
        binding.pa_gather_cache_int4(*cache, torch.from_numpy(back).cuda(), ko, vo)
        assert binding.pa_check_device_errors() == 0
        live = back >= 0
        for out, codes, scale in ((ko, host[0], host[2]), (vo, host[1], host[3])):
            want = torch.full(out.shape, 0.5, dtype=out_dtype)
            val = o.gather_int4(codes, scale, back[live]).astype(np.float32)
            want[torch.from_numpy(live)] = torch.from_numpy(val).to(out_dtype)
            assert torch.equal(out.cpu().view(torch.int16), want.view(torch.int16))


@pytest.mark.parametrize("fmt", ["int8", "fp8"])
@pytest.mark.parametrize("T,bs,Hkv,dtype", [(1, 8, 1, torch.float16), (77, 16, 3, torch.bfloat16),
                                            (1001, 32, 4, torch.float16)])
def test_read_back_of_8_bit_caches_bit_exact(fmt, T, bs, Hkv, dtype):
    d, N = 128, (T + 40) // bs + 3
    rng = np.random.default_rng(T + bs)
    slots = rng.choice(N * bs, size=T, replace=False).astype(np.int64)
    slots[2::9] = -1
    kc, vc = (np.zeros((N, bs, Hkv, d), np.uint8) for _ in "kv")
    ks, vs = (np.zeros((N, Hkv, bs), np.float32) for _ in "kv")
    put = oracle.reshape_and_cache_int8 if fmt == "int8" else oracle.reshape_and_cache_fp8
    put(_rows(T, Hkv, d, dtype, 1), _rows(T, Hkv, d, dtype, 2), slots, kc, vc, ks, vs)
    ko, vo = (torch.full((T, Hkv, d), 0.25, dtype=dtype, device="cuda") for _ in "kv")
    read = binding.pa_gather_cache_int8 if fmt == "int8" else binding.pa_gather_cache_fp8
    read(*dev(kc, vc, ks, vs), torch.from_numpy(slots).cuda(), ko, vo)
    assert binding.pa_check_device_errors() == 0
    live = slots >= 0
    b, r = slots[live] // bs, slots[live] % bs
    for out, c, s in ((ko, kc, ks), (vo, vc, vs)):
        val = (c[b, r].view(np.int8).astype(np.float32) if fmt == "int8"
               else oracle.e4m3_to_double(c[b, r]).astype(np.float32)) * s[b, :, r][..., None]
        want = torch.full(out.shape, 0.25, dtype=dtype)
        want[torch.from_numpy(live)] = torch.from_numpy(val).to(dtype)
        assert torch.equal(out.cpu().view(torch.int16), want.view(torch.int16))


def test_slots_outside_the_pool_are_flagged_and_left():
    N, bs, Hkv, d = 4, 8, 2, 64
    host = _empty(N, Hkv, bs, d)
    cache = dev(*host)
    kn = _rows(3, Hkv, d, torch.float16, 4)
    slots = torch.tensor([N * bs, 3, 1 << 40], device="cuda")
    binding.pa_reshape_and_cache_int4(kn.cuda(), kn.cuda(), slots, *cache)
    assert binding.pa_check_device_errors() == binding.DEVERR["SLOT"]
    o.reshape_and_cache_int4(kn, kn, [-1, 3, -1], *host)
    for got, want in zip(cache, host):
        assert np.array_equal(got.cpu().numpy().view(np.uint8), want.view(np.uint8))
    out = [torch.full((3, Hkv, d), 2.0, dtype=torch.float16, device="cuda") for _ in "kv"]
    binding.pa_gather_cache_int4(*cache, slots, *out)
    assert binding.pa_check_device_errors() == binding.DEVERR["SLOT"]
    for x in out:
        assert (x[0] == 2).all() and (x[2] == 2).all() and not (x[1] == 2).all()


def test_slots_beyond_32_bits_of_code_bytes():
    """A pool whose codes pass 4 GiB: the last block is written and read back."""
    Hkv, bs, d = 8, 32, 128
    N = (1 << 32) // (Hkv * bs * d // 2) + 2
    if torch.cuda.mem_get_info()[0] < 14 << 30:
        pytest.skip("needs 14 GB")
    cache = [torch.zeros(N, Hkv, bs, d // 2, dtype=torch.uint8, device="cuda") for _ in "kv"]
    cache += [torch.zeros(N, Hkv, bs, 2, 2, dtype=torch.float16, device="cuda") for _ in "kv"]
    kn, vn = _rows(2, Hkv, d, torch.bfloat16, 9) + 1, _rows(2, Hkv, d, torch.bfloat16, 10)
    slots = torch.tensor([N * bs - 1, 5], device="cuda")
    binding.pa_reshape_and_cache_int4(kn.cuda(), vn.cuda(), slots, *cache)
    out = [torch.zeros(2, Hkv, d, dtype=torch.bfloat16, device="cuda") for _ in "kv"]
    binding.pa_gather_cache_int4(*cache, slots, *out)
    assert binding.pa_check_device_errors() == 0
    for new, got in ((kn, out[0]), (vn, out[1])):
        want = torch.from_numpy(o.int4_values(*o.quantize_rows_int4(new.float().numpy())).astype(np.float32))
        assert torch.equal(got.cpu(), want.bfloat16())


def test_on_a_side_stream_and_in_a_graph():
    T, N, bs, Hkv, d = 40, 12, 16, 4, 128
    slots_h = np.random.default_rng(0).permutation(N * bs)[:T].astype(np.int64)
    slots = torch.from_numpy(slots_h).cuda()
    kn, vn = (torch.empty(T, Hkv, d, dtype=torch.bfloat16, device="cuda") for _ in "kv")
    cache = dev(*_empty(N, Hkv, bs, d))
    out = [torch.empty_like(kn) for _ in "kv"]
    binding.load()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        binding.pa_reshape_and_cache_int4(kn, vn, slots, *cache)
        binding.pa_gather_cache_int4(*cache, slots, *out)
    for seed in (1, 2):
        k, v = _rows(T, Hkv, d, torch.bfloat16, seed), _rows(T, Hkv, d, torch.bfloat16, seed + 5)
        kn.copy_(k)
        vn.copy_(v)
        graph.replay()
        assert binding.pa_check_device_errors() == 0
        for new, got in ((k, out[0]), (v, out[1])):
            want = o.int4_values(*o.quantize_rows_int4(new.float().numpy())).astype(np.float32)
            assert torch.equal(got.cpu(), torch.from_numpy(want).bfloat16())
