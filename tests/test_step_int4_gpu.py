"""The decode step executor over a 4-bit cache: codes and scales bit for bit as the oracle's after
each step's copy-on-write and append, the output within decode_bound of the oracle's."""
import numpy as np
import pytest
import torch

import oracle
from oracle import cache4 as o
from paged_kv_cache_103_gb300 import binding
from paged_kv_cache_103_gb300 import workloads as wl

from _cache4 import decode_bound, dev, int4_cache

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from paged_kv_cache_103_gb300 import build
    build.build()
    binding.load()


@pytest.mark.parametrize("H,Hkv,d,bs,dtype,depth", [(8, 2, 128, 16, torch.bfloat16, 1),
                                                    (4, 4, 64, 8, torch.float16, 2),
                                                    (14, 2, 128, 32, torch.float16, 2)])
def test_steps_with_copy_on_write(H, Hkv, d, bs, dtype, depth):
    B, N, first = 6, 60, 37
    order = np.random.default_rng(13).permutation(N).astype(np.int32)
    cpp, model = binding.Allocator(N, bs, order), oracle.BlockManagerModel(N, bs, order)
    cpp.alloc(0, first)
    model.allocate(0, first)
    for c in range(1, B):
        cpp.fork(0, c)
        model.fork(0, c)
    cache = int4_cache(N, Hkv, bs, d, 3)
    dc = dev(*cache)
    mb, scale = -(-(first + 4) // bs), 0.09
    step = binding.Step(cpp, B, H, Hkv, d, mb, mb * bs, dc[0], dc[1], scale, k_scale=dc[2], v_scale=dc[3],
                        dtype=dtype, depth=depth, kv_format="int4")
    ids = [4, 1, 0, 5, 3, 2]
    for k in range(3):
        xs = [wl.normal_tensor(shape, dtype, 10 * k + j)
              for j, shape in enumerate([(B, H, d), (B, Hkv, d), (B, Hkv, d)])]
        slot = step.slot(k % depth)
        for name, x in zip(("q", "k_new", "v_new"), xs):
            slot[name].copy_(x)
        step.wait(step.submit(ids))
        assert binding.pa_check_device_errors() == 0
        slots, pairs = model.append_batch(ids)
        if k == 0:
            assert len(pairs) == (B - 1 if first % bs else 0)
        for s, t in pairs:
            for a in cache:
                a[t] = a[s]
        o.reshape_and_cache_int4(xs[1], xs[2], slots, *cache)
        for got, want in zip(dc, cache):
            assert np.array_equal(got.cpu().numpy().view(np.uint8), want.view(np.uint8))
        tbl, lens = model.export(ids, mb)
        q = xs[0].double().numpy()
        ref = o.decode_int4(q, *cache, tbl, lens, scale)
        err = np.abs(slot["out"].double().numpy() - ref)
        assert (err <= decode_bound(q, cache, tbl, lens, scale, dtype, ref)).all()
    step.close()


def test_blocks_swap_to_the_host_and_back():
    """pa_swap_blocks moves a 4-bit cache's codes and scales as pools of their own block sizes."""
    N, Hkv, bs, d = 9, 3, 16, 128
    cache = int4_cache(N, Hkv, bs, d, 5)
    dc = dev(*cache)
    host = [torch.zeros((4,) + a.shape[1:], dtype=t.dtype).pin_memory() for a, t in zip(cache, dc)]
    out = torch.tensor([[2, 0], [7, 3]], dtype=torch.int32, device="cuda")
    back = torch.tensor([[0, 5], [3, 1]], dtype=torch.int32, device="cuda")
    for t, h in zip(dc, host):
        binding.pa_swap_blocks([t], [h], out)
        binding.pa_swap_blocks([h], [t], back)
    assert binding.pa_check_device_errors() == 0
    for a, t in zip(cache, dc):
        a[5], a[1] = a[2], a[7]
        assert np.array_equal(t.cpu().numpy().view(np.uint8), a.view(np.uint8))
