"""The decode step executor over a block-scaled 8-bit cache: codes and scales bit for bit as the
oracle's after each step's copy-on-write and append, the output within decode_bound of the oracle's."""
import ctypes

import numpy as np
import pytest
import torch

import oracle
from oracle import block8 as o
from paged_kv_cache_103_gb300 import binding
from paged_kv_cache_103_gb300 import build as pa_build
from paged_kv_cache_103_gb300 import workloads as wl

from _block8 import FMTS, cache, decode_bound
from _cache4 import dev


def test_descriptions():
    pa_build.build()
    lib, L = binding.load(), binding.StepLayout()

    def layout(q8, d, Hkv):
        desc = binding.StepDesc(4, 8, Hkv, d, 16, 32, 8, 128, 0, 0.088, q8, 1)
        return lib.pa_step_layout_get(ctypes.byref(desc), ctypes.byref(L))
    for q8 in (17, 18):
        assert layout(q8, 64, 4) == layout(q8, 128, 8) == 0
        assert layout(q8, 128, 2) == 1 and layout(q8, 96, 4) == 1      # scales of a block: 16 bytes at a time
    assert layout(16, 128, 4) == layout(19, 128, 4) == 1
    N, bs, Hkv, d = 8, 16, 4, 128
    c, s = torch.zeros(N, Hkv, bs, d, dtype=torch.uint8), torch.zeros(N, Hkv)
    alloc = binding.Allocator(N, bs)
    for bad in (dict(k_cache=c.transpose(1, 2)), dict(v_cache=c[:4]), dict(k_scale=s.half()), dict(v_scale=s[:, :1]),
                dict(k_scale=None), dict(dtype=torch.float32), dict(k_cache=c.to(torch.int8), v_cache=c.to(torch.int8))):
        kw = dict(dict(k_cache=c, v_cache=c, k_scale=s, v_scale=s, dtype=torch.float16), **bad)
        with pytest.raises(ValueError):
            binding.Step(alloc, 2, 4, Hkv, d, 4, 64, scale=0.1, kv_format="int8_block", **kw)


@pytest.mark.gpu
@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("H,Hkv,d,bs,dtype,depth", [(8, 4, 128, 16, torch.bfloat16, 1), (4, 4, 64, 8, torch.float16, 2),
                                                    (56, 8, 128, 32, torch.float16, 2)])
def test_steps_with_copy_on_write(fmt, H, Hkv, d, bs, dtype, depth):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    B, N, first = 6, 60, 37
    order = np.random.default_rng(13).permutation(N).astype(np.int32)
    cpp, model = binding.Allocator(N, bs, order), oracle.BlockManagerModel(N, bs, order)
    cpp.alloc(0, first)
    model.allocate(0, first)
    for c in range(1, B):
        cpp.fork(0, c)
        model.fork(0, c)
    host = cache(N, Hkv, bs, d, fmt, 3)
    dc = dev(*host)
    mb, scale = -(-(first + 4) // bs), 0.09
    step = binding.Step(cpp, B, H, Hkv, d, mb, mb * bs, dc[0], dc[1], scale, k_scale=dc[2], v_scale=dc[3],
                        dtype=dtype, depth=depth, kv_format=fmt + "_block")
    ids = [4, 1, 0, 5, 3, 2]
    for k in range(3):
        xs = [wl.normal_tensor(shape, dtype, 10 * k + j) * (1 + k)
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
            for a in host:
                a[t] = a[s]
        o.append(xs[1].float().numpy(), slots, host[0], host[2], fmt)
        o.append(xs[2].float().numpy(), slots, host[1], host[3], fmt)
        for got, want in zip(dc, host):
            assert np.array_equal(got.cpu().numpy().view(np.uint8), want.view(np.uint8))
        tbl, lens = model.export(ids, mb)
        q = xs[0].double().numpy()
        ref = o.decode(q, *host, tbl, lens, scale, fmt)
        err = np.abs(slot["out"].double().numpy() - ref)
        assert (err <= decode_bound(q, host, tbl, lens, scale, dtype, ref, fmt)).all()
    step.close()
