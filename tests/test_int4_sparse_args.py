"""Refusals of the 4-bit-cache and block-sparse entry points, without a GPU: the C ABI's host
checks answer before any pointer is used, the binding's before the library is called."""
import ctypes

import pytest
import torch

from paged_kv_cache_103_gb300 import binding
from paged_kv_cache_103_gb300 import build as pa_build

P = ctypes.c_void_p(16 * 1024)      # aligned, never dereferenced
ODD = ctypes.c_void_p(16 * 1024 + 4)
OK, INVALID, UNSUPPORTED = 0, 1, 6


@pytest.fixture(scope="module")
def lib():
    pa_build.build()
    return binding.load()


def _append(lib, T=1, N=8, bs=16, Hkv=2, d=64, dt=0, k=P, kc=P, ks=P):
    return lib.pa_reshape_and_cache_int4(k, P, P, T, kc, P, ks, P, N, bs, Hkv, d, dt, None)


def test_append(lib):
    assert _append(lib, T=0) == OK and _append(lib, T=0, k=None) == OK
    assert _append(lib, T=-1) == INVALID and _append(lib, Hkv=0) == INVALID
    assert _append(lib, k=None) == INVALID and _append(lib, k=ODD) == INVALID
    assert _append(lib, kc=ODD) == INVALID and _append(lib, ks=ctypes.c_void_p(16386)) == INVALID
    for bad in (dict(dt=2), dict(d=96), dict(d=256), dict(bs=4), dict(bs=24), dict(bs=64)):
        assert _append(lib, **bad) == UNSUPPORTED, bad


def test_read_back(lib):
    def read(name, T=1, bs=16, d=128, dt=0, out=P):
        return getattr(lib, name)(P, P, P, P, P, T, out, P, 8, bs, 2, d, dt, None)
    for name in ("pa_gather_cache_int4", "pa_gather_cache_int8", "pa_gather_cache_fp8"):
        assert read(name, T=0) == OK
        assert read(name, T=-1) == INVALID and read(name, out=None) == INVALID
        assert read(name, out=ODD) == INVALID
        assert read(name, bs=7) == UNSUPPORTED and read(name, dt=9) == UNSUPPORTED
        assert read(name, d=96) == UNSUPPORTED
    assert read("pa_gather_cache_int8", d=64) == UNSUPPORTED


def test_decode_int4(lib):
    def call(B=2, H=4, Hkv=2, d=128, bs=16, N=8, mb=4, n=64, dt=0, ws=1 << 24, scale=0.1, q=P, kc=P, out=P):
        return lib.pa_decode_int4(q, kc, P, P, P, P, mb, P, n, B, H, Hkv, d, bs, N, scale, dt, out, P, ws, None)
    assert call(B=0) == OK
    for bad in (dict(B=-1), dict(H=0), dict(mb=0), dict(N=0), dict(n=-1), dict(scale=float("nan")),
                dict(ws=64), dict(q=None), dict(q=ODD), dict(kc=ODD), dict(out=ODD), dict(out=None)):
        assert call(**bad) == INVALID, bad
    for bad in (dict(H=5), dict(H=34), dict(d=96), dict(bs=64), dict(dt=2), dict(B=4097, ws=1 << 28),
                dict(mb=1 << 27, N=1 << 20)):
        assert call(**bad) == UNSUPPORTED, bad


def test_summaries(lib):
    def call(n=1, N=8, bs=16, Hkv=2, d=64, dt=0, k=P, boxes=P):
        return lib.pa_summarize_blocks(k, P, None, n, boxes, P, N, bs, Hkv, d, dt, None)
    assert call(n=0) == OK
    assert call(n=-1) == INVALID and call(k=None) == INVALID and call(k=ODD) == INVALID and call(boxes=ODD) == INVALID
    for bad in (dict(d=32), dict(bs=12), dict(dt=3)):
        assert call(**bad) == UNSUPPORTED, bad


def test_selection(lib):
    def call(B=2, H=4, Hkv=2, d=64, bs=16, N=8, keep=4, first=1, last=1, mb=4, dt=0, ws=1 << 20, q=P, sel=P):
        return lib.pa_select_blocks(q, P, P, P, mb, P, B, H, Hkv, d, bs, N, keep, first, last, dt, sel, P, P, ws,
                                    None)
    assert call(B=0) == OK
    for bad in (dict(first=-1), dict(last=0), dict(keep=1), dict(first=3, last=2), dict(mb=0), dict(ws=8),
                dict(q=None), dict(q=ODD), dict(sel=None), dict(keep=0)):
        assert call(**bad) == INVALID, bad
    for bad in (dict(H=5), dict(H=2 * 129), dict(d=96), dict(bs=9), dict(dt=2), dict(B=4097, ws=1 << 28)):
        assert call(**bad) == UNSUPPORTED, bad
    assert lib.pa_select_blocks_workspace_size(2, 4, 100) >= 2 * 4 * 100 * 4
    assert lib.pa_select_blocks_workspace_size(2, 0, 100) == 0


def test_decode_selected(lib):
    def call(B=2, H=4, Hkv=2, d=64, bs=16, N=8, keep=4, n=64, dt=0, ws=1 << 24, k=P):
        return lib.pa_decode_selected(P, k, P, P, keep, P, n, B, H, Hkv, d, bs, N, 0.1, dt, P, P, ws, None)
    assert call(B=0) == OK
    assert call(keep=0) == INVALID and call(ws=16) == INVALID and call(k=ODD) == INVALID and call(B=-1) == INVALID
    for bad in (dict(H=5), dict(B=4096, ws=1 << 28), dict(d=96), dict(bs=64), dict(dt=2)):
        assert call(**bad) == UNSUPPORTED, bad


def test_binding_refuses_tensors_that_do_not_fit():
    """Shapes are checked before any pointer is taken, so host tensors show it."""
    N, Hkv, bs, d, T = 4, 2, 8, 64, 3
    x = torch.zeros(T, Hkv, d, dtype=torch.float16)
    c, s = torch.zeros(N, Hkv, bs, d // 2, dtype=torch.uint8), torch.zeros(N, Hkv, bs, 1, 2, dtype=torch.float16)
    slots = torch.zeros(T, dtype=torch.int64)
    for args in ((x, x[:2], slots, c, c, s, s), (x, x, slots[:2], c, c, s, s), (x, x, slots, c, c[:3], s, s),
                 (x, x, slots, c.transpose(1, 2), c, s, s), (x, x, slots, c, c, s[..., :1], s),
                 (x, x, slots, c, c, s[:, :1], s)):
        with pytest.raises(ValueError):
            binding.pa_reshape_and_cache_int4(*args)
        with pytest.raises(ValueError):
            binding.pa_gather_cache_int4(*args[3:], args[2], args[0], args[1])
    q = torch.zeros(2, 4, d, dtype=torch.float16)
    tbl, ln = torch.zeros(2, 3, dtype=torch.int32), torch.zeros(2, dtype=torch.int32)
    for bad in (dict(t=tbl[:1]), dict(n=ln[:1]), dict(out=q[:1]), dict(c=c[:, :, :, :16])):
        with pytest.raises(ValueError):
            cc = bad.get("c", c)
            binding.pa_decode_int4(q, cc, cc, s, s, bad.get("t", tbl), bad.get("n", ln), 8, 0.1,
                                   bad.get("out", q), torch.zeros(8))
    k = torch.zeros(N, bs, Hkv, d, dtype=torch.float16)
    box, S = torch.zeros(N, Hkv, 2, d, dtype=torch.int8), torch.zeros(N, Hkv)
    ids = torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError):
        binding.pa_summarize_blocks(k, ids, box[:, :1], S)
    with pytest.raises(ValueError):
        binding.pa_summarize_blocks(k, ids, box, S[:2])
    sel, n = torch.zeros(2, Hkv, 3, dtype=torch.int32), torch.zeros(2, Hkv, dtype=torch.int32)
    with pytest.raises(ValueError):
        binding.pa_select_blocks(q, box, S, tbl, ln, bs, 0, 1, sel[:, :1], n, torch.zeros(8))
    with pytest.raises(ValueError):
        binding.pa_decode_selected(q, k, k[:3], sel, n, 8, 0.1, q, torch.zeros(8))
    with pytest.raises(ValueError):
        binding.pa_decode_selected(q, k, k, sel, n[:1], 8, 0.1, q, torch.zeros(8))


def test_step_executor_takes_a_4_bit_cache(lib):
    L = binding.StepLayout()

    def layout(q8, d):
        desc = binding.StepDesc(4, 8, 2, d, 16, 32, 8, 128, 0, 0.088, q8, 1)
        return lib.pa_step_layout_get(ctypes.byref(desc), ctypes.byref(L))
    assert layout(4, 64) == OK and layout(4, 128) == OK
    assert layout(3, 128) == INVALID and layout(5, 128) == INVALID and layout(1, 64) == INVALID
    N, bs, Hkv, d = 8, 16, 2, 128
    c = torch.zeros(N, Hkv, bs, d // 2, dtype=torch.uint8)
    s = torch.zeros(N, Hkv, bs, 2, 2, dtype=torch.float16)
    alloc = binding.Allocator(N, bs)
    for bad in (dict(k_cache=c.transpose(1, 2)), dict(v_cache=c[:4]), dict(k_scale=s.float()), dict(v_scale=s[:, :1]),
                dict(k_scale=None), dict(dtype=torch.float32), dict(k_cache=c.to(torch.int8), v_cache=c.to(torch.int8))):
        kw = dict(dict(k_cache=c, v_cache=c, k_scale=s, v_scale=s, dtype=torch.float16), **bad)
        with pytest.raises(ValueError):
            binding.Step(alloc, 2, 4, Hkv, d, 4, 64, scale=0.1, kv_format="int4", **kw)


def test_workspaces_that_would_fault(lib):
    """Partial results are stored 16 bytes at a time, so a workspace between two such places is refused."""
    for ws, want in ((ODD, INVALID), (ctypes.c_void_p(16 * 1024 + 8), INVALID), (None, INVALID)):
        assert lib.pa_decode_int4(P, P, P, P, P, P, 4, P, 64, 2, 4, 2, 128, 16, 8, 0.1, 0, P, ws, 1 << 24,
                                  None) == want
        assert lib.pa_decode_selected(P, P, P, P, 4, P, 64, 2, 4, 2, 128, 16, 8, 0.1, 0, P, ws, 1 << 24,
                                      None) == want


def test_selection_refuses_more_kv_heads_than_a_grid_has_rows(lib):
    assert lib.pa_select_blocks(P, P, P, P, 4, P, 1, 1 << 17, 1 << 17, 64, 16, 8, 2, 0, 1, 0, P, P, P, 1 << 30,
                                None) == UNSUPPORTED
