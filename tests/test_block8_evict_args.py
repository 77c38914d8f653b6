"""Refusals of the block-scaled 8-bit cache's and of the eviction's entry points, without a GPU: the
C ABI's host checks answer before any pointer is used, the binding's before the library is called."""
import ctypes

import pytest
import torch

from paged_kv_cache_103_gb300 import binding
from paged_kv_cache_103_gb300 import build as pa_build

P = ctypes.c_void_p(16 * 1024)      # aligned, never dereferenced
ODD = ctypes.c_void_p(16 * 1024 + 4)
ODD2 = ctypes.c_void_p(16 * 1024 + 2)
OK, INVALID, UNSUPPORTED = 0, 1, 6


@pytest.fixture(scope="module")
def lib():
    pa_build.build()
    return binding.load()


@pytest.mark.parametrize("fmt", ["int8", "fp8"])
def test_append(lib, fmt):
    def call(T=1, N=8, bs=16, Hkv=2, d=64, dt=0, k=P, kc=P, ks=P, slots=P):
        return getattr(lib, "pa_reshape_and_cache_%s_block" % fmt)(k, P, slots, T, kc, P, ks, P, N, bs, Hkv, d, dt, None)
    assert call(T=0) == OK and call(T=0, k=None) == OK
    for bad in (dict(T=-1), dict(Hkv=0), dict(k=None), dict(k=ODD), dict(kc=ODD), dict(ks=ODD2), dict(slots=ODD)):
        assert call(**bad) == INVALID, bad
    for bad in (dict(dt=2), dict(d=96), dict(d=256), dict(bs=4), dict(bs=24), dict(bs=64), dict(Hkv=1 << 21)):
        assert call(**bad) == UNSUPPORTED, bad


@pytest.mark.parametrize("fmt", ["int8", "fp8"])
def test_read_back(lib, fmt):
    def call(T=1, bs=16, d=128, dt=0, out=P, ks=P):
        return getattr(lib, "pa_gather_cache_%s_block" % fmt)(P, P, ks, P, P, T, out, P, 8, bs, 2, d, dt, None)
    assert call(T=0) == OK
    for bad in (dict(T=-1), dict(out=None), dict(out=ODD), dict(ks=ODD2), dict(ks=None)):
        assert call(**bad) == INVALID, bad
    for bad in (dict(bs=7), dict(dt=9), dict(d=96)):
        assert call(**bad) == UNSUPPORTED, bad


@pytest.mark.parametrize("fmt", ["int8", "fp8"])
def test_decode(lib, fmt):
    def call(B=2, H=4, Hkv=2, d=128, bs=16, N=8, mb=4, n=64, dt=0, ws=1 << 24, scale=0.1, q=P, kc=P, ks=P, out=P, w=P):
        return getattr(lib, "pa_decode_%s_block" % fmt)(q, kc, P, ks, P, P, mb, P, n, B, H, Hkv, d, bs, N, scale, dt,
                                                        out, w, ws, None)
    assert call(B=0) == OK
    for bad in (dict(B=-1), dict(H=0), dict(mb=0), dict(N=0), dict(n=-1), dict(scale=float("nan")), dict(ws=64),
                dict(q=None), dict(q=ODD), dict(kc=ODD), dict(ks=ODD2), dict(out=ODD), dict(out=None), dict(w=ODD)):
        assert call(**bad) == INVALID, bad
    for bad in (dict(H=5), dict(H=34), dict(d=96), dict(bs=64), dict(dt=2), dict(B=4097, ws=1 << 28),
                dict(mb=1 << 27, N=1 << 20)):
        assert call(**bad) == UNSUPPORTED, bad


def test_decode_weights(lib):
    size = lib.pa_decode_weights_workspace_size
    assert size(2, 4, 2, 128, 0) > lib.pa_decode_workspace_size(2, 4, 128)
    assert size(2, 4, 2, 128, 1000) == size(2, 4, 2, 128, 0) + 1000 * 4 * 4
    assert size(2, 4, 2, 96, 8) == size(2, 4, 0, 128, 8) == size(2, 5, 2, 128, 8) == size(2, 4, 2, 128, -1) == 0

    def call(B=2, H=4, Hkv=2, d=128, bs=16, N=8, mb=4, n=64, dt=0, ws=1 << 24, scale=0.1, q=P, out=P, w=P, rows=P, R=3,
             W=64, work=P):
        return lib.pa_decode_weights(q, P, P, P, mb, P, n, B, H, Hkv, d, bs, N, scale, dt, out, w, rows, R, W, work, ws,
                                     None)
    assert call(B=0) == OK
    for bad in (dict(B=-1), dict(R=0), dict(W=0), dict(W=-1), dict(n=-1), dict(w=None), dict(w=ODD2), dict(rows=None),
                dict(rows=ODD2), dict(q=None), dict(out=ODD), dict(work=ODD), dict(work=None), dict(scale=float("inf")),
                dict(ws=size(2, 4, 2, 128, 0) - 1)):
        assert call(**bad) == INVALID, bad
    for bad in (dict(H=5), dict(H=34), dict(d=96), dict(bs=64), dict(dt=2), dict(B=4097, ws=1 << 28)):
        assert call(**bad) == UNSUPPORTED, bad


def test_select_tokens(lib):
    def call(w=P, R=3, W=64, rows=P, B=2, Hkv=2, keep=8, first=1, last=2, kept=P, new=P):
        return lib.pa_select_tokens(w, R, W, rows, P, B, Hkv, keep, first, last, kept, P, new, None)
    assert call(B=0) == OK
    for bad in (dict(B=-1), dict(R=0), dict(W=0), dict(Hkv=0), dict(keep=0, first=0, last=0), dict(first=-1),
                dict(last=-1), dict(keep=2), dict(first=2 ** 31 - 1, last=2 ** 31 - 1), dict(w=None), dict(w=ODD2),
                dict(kept=None), dict(rows=None), dict(new=ODD2)):
        assert call(**bad) == INVALID, bad
    assert call(B=4097) == UNSUPPORTED


def test_compact_tokens(lib):
    def call(k=P, kept=P, keep=8, mb=4, new=P, nmb=1, B=2, Hkv=2, d=64, bs=16, N=8, dt=0):
        return lib.pa_compact_tokens(k, P, kept, keep, P, P, mb, new, nmb, B, Hkv, d, bs, N, dt, None)
    assert call(B=0) == OK
    for bad in (dict(B=-1), dict(Hkv=0), dict(keep=0), dict(mb=0), dict(nmb=0), dict(N=0), dict(k=None), dict(k=ODD),
                dict(kept=None), dict(kept=ODD2), dict(new=None)):
        assert call(**bad) == INVALID, bad
    for bad in (dict(d=96), dict(bs=12), dict(dt=3), dict(B=4097), dict(N=1 << 28, bs=16)):
        assert call(**bad) == UNSUPPORTED, bad


def test_binding_refuses_tensors_that_do_not_fit():
    """Shapes are checked before any pointer is taken, so host tensors show it."""
    N, Hkv, bs, d, T = 4, 2, 8, 64, 3
    x = torch.zeros(T, Hkv, d, dtype=torch.float16)
    c, s = torch.zeros(N, Hkv, bs, d, dtype=torch.uint8), torch.zeros(N, Hkv)
    slots = torch.zeros(T, dtype=torch.int64)
    for append, gather in ((binding.pa_reshape_and_cache_int8_block, binding.pa_gather_cache_int8_block),
                           (binding.pa_reshape_and_cache_fp8_block, binding.pa_gather_cache_fp8_block)):
        for args in ((x, x[:2], slots, c, c, s, s), (x, x, slots[:2], c, c, s, s), (x, x, slots, c, c[:3], s, s),
                     (x, x, slots, c.transpose(1, 2), c, s, s), (x, x, slots, c, c, s[:, :1], s),
                     (x, x, slots, c, c, s, s[:2]), (x, x, slots, c[..., :32], c, s, s)):
            with pytest.raises(ValueError):
                append(*args)
            with pytest.raises(ValueError):
                gather(*args[3:], args[2], args[0], args[1])
    q = torch.zeros(2, 4, d, dtype=torch.float16)
    tbl, ln = torch.zeros(2, 3, dtype=torch.int32), torch.zeros(2, dtype=torch.int32)
    for decode in (binding.pa_decode_int8_block, binding.pa_decode_fp8_block):
        for bad in (dict(t=tbl[:1]), dict(n=ln[:1]), dict(out=q[:1]), dict(c=c[..., :32]), dict(s=s[:1])):
            cc, ss = bad.get("c", c), bad.get("s", s)
            with pytest.raises(ValueError):
                decode(q, cc, cc, ss, ss, bad.get("t", tbl), bad.get("n", ln), 8, 0.1, bad.get("out", q), torch.zeros(8))
    k, w = torch.zeros(N, bs, Hkv, d, dtype=torch.float16), torch.zeros(3, Hkv, 20)
    for bad in (dict(w=w[:, :1]), dict(r=ln[:1]), dict(n=ln[:1]), dict(t=tbl[:1]), dict(v=k[:2]), dict(out=q[:1])):
        with pytest.raises(ValueError):
            binding.pa_decode_weights(q, k, bad.get("v", k), bad.get("t", tbl), bad.get("n", ln), 8, 0.1,
                                      bad.get("out", q), bad.get("w", w), bad.get("r", ln), torch.zeros(8))
    kept = torch.zeros(2, Hkv, 5, dtype=torch.int32)
    for bad in (dict(w=w[:, :1]), dict(r=ln[:1]), dict(n=ln[:1]), dict(m=ln[:1]), dict(new=w[:2])):
        with pytest.raises(ValueError):
            binding.pa_select_tokens(bad.get("w", w), bad.get("r", ln), bad.get("n", ln), 1, 1, kept, bad.get("m", ln),
                                     bad.get("new", w))
    for bad in (dict(v=k[:2]), dict(kept=kept[:, :1]), dict(m=ln[:1]), dict(t=tbl[:1]), dict(new=tbl[:1])):
        with pytest.raises(ValueError):
            binding.pa_compact_tokens(k, bad.get("v", k), bad.get("kept", kept), bad.get("m", ln), bad.get("t", tbl),
                                      bad.get("new", tbl))
