"""Kernels that are launched before their predecessor in the stream has ended.

On the CPU: what such a kernel reads behind its wait goes through coherent reads.  On the GPU: rows
read on one stream while their neighbours are written and read back on another."""
import os
import re

import pytest
import torch

from paged_kv_cache_103_gb300 import binding
from paged_kv_cache_103_gb300 import build as pa_build
from paged_kv_cache_103_gb300 import workloads as wl

from _cache4 import workspace

gpu = pytest.mark.gpu


def kernel_body(name, source):
    text = open(os.path.join(pa_build.CSRC, source)).read()
    start = text.index(name + "(")
    depth, at = 0, text.index("{", text.index(") {", start))
    for end in range(at, len(text)):
        depth += {"{": 1, "}": -1}.get(text[end], 0)
        if depth == 0:
            return text[start: end]
    raise AssertionError("no end of " + name)


@pytest.mark.parametrize("name,source", [("gather_cache_kernel", "pa_cache_int4.cu"),
                                         ("decode_int4_kernel", "pa_decode_int4.cu"),
                                         ("paged_decode_kernel", "pa_decode.cu")])
def test_reads_behind_the_wait_are_coherent(name, source):
    """No read through the read-only path, asked for (__ldg) or offered (const __restrict__)."""
    body = kernel_body(name, source)
    assert "griddepcontrol.wait" in body
    assert not re.search(r"\b__ldg\(", body)
    assert "__restrict__" not in body


@pytest.fixture(scope="module")
def lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    pa_build.build()
    binding.load()


class Chain:
    """Calls over buffers of their own; run() makes all of them, each with its own outputs."""

    def __init__(self, T, Hkv, G, d=128, bs=16, keep=4, dtype=torch.bfloat16):
        N = -(-T // bs) + 2
        self.T, self.scale, self.bs, self.keep = T, d ** -0.5, bs, min(keep, -(-T // bs))
        self.rows = [[wl.normal_tensor((T, Hkv, d), dtype, 10 * i + j).cuda() for j in range(2)] for i in range(3)]
        self.qs = [wl.normal_tensor((1, Hkv * G, d), dtype, 70 + i).cuda() for i in range(3)]
        self.slots = torch.arange(T).cuda()
        self.tbl = torch.randperm(N, generator=torch.Generator().manual_seed(T)).int().view(1, N).cuda()
        self.slots = (self.tbl[0].long()[self.slots // bs] * bs + self.slots % bs)
        self.lens = torch.tensor([T], dtype=torch.int32).cuda()
        self.cache = [torch.zeros(N, Hkv, bs, d // 2, dtype=torch.uint8).cuda() for _ in "kv"]
        self.cache += [torch.zeros(N, Hkv, bs, d // 64, 2, dtype=torch.float16).cuda() for _ in "kv"]
        self.k16 = wl.normal_tensor((N, bs, Hkv, d), dtype, 5).cuda()
        self.boxes = torch.zeros(N, Hkv, 2, d, dtype=torch.int8).cuda()
        self.S = torch.zeros(N, Hkv).cuda()
        binding.pa_summarize_blocks(self.k16, torch.arange(N, dtype=torch.int32).cuda(), self.boxes, self.S)
        self.sel = torch.zeros(1, Hkv, self.keep, dtype=torch.int32).cuda()
        self.sel_n = torch.zeros(1, Hkv, dtype=torch.int32).cuda()
        self.ws = workspace(1, Hkv * G, d)
        self.wsel = torch.zeros(binding.pa_select_blocks_workspace_size(1, Hkv, N), dtype=torch.uint8).cuda()
        self.x = torch.zeros_like(self.qs[0])

    def append(self, i):
        binding.pa_reshape_and_cache_int4(*self.rows[i % 3], self.slots, *self.cache)

    def gather(self, i, out):
        binding.pa_gather_cache_int4(*self.cache, self.slots, out[0], out[1])

    def decode(self, q, out):
        binding.pa_decode_int4(q, *self.cache, self.tbl, self.lens, self.T, self.scale, out, self.ws)

    def select(self, q):
        binding.pa_select_blocks(q, self.boxes, self.S, self.tbl, self.lens, self.bs, 0, 1, self.sel, self.sel_n,
                                 self.wsel)

    def selected(self, q, out):
        binding.pa_decode_selected(q, self.k16, self.k16, self.sel, self.sel_n, self.keep * self.bs, self.scale, out,
                                   self.ws)


@gpu
def test_rows_read_on_another_stream_while_their_neighbours_are_written(lib):
    """Rows that share a cache line with rows being appended are read all the time on a second
    stream; what is read back behind the append is new all the same."""
    T, Hkv, d, bs = 512, 2, 128, 16
    c = Chain(T, Hkv, 2, d, bs)
    c.append(0)
    even, odd = c.slots[0::2].contiguous(), c.slots[1::2].contiguous()
    side = torch.cuda.Stream()
    other = torch.empty(2, T // 2, Hkv, d, dtype=c.x.dtype, device="cuda")
    outs = [torch.zeros_like(other) for _ in range(30)]
    new = [[r[0::2].contiguous() for r in rows] for rows in c.rows]
    want = []
    for i in range(3):
        binding.pa_reshape_and_cache_int4(*new[i], even, *c.cache)
        w = torch.zeros_like(other)
        torch.cuda.synchronize()
        binding.pa_gather_cache_int4(*c.cache, even, w[0], w[1])
        torch.cuda.synchronize()
        want.append(w)
    torch.cuda._sleep(4_000_000)
    side.wait_stream(torch.cuda.current_stream())
    for i, out in enumerate(outs):
        binding.pa_gather_cache_int4(*c.cache, odd, other[0], other[1], stream=side)
        binding.pa_reshape_and_cache_int4(*new[i % 3], even, *c.cache)
        binding.pa_gather_cache_int4(*c.cache, even, out[0], out[1])
    torch.cuda.synchronize()
    assert binding.pa_check_device_errors() == 0
    for i, out in enumerate(outs):
        assert torch.equal(out, want[i % 3]), i
