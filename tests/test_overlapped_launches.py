"""Kernels that are launched before their predecessor in the stream has ended.

On the CPU: what such a kernel reads behind its wait goes through coherent reads.  On the GPU: whole
chains of calls enqueued behind a delay, so that every call is there before the first one starts and
each of them is launched early, against the same calls waited for one by one; the pairs of calls that
may overlap stand next to each other, in a stream and in a captured graph."""
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


def append_gather(c, n, wait):
    """Every append overwrites the rows that the read back before it read."""
    outs = [torch.zeros(2, *c.rows[0][0].shape, dtype=c.x.dtype, device="cuda") for _ in range(n)]
    yield outs
    for i in range(n):
        c.append(i)
        wait()
        c.gather(i, outs[i])
        wait()


def append_decode(c, n, wait):
    outs = [torch.zeros_like(c.x) for _ in range(n)]
    yield outs
    for i in range(n):
        c.append(i)
        wait()
        c.decode(c.qs[i % 3], outs[i])
        wait()


def decode_decode(c, n, wait):
    """A decode's output is the next one's query; one workspace."""
    outs = [torch.zeros_like(c.x) for _ in range(n)]
    c.append(0)
    yield outs
    for i in range(n):
        c.decode(outs[i - 1] if i else c.qs[0], outs[i])
        wait()


def decode_gather(c, n, wait):
    outs = [torch.zeros(2, *c.rows[0][0].shape, dtype=c.x.dtype, device="cuda") for _ in range(n)]
    mid = [torch.zeros_like(c.x) for _ in range(n)]
    c.append(0)
    yield outs + mid
    for i in range(n):
        c.decode(c.qs[i % 3], mid[i])
        wait()
        c.gather(i, outs[i])
        wait()


def select_decode(c, n, wait):
    """The lists are overwritten by the next selection, whose query is this decode's output."""
    outs = [torch.zeros_like(c.x) for _ in range(n)]
    yield outs
    for i in range(n):
        q = outs[i - 1] if i % 3 else c.qs[i % 2]
        c.select(q)
        wait()
        c.selected(q, outs[i])
        wait()


def decode_then_selected(c, n, wait):
    """A 4-bit decode's output is the query of the decode behind it, over lists made before."""
    outs = [torch.zeros_like(c.x) for _ in range(2 * n)]
    c.append(0)
    c.select(c.qs[0])
    yield outs
    for i in range(n):
        c.decode(outs[2 * i - 1] if i else c.qs[0], outs[2 * i])
        wait()
        c.selected(outs[2 * i], outs[2 * i + 1])
        wait()


CHAINS = [append_gather, append_decode, decode_decode, decode_gather, select_decode, decode_then_selected]


@gpu
@pytest.mark.parametrize("captured", [False, True])
@pytest.mark.parametrize("T,Hkv,G", [(5, 1, 2), (700, 8, 4), (6000, 4, 1)])
@pytest.mark.parametrize("chain", CHAINS)
def test_chains_behind_a_delay(lib, chain, T, Hkv, G, captured):
    n = 24
    c = Chain(T, Hkv, G)

    def calls(wait):
        gen = chain(c, n, wait)
        outs = next(gen)
        return outs, lambda: next(gen, None)
    want, go = calls(torch.cuda.synchronize)
    go()
    torch.cuda.synchronize()
    if captured:
        got, go = calls(lambda: None)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            go()
        for _ in range(3):
            for x in got:
                x.zero_()
            torch.cuda.synchronize()
            graph.replay()
            torch.cuda.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(got, want))
    else:
        for _ in range(3):
            got, go = calls(lambda: None)
            torch.cuda.synchronize()
            torch.cuda._sleep(4_000_000)      # two milliseconds, in which all calls are enqueued
            go()
            torch.cuda.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(got, want))
    assert binding.pa_check_device_errors() == 0
    assert want[0].abs().amax() > 0


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
