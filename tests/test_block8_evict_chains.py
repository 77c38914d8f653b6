"""Runs of the block-scaled cache's and the eviction's calls: enqueued behind a delay so that each is
launched while the one before it runs, captured and replayed, on two streams at once, over pools and
accumulators beyond 4 GiB, of the largest batch."""
import re

import numpy as np
import pytest
import torch

from oracle import block8 as ob
from oracle import evict as oe
from paged_kv_cache_103_gb300 import binding
from paged_kv_cache_103_gb300 import build as pa_build
from paged_kv_cache_103_gb300 import workloads as wl

from _block8 import decode_bound
from _cache4 import dev, workspace
from test_overlapped_launches import kernel_body

gpu = pytest.mark.gpu
F16, BF16 = torch.float16, torch.bfloat16


@pytest.mark.parametrize("name,source", [("decode_block8_kernel", "pa_decode_block8.cuh"),
                                         ("select_tokens_kernel", "pa_evict.cu"), ("compact_kernel", "pa_evict.cu"),
                                         ("add_weights_kernel", "pa_decode.cu")])
def test_reads_behind_the_wait_are_coherent(name, source):
    body = kernel_body(name, source)
    assert "griddepcontrol.wait" in body
    assert not re.search(r"\b__ldg\(", body) and "__restrict__" not in body
    if source.endswith("8.cuh"):
        text = open(pa_build.CSRC + "/pa_runs.cuh").read()
        assert not re.search(r"\b__ldg\(", text) and "__restrict__" not in text


@pytest.fixture(scope="module")
def lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    pa_build.build()
    binding.load()


class Block8:
    """Appends, read backs and decodes of one block-scaled cache; run(wait) makes the calls."""

    def __init__(self, fmt, T, Hkv, G, d=128, bs=16, seed=0):
        N = -(-T // bs) + 1
        self.fmt, self.T, self.scale = fmt, T, d ** -0.5
        gen = torch.Generator().manual_seed(seed)
        self.rows = [[(wl.normal_tensor((T, Hkv, d), BF16, seed + 10 * i + j) * 2 ** i).cuda() for j in range(2)]
                     for i in range(3)]
        self.qs = [wl.normal_tensor((1, Hkv * G, d), BF16, seed + 70 + i).cuda() for i in range(3)]
        self.tbl = torch.randperm(N, generator=gen).int().view(1, N).cuda()
        self.slots = torch.arange(T).cuda()
        self.slots = self.tbl[0].long()[self.slots // bs] * bs + self.slots % bs
        self.lens = torch.tensor([T], dtype=torch.int32).cuda()
        self.cache = [torch.zeros(N, Hkv, bs, d, dtype=torch.uint8).cuda() for _ in "kv"]
        self.cache += [torch.zeros(N, Hkv).cuda() for _ in "kv"]
        self.ws = workspace(1, Hkv * G, d)
        self.append_, self.gather_, self.decode_ = (getattr(binding, "pa_%s_%s_block" % (x, fmt)) for x in
                                                    ("reshape_and_cache", "gather_cache", "decode"))

    def outs(self, n):
        return ([torch.zeros(2, *self.rows[0][0].shape, dtype=BF16, device="cuda") for _ in range(n)]
                + [torch.zeros_like(self.qs[0]) for _ in range(2 * n)])

    def run(self, n, outs, wait=lambda: None, stream=None):
        for i in range(n):
            self.append_(*self.rows[i % 3], self.slots, *self.cache, stream=stream)
            wait()
            self.gather_(*self.cache, self.slots, outs[i][0], outs[i][1], stream=stream)
            wait()
            a, b = outs[n + 2 * i], outs[n + 2 * i + 1]
            self.decode_(self.qs[i % 3], *self.cache, self.tbl, self.lens, self.T, self.scale, a, self.ws,
                         stream=stream)
            wait()
            self.decode_(a, *self.cache, self.tbl, self.lens, self.T, self.scale, b, self.ws, stream=stream)
            wait()


class Evict:
    """Decodes with weights, each followed by a choice and a move in place, of two sequences."""

    def __init__(self, n, Hkv, G, d=128, bs=16, seed=0):
        nb = -(-n // bs)
        gen = torch.Generator().manual_seed(seed)
        self.n, self.scale, self.first = n, 0.3, 2
        self.tbl = torch.randperm(2 * nb, generator=gen).int().view(2, nb).cuda()
        self.kv = [wl.normal_tensor((2 * nb, bs, Hkv, d), F16, seed + x).cuda() for x in (1, 2)]
        self.q = wl.normal_tensor((2, Hkv * G, d), F16, seed + 3).cuda()
        self.lens = torch.tensor([n, n - 5], dtype=torch.int32).cuda()
        self.rows = torch.tensor([2, 0], dtype=torch.int32).cuda()
        self.keep = n // 2
        self.kept = torch.zeros(2, Hkv, self.keep, dtype=torch.int32).cuda()
        self.kept_lens = torch.zeros(2, dtype=torch.int32).cuda()
        self.shape = (3, Hkv, n + 3)
        self.ws = torch.zeros(binding.pa_decode_weights_workspace_size(2, Hkv * G, Hkv, d, 2 * n), dtype=torch.uint8,
                              device="cuda")

    def outs(self, n):
        return ([torch.zeros(self.shape, device="cuda") for _ in range(n)]
                + [torch.zeros_like(self.kept) for _ in range(n)] + [torch.zeros_like(self.q) for _ in range(2 * n)]
                + [x.clone() for x in self.kv])

    def run(self, n, outs, wait=lambda: None, stream=None):
        k, v = outs[-2:]
        for i in range(n):
            w, kept, a, b = outs[i], outs[n + i], outs[2 * n + 2 * i], outs[2 * n + 2 * i + 1]
            binding.pa_decode_weights(self.q, k, v, self.tbl, self.lens, self.n, self.scale, a, w, self.rows, self.ws,
                                      stream=stream)
            wait()
            binding.pa_select_tokens(w, self.rows, self.lens, self.first, 7, kept, self.kept_lens, w, stream=stream)
            wait()
            binding.pa_compact_tokens(k, v, kept, self.kept_lens, self.tbl, self.tbl, stream=stream)
            wait()
            binding.pa_decode_weights(a, k, v, self.tbl, self.kept_lens, self.keep, self.scale, b, w, self.rows, self.ws,
                                      stream=stream)
            wait()


def make(kind):
    return {"int8": lambda s: Block8("int8", 700, 2, 4, seed=s), "fp8": lambda s: Block8("fp8", 333, 3, 1, 64, 8, s),
            "small": lambda s: Block8("int8", 40, 1, 8, 64, 32, s), "evict": lambda s: Evict(900, 2, 4, seed=s),
            "evict_small": lambda s: Evict(60, 1, 1, 64, 8, s), "evict_wide": lambda s: Evict(300, 8, 16, seed=s)}[kind](0)


KINDS = ("int8", "fp8", "small", "evict", "evict_small", "evict_wide")


def reference(c, n):
    want = c.outs(n)
    c.run(n, want, torch.cuda.synchronize)
    torch.cuda.synchronize()
    assert all(x.float().abs().amax() > 0 for x in want)
    return want


def same(got, want):
    torch.cuda.synchronize()
    assert binding.pa_check_device_errors() == 0
    for i, (a, b) in enumerate(zip(got, want)):
        assert torch.equal(a, b), i


@gpu
@pytest.mark.parametrize("kind", KINDS)
def test_calls_behind_a_delay(lib, kind):
    c, n = make(kind), 8
    want = reference(c, n)
    for _ in range(3):
        got = c.outs(n)
        torch.cuda.synchronize()
        torch.cuda._sleep(4_000_000)      # two milliseconds, in which all calls are enqueued
        c.run(n, got)
        same(got, want)


@gpu
@pytest.mark.parametrize("kind", KINDS)
def test_captured_and_replayed(lib, kind):
    c, n = make(kind), 4
    want = reference(c, n)
    got, first = c.outs(n), c.outs(n)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        c.run(n, got)
    for _ in range(3):
        for a, b in zip(got, first):
            a.copy_(b)
        graph.replay()
        same(got, want)


@gpu
@pytest.mark.parametrize("kind", KINDS)
def test_two_streams_at_once(lib, kind):
    """Two users of the library, each with buffers and a workspace of its own; streams given as objects
    and as handles."""
    cs, n = [make(kind), make(kind)], 6
    want = reference(cs[0], n)
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(3):
        got = [c.outs(n) for c in cs]
        torch.cuda.synchronize()
        for c, g, s in zip(cs, got, (streams[0], streams[1].cuda_stream)):
            c.run(n, g, stream=s)
        for g in got:
            same(g, want)


@gpu
@pytest.mark.parametrize("fmt", ["int8", "fp8"])
def test_block8_pools_beyond_4_gib(lib, fmt):
    """5.4 GB of codes each: the same few blocks at the pool's start and at its end."""
    N, Hkv, bs, d, G, T = 164_000, 8, 32, 128, 4, 200
    nb = -(-T // bs)
    caches = [torch.zeros(N, Hkv, bs, d, dtype=torch.uint8, device="cuda") for _ in "kv"]
    scales = [torch.zeros(N, Hkv, device="cuda") for _ in "kv"]
    assert caches[0].nbytes > 4 << 30
    kn, vn = (wl.normal_tensor((T, Hkv, d), BF16, x).cuda() for x in (1, 2))
    q = wl.normal_tensor((2, Hkv * G, d), BF16, 3).cuda()
    tbl = torch.stack([torch.arange(nb), N - 1 - torch.arange(nb)]).int().cuda()
    pos = torch.arange(T, device="cuda")
    append, gather, decode = (getattr(binding, "pa_%s_%s_block" % (x, fmt)) for x in
                              ("reshape_and_cache", "gather_cache", "decode"))
    outs = []
    for i in range(2):
        slots = tbl[i].long()[pos // bs] * bs + pos % bs
        append(kn, vn, slots, *caches, *scales)
        ko, vo = torch.zeros_like(kn), torch.zeros_like(vn)
        gather(*caches, *scales, slots, ko, vo)
        outs.append((ko, vo))
    assert all(torch.equal(a, b) for a, b in zip(*outs)) and (outs[0][0].float() - kn.float()).abs().max() < 0.2
    out = torch.zeros_like(q[:1]).expand(2, -1, -1).contiguous()
    decode(q[:1].expand(2, -1, -1).contiguous(), *caches, *scales, tbl,
           torch.tensor([T, T], dtype=torch.int32, device="cuda"), T, d ** -0.5, out, workspace(2, Hkv * G, d))
    assert binding.pa_check_device_errors() == 0
    host = [x[tbl[1].long()].cpu().numpy() for x in (*caches, *scales)]
    qn, one = q[:1].double().cpu().numpy(), np.arange(nb)[None]
    ref = ob.decode(qn, *host, one, [T], d ** -0.5, fmt)
    bound = decode_bound(qn, host, one, [T], d ** -0.5, BF16, ref, fmt)
    for i in range(2):
        assert (np.abs(out[i: i + 1].double().cpu().numpy() - ref) <= bound).all()


@gpu
def test_eviction_beyond_4_gib(lib):
    """A 16-bit pool of 5.2 GB each and 9.6 GB of accumulators, the sequence at the end of both."""
    N, bs, Hkv, d, n, keep = 20_000, 32, 32, 128, 500, 200
    k, v = (torch.zeros(N, bs, Hkv, d, dtype=F16, device="cuda") for _ in "kv")
    assert k.nbytes > 4 << 30
    R, W = 1500, 50_000
    weights = torch.zeros(R, Hkv, W, device="cuda")
    nb = -(-n // bs)
    tbl = (N - 1 - torch.arange(nb)).int()[None].cuda()
    for x, s in ((k, 1), (v, 2)):
        x[tbl[0].long()] = wl.normal_tensor((nb, bs, Hkv, d), F16, s).cuda()
    q, out = wl.normal_tensor((1, Hkv, d), F16, 3).cuda(), torch.zeros(1, Hkv, d, dtype=F16, device="cuda")
    lens, rows = torch.tensor([n], dtype=torch.int32).cuda(), torch.tensor([R - 1], dtype=torch.int32).cuda()
    ws = torch.zeros(binding.pa_decode_weights_workspace_size(1, Hkv, Hkv, d, n), dtype=torch.uint8, device="cuda")
    binding.pa_decode_weights(q, k, v, tbl, lens, n, 0.1, out, weights, rows, ws)
    got = weights[R - 1, :, :n].cpu().numpy()
    assert np.abs(got.sum(1) - 1).max() < 1e-5 and weights[: R - 1].abs().amax() == 0
    was = [x[tbl[0].long()].cpu().numpy().view(np.int16) for x in (k, v)]
    kept = torch.zeros(1, Hkv, keep, dtype=torch.int32, device="cuda")
    m = torch.zeros(1, dtype=torch.int32, device="cuda")
    binding.pa_select_tokens(weights, rows, lens, 3, 9, kept, m, weights)
    want, _ = oe.select_tokens(got[None], [0], [n], keep, 3, 9)
    assert np.array_equal(kept.cpu().numpy(), want)
    assert torch.equal(weights[R - 1, :, :keep].cpu(), torch.from_numpy(np.take_along_axis(got, want[0].astype(int), 1)))
    binding.pa_compact_tokens(k, v, kept, m, tbl, tbl)
    assert binding.pa_check_device_errors() == 0
    one = np.arange(nb)[None]
    for x, w in zip((k, v), was):
        oe.compact_tokens(w, want, [keep], one, one)
        assert np.array_equal(x[tbl[0].long()].cpu().numpy().view(np.int16), w)


@gpu
def test_largest_batch(lib):
    """4096 sequences of 0 .. 40 tokens: decode, weights, choice and move."""
    B, Hkv, G, d, bs = 4096, 2, 2, 64, 8
    rng = np.random.default_rng(0)
    lens = rng.integers(0, 41, B).astype(np.int32)
    nb = -(-lens // bs)
    N = int(nb.sum()) + 1
    tbl = np.full((B, 5), -1, np.int32)
    order, at = rng.permutation(N), 0
    for i in range(B):
        tbl[i, : nb[i]] = order[at: at + nb[i]]
        at += nb[i]
    dt, dl = dev(tbl, lens)
    q = wl.normal_tensor((B, Hkv * G, d), F16, 1)
    c = [rng.integers(0, 256, (N, Hkv, bs, d)).astype(np.uint8) for _ in "kv"]
    c += [rng.random((N, Hkv)).astype(np.float32) * 0.02 for _ in "kv"]
    out = torch.full((B, Hkv * G, d), 7.0, dtype=F16, device="cuda")
    binding.pa_decode_int8_block(q.cuda(), *dev(*c), dt, dl, 40, 0.125, out, workspace(B, Hkv * G, d))
    ref = ob.decode(q.double().numpy(), *c, tbl, lens, 0.125, "int8")
    bound = decode_bound(q.double().numpy(), c, tbl, lens, 0.125, F16, ref, "int8")
    assert (np.abs(out.double().cpu().numpy() - ref) <= bound).all()
    k, v = (wl.normal_tensor((N, bs, Hkv, d), F16, x) for x in (2, 3))
    kd, vd = k.cuda(), v.cuda()
    weights = torch.zeros(B, Hkv, 41, device="cuda")
    rows = rng.permutation(B).astype(np.int32)
    ws = torch.zeros(binding.pa_decode_weights_workspace_size(B, Hkv * G, Hkv, d, int(lens.sum())), dtype=torch.uint8,
                     device="cuda")
    binding.pa_decode_weights(q.cuda(), kd, vd, dt, dl, 40, 0.125, out, weights, dev(rows)[0], ws)
    ref, w = oe.decode_weights(*(x.double().numpy() for x in (q, k, v)), tbl, lens, 0.125)
    assert np.abs(out.double().cpu().numpy() - ref).max() < 2e-3
    got = weights.cpu().numpy()
    for i in range(B):
        assert np.abs(got[rows[i], :, : lens[i]] - w[i]).max(initial=0) < 1e-5 and (got[rows[i], :, lens[i]:] == 0).all()
    kept, m = torch.empty(B, Hkv, 17, dtype=torch.int32, device="cuda"), torch.empty(B, dtype=torch.int32, device="cuda")
    binding.pa_select_tokens(weights, *dev(rows, lens), 1, 4, kept, m, weights)
    want, want_m = oe.select_tokens(got, rows, lens, 17, 1, 4)
    assert np.array_equal(kept.cpu().numpy(), want) and np.array_equal(m.cpu().numpy(), want_m)
    binding.pa_compact_tokens(kd, vd, kept, m, dt, dt)
    assert binding.pa_check_device_errors() == 0
    for x, y in ((kd, k), (vd, v)):
        host = y.numpy().view(np.int16)
        oe.compact_tokens(host, want, want_m, tbl, tbl)
        assert np.array_equal(x.cpu().numpy().view(np.int16), host)
