"""Calls of the 4-bit cache and of block-sparse decode queued behind each other: a call that is
launched while the one before it runs must read what that one writes and must not write what it still
reads, so a queue of calls gives bit for bit what the same calls give one at a time."""
import numpy as np
import pytest
import torch

from paged_kv_cache_103_gb300 import binding
from paged_kv_cache_103_gb300 import workloads as wl

from _cache4 import workspace

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from paged_kv_cache_103_gb300 import build
    build.build()
    binding.load()


def _both(step, n):
    """Outputs of n steps queued, and of n steps with a wait after every call."""
    def wait():
        torch.cuda.synchronize()
    queued = [step(i, lambda: None) for i in range(n)]
    torch.cuda.synchronize()
    single = [step(i, wait) for i in range(n)]
    torch.cuda.synchronize()
    return queued, single


@pytest.mark.parametrize("T,Hkv", [(3, 1), (64, 8), (2000, 8)])
def test_append_read_back_and_decode(T, Hkv):
    """Every step overwrites the same slots, then decodes over them and reads them back."""
    bs, d, G = 16, 128, 4
    N = -(-T // bs) + 3
    rows = [[wl.normal_tensor((T, Hkv, d), torch.bfloat16, 10 * i + j).cuda() for j in range(2)] for i in range(6)]
    q = wl.normal_tensor((1, Hkv * G, d), torch.bfloat16, 5).cuda()
    slots = torch.arange(T).cuda()
    tbl = torch.arange(N, dtype=torch.int32).view(1, N).cuda()
    lens = torch.tensor([T], dtype=torch.int32).cuda()
    ws = workspace(1, Hkv * G, d)
    codes = [torch.zeros(N, Hkv, bs, d // 2, dtype=torch.uint8).cuda() for _ in "kv"]
    scales = [torch.zeros(N, Hkv, bs, d // 64, 2, dtype=torch.float16).cuda() for _ in "kv"]
    bufs = [[[torch.empty_like(q)] + [torch.empty_like(r) for r in rows[0]] for _ in range(24)] for _ in range(2)]
    runs = iter(bufs[0] + bufs[1])

    def step(i, wait):
        out, kb, vb = next(runs)
        binding.pa_reshape_and_cache_int4(*rows[i % 6], slots, *codes, *scales)
        wait()
        binding.pa_decode_int4(q, *codes, *scales, tbl, lens, T, 0.1, out, ws)
        wait()
        binding.pa_gather_cache_int4(*codes, *scales, slots, kb, vb)
        wait()
        return out, kb, vb
    queued, single = _both(step, 24)
    assert binding.pa_check_device_errors() == 0
    for i, (a, b) in enumerate(zip(queued, single)):
        assert all(torch.equal(x, y) for x, y in zip(a, b)), i
    assert not torch.equal(queued[0][0], queued[1][0])


@pytest.mark.parametrize("n,keep", [(40, 8), (900, 6), (9000, 40)])
def test_summaries_selection_and_selected_decode(n, keep):
    """Every step has another query and other keys in the same buffers; the lists are overwritten."""
    bs, Hkv, G, d, B = 16, 2, 4, 64, 3
    nb = -(-n // bs)
    N = B * nb
    keys = [wl.normal_tensor((N, bs, Hkv, d), torch.float16, 70 + i).cuda() for i in range(3)]
    v = wl.normal_tensor((N, bs, Hkv, d), torch.float16, 4).cuda()
    k = torch.empty_like(v)
    qs = [wl.normal_tensor((B, Hkv * G, d), torch.float16, 90 + i).cuda() for i in range(4)]
    ids = torch.arange(N, dtype=torch.int32).cuda()
    tbl = torch.from_numpy(np.random.default_rng(1).permutation(N).astype(np.int32).reshape(B, nb)).cuda()
    lens = torch.tensor([n, max(1, n - 17), 0], dtype=torch.int32).cuda()
    boxes, S = torch.zeros(N, Hkv, 2, d, dtype=torch.int8).cuda(), torch.zeros(N, Hkv).cuda()
    sel, sn = torch.zeros(B, Hkv, keep, dtype=torch.int32).cuda(), torch.zeros(B, Hkv, dtype=torch.int32).cuda()
    wsel = torch.zeros(binding.pa_select_blocks_workspace_size(B, Hkv, nb), dtype=torch.uint8).cuda()
    ws = workspace(B, Hkv * G, d)
    outs = iter([torch.empty_like(qs[0]) for _ in range(48)])

    def step(i, wait):
        out = next(outs)
        k.copy_(keys[i % 3])
        wait()
        binding.pa_summarize_blocks(k, ids, boxes, S)
        wait()
        binding.pa_select_blocks(qs[i % 4], boxes, S, tbl, lens, bs, 1, 1, sel, sn, wsel)
        wait()
        binding.pa_decode_selected(qs[i % 4], k, v, sel, sn, keep * bs, 0.125, out, ws)
        wait()
        return out, sel.clone(), sn.clone()
    queued, single = _both(step, 24)
    assert binding.pa_check_device_errors() == 0
    for i, (a, b) in enumerate(zip(queued, single)):
        assert all(torch.equal(x, y) for x, y in zip(a, b)), i
    assert not torch.equal(queued[0][0], queued[1][0])


def test_two_streams_with_workspaces_of_their_own():
    """Two decodes and two selections at once, each pair on its own stream, over one cache."""
    bs, Hkv, G, d, n = 16, 4, 4, 128, 3000
    nb = -(-n // bs)
    codes = [torch.randint(0, 256, (nb, Hkv, bs, d // 2), dtype=torch.uint8).cuda() for _ in "kv"]
    scales = [torch.rand(nb, Hkv, bs, 2, 2).half().cuda() for _ in "kv"]
    k = wl.normal_tensor((nb, bs, Hkv, d), torch.float16, 3).cuda()
    boxes, S = torch.zeros(nb, Hkv, 2, d, dtype=torch.int8).cuda(), torch.zeros(nb, Hkv).cuda()
    ids = torch.arange(nb, dtype=torch.int32).cuda()
    tbl, lens = ids.view(1, nb), torch.tensor([n], dtype=torch.int32).cuda()
    binding.pa_summarize_blocks(k, ids, boxes, S)
    q = [wl.normal_tensor((1, Hkv * G, d), torch.float16, 40 + i).cuda() for i in range(2)]

    def calls(i, own, stream):
        out, sel, sn, ws, wsel = own
        for _ in range(20):
            binding.pa_decode_int4(q[i], *codes, *scales, tbl, lens, n, 0.05, out[0], ws, stream)
            binding.pa_select_blocks(q[i], boxes, S, tbl, lens, bs, 1, 2, sel, sn, wsel, stream)
            binding.pa_decode_selected(q[i], k, k, sel, sn, 20 * bs, 0.05, out[1], ws, stream)

    def own():
        return (torch.empty(2, 1, Hkv * G, d, dtype=torch.float16).cuda(),
                torch.empty(1, Hkv, 20, dtype=torch.int32).cuda(), torch.empty(1, Hkv, dtype=torch.int32).cuda(),
                workspace(1, Hkv * G, d),
                torch.empty(binding.pa_select_blocks_workspace_size(1, Hkv, nb), dtype=torch.uint8).cuda())
    alone, at_once = [own(), own()], [own(), own()]
    torch.cuda.synchronize()
    for i in range(2):
        calls(i, alone[i], None)
        torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for i in range(2):
        calls(i, at_once[i], streams[i])
    torch.cuda.synchronize()
    assert binding.pa_check_device_errors() == 0
    for i in range(2):
        for x, y in zip(alone[i][:3], at_once[i][:3]):
            assert torch.equal(x, y), i


@pytest.mark.parametrize("captured", [False, True])
def test_behind_copies_and_joined_streams(captured):
    """What the calls wait for may be a copy, a memset, or work that joins from another stream, in a
    stream as in a captured graph."""
    bs, Hkv, G, d, T = 16, 4, 4, 128, 1500
    N = -(-T // bs)
    src = [wl.normal_tensor((T, Hkv, d), torch.float16, 20 + i).cuda() for i in range(2)]
    qsrc = wl.normal_tensor((1, Hkv * G, d), torch.float16, 30).cuda()
    k16 = wl.normal_tensor((N, bs, Hkv, d), torch.float16, 31).cuda()
    slots = torch.arange(T).cuda()
    tbl = torch.arange(N, dtype=torch.int32).view(1, N).cuda()
    lens = torch.tensor([T], dtype=torch.int32).cuda()
    boxes, S = torch.zeros(N, Hkv, 2, d, dtype=torch.int8).cuda(), torch.zeros(N, Hkv).cuda()
    binding.pa_summarize_blocks(k16, tbl[0], boxes, S)
    codes = [torch.zeros(N, Hkv, bs, d // 2, dtype=torch.uint8).cuda() for _ in "kv"]
    scales = [torch.zeros(N, Hkv, bs, 2, 2, dtype=torch.float16).cuda() for _ in "kv"]
    new = [torch.zeros_like(x) for x in src]
    q = torch.zeros_like(qsrc)
    out = torch.zeros(2, 1, Hkv * G, d, dtype=torch.float16).cuda()
    back = [torch.zeros_like(x) for x in src]
    sel, sn = torch.zeros(1, Hkv, 12, dtype=torch.int32).cuda(), torch.zeros(1, Hkv, dtype=torch.int32).cuda()
    ws, ws2 = workspace(1, Hkv * G, d), workspace(1, Hkv * G, d)
    wsel = torch.zeros(binding.pa_select_blocks_workspace_size(1, Hkv, N), dtype=torch.uint8).cuda()
    side = torch.cuda.Stream()

    def work():
        main = torch.cuda.current_stream()
        side.wait_stream(main)
        with torch.cuda.stream(side):
            for a, b in zip(new, src):
                a.copy_(b)
            binding.pa_reshape_and_cache_int4(*new, slots, *codes, *scales)
        q.copy_(qsrc)
        binding.pa_select_blocks(q, boxes, S, tbl, lens, bs, 1, 1, sel, sn, wsel)
        main.wait_stream(side)                      # behind the selection and the append
        binding.pa_decode_selected(q, k16, k16, sel, sn, 12 * bs, 0.1, out[1], ws2)
        out[0].zero_()
        binding.pa_decode_int4(q, *codes, *scales, tbl, lens, T, 0.1, out[0], ws)
        for x in back:
            x.zero_()
        binding.pa_gather_cache_int4(*codes, *scales, slots, *back)

    # one call after the other, each waited for
    for a, b in zip(new, src):
        a.copy_(b)
    q.copy_(qsrc)
    steps = [lambda: binding.pa_reshape_and_cache_int4(*new, slots, *codes, *scales),
             lambda: binding.pa_select_blocks(q, boxes, S, tbl, lens, bs, 1, 1, sel, sn, wsel),
             lambda: binding.pa_decode_selected(q, k16, k16, sel, sn, 12 * bs, 0.1, out[1], ws2),
             lambda: binding.pa_decode_int4(q, *codes, *scales, tbl, lens, T, 0.1, out[0], ws),
             lambda: binding.pa_gather_cache_int4(*codes, *scales, slots, *back)]
    for f in steps:
        f()
        torch.cuda.synchronize()
    results = [*codes, *scales, sel, sn, out, *back]
    want = [x.clone() for x in results]
    assert out.abs().amax() > 0 and back[0].abs().amax() > 0
    run = work
    if captured:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            work()
        run = graph.replay
    for _ in range(3):
        for x in results + new + [q]:
            x.zero_()
        torch.cuda.synchronize()
        run()
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(results, want))
    assert binding.pa_check_device_errors() == 0
