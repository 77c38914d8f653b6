"""pa_compact_tokens: no row is written over before every CTA of the cluster has read its
own.  On the CPU: what the kernel's source asks of the barrier.  On the GPU: moves in place by a few
places, several stretches of every cluster size, while another stream keeps the memory busy."""
import numpy as np
import pytest
import torch

from oracle import evict as oe
from paged_kv_cache_103_gb300 import binding
from paged_kv_cache_103_gb300 import build as pa_build
from paged_kv_cache_103_gb300 import workloads as wl

from _cache4 import dev, rand_tables
from test_overlapped_launches import kernel_body

F16, BF16 = torch.float16, torch.bfloat16


def test_the_meeting_orders_reads_before_writes():
    """Reads before a barrier come before writes behind it only where the arrival releases and the wait
    acquires (one CTA: __syncthreads); a relaxed arrival orders nothing."""
    body = kernel_body("compact_kernel", "pa_evict.cu")
    assert ".relaxed" not in body
    reads = body.rindex("pa::ld_behind_wait(p.v_cache")
    writes = body.index("p.k_cache[piece(now[u])] =")
    for barrier in ("barrier.cluster.arrive.release.aligned", "barrier.cluster.wait.acquire.aligned", "__syncthreads()"):
        assert body.count(barrier) == 1 and reads < body.index(barrier) < writes, barrier


@pytest.mark.gpu
@pytest.mark.parametrize("B,Hkv,keep,d,bs,dtype", [
    (1, 1, 9000, 128, 16, BF16),      # a cluster of eight CTAs of 1024 threads, stretches of 2048 rows
    (5, 8, 5000, 64, 8, F16),         # eight of 512, stretches of 2048
    (10, 10, 2000, 128, 32, BF16),    # eight of 256, stretches of 512
    (13, 10, 250, 128, 16, F16),      # four, one stretch
    (13, 10, 120, 128, 16, BF16),     # two, one stretch
    (20, 8, 1000, 128, 16, F16),      # more pairs than SMs
    (90, 8, 300, 128, 8, BF16)])      # many more: a CTA of 256 threads each, stretches of 64 rows
def test_moves_in_place_by_a_few_places(B, Hkv, keep, d, bs, dtype):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    pa_build.build()
    n = keep + 63
    tbl, N = rand_tables([n] * B, bs, 1)
    rng = np.random.default_rng(2)
    was = [wl.normal_tensor((N, bs, Hkv, d), dtype, x).cuda() for x in (1, 2)]
    kv = [torch.empty_like(x) for x in was]
    lens = dev(np.full(B, keep, np.int32))[0]
    tables = dev(tbl)[0]
    noise = [torch.zeros(1 << 27, dtype=torch.uint8, device="cuda") for _ in range(2)]
    other = torch.cuda.Stream()
    for turn in range(8):
        shift = rng.integers(1, 64, (B, Hkv, 1)) if turn else np.ones((B, Hkv, 1), np.int64)
        late = rng.integers(0, keep, (B, Hkv, 1))        # from this row on by one more, as far as there is room
        pos = np.arange(keep)
        kept = pos + np.minimum(shift + (pos >= late), 63)
        kept_d = dev(kept.astype(np.int32))[0]
        src = tables.long()[torch.arange(B, device="cuda")[:, None, None], kept_d.long() // bs], kept_d.long() % bs
        dst = tables.long()[:, None, :].expand(-1, Hkv, -1)[:, :, torch.arange(keep, device="cuda") // bs]
        heads = torch.arange(Hkv, device="cuda")[None, :, None]
        want = []
        for x, y in zip(was, kv):
            y.copy_(x)
            w = x.clone()
            w[dst, torch.arange(keep, device="cuda") % bs, heads] = x[src[0], src[1], heads]
            want.append(w)
        torch.cuda.synchronize()
        with torch.cuda.stream(other):
            for _ in range(8):
                noise[1].copy_(noise[0])
        binding.pa_compact_tokens(*kv, kept_d, lens, tables, tables)
        torch.cuda.synchronize()
        assert binding.pa_check_device_errors() == 0
        for got, w in zip(kv, want):
            assert torch.equal(got.view(torch.int16), w.view(torch.int16)), turn


@pytest.mark.gpu
@pytest.mark.parametrize("batch", [False, True])
@pytest.mark.parametrize("B,Hkv,n,keep,d,bs,dtype", [
    (32, 8, 701, 300, 128, 16, BF16), (90, 8, 500, 333, 128, 8, F16), (7, 2, 3000, 2900, 64, 32, F16)])
def test_forks_cut_for_one_move(B, Hkv, n, keep, d, bs, dtype, batch):
    """Forks of one sequence, some of them grown on, all cut and moved in one call: what one moves
    is what was there before the call, whatever the others write."""
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    pa_build.build()
    rng = np.random.default_rng(B)
    need = -(-n // bs)
    a = binding.Allocator(need + B * (-(-keep // bs) + 3), bs)
    a.alloc(0, n)
    ids = list(range(B))
    for i in ids[1:]:
        a.fork(0, i)
    for _ in range(bs + 1):
        a.append_batch(ids[::2])
    old, lens = a.export(ids, need + 3)
    if batch:
        a.evict_batch(ids, [keep] * B)
    else:
        for i in ids:
            a.evict(i, keep)
    new, _ = a.export(ids, need + 3)
    for i in ids:
        others = np.delete(old, i, 0)
        assert not np.isin(new[i][new[i] >= 0], others).any()
    kept = np.empty((B, Hkv, keep), np.int32)
    for i in ids:
        for g in range(Hkv):
            kept[i, g] = np.sort(rng.choice(lens[i], keep, replace=False))
    host = [rng.integers(-2 ** 15, 2 ** 15, (a.stats()["num_blocks"], bs, Hkv, d)).astype(np.int16) for _ in "kv"]
    kv = [x.view(dtype) for x in dev(*host)]
    binding.pa_compact_tokens(*kv, *dev(kept, np.full(B, keep, np.int32), old, new))
    assert binding.pa_check_device_errors() == 0
    for got, want in zip(kv, host):
        oe.compact_tokens(want, kept, [keep] * B, old, new)
        assert np.array_equal(got.view(torch.int16).cpu().numpy(), want)
