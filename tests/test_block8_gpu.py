"""The block-scaled 8-bit cache on the GPU: append and read back bit for bit against the oracle, decode
within the rounding of its steps."""
import numpy as np
import pytest
import torch

from oracle import block8 as o
from paged_kv_cache_103_gb300 import binding
from paged_kv_cache_103_gb300 import workloads as wl

from _block8 import FMTS, behind, cache, decode_bound
from _cache4 import dev, max_blocks_of, rand_tables, workspace

pytestmark = pytest.mark.gpu
F16, BF16 = torch.float16, torch.bfloat16
APPEND = {"int8": binding.pa_reshape_and_cache_int8_block, "fp8": binding.pa_reshape_and_cache_fp8_block}
GATHER = {"int8": binding.pa_gather_cache_int8_block, "fp8": binding.pa_gather_cache_fp8_block}
DECODE = {"int8": binding.pa_decode_int8_block, "fp8": binding.pa_decode_fp8_block}


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from paged_kv_cache_103_gb300 import build
    build.build()
    binding.load()


def rows(T, Hkv, d, dtype, seed):
    """Rows of very different sizes, zeros and ties among them."""
    x = wl.normal_tensor((T, Hkv, d), torch.float32, seed)
    x = x * (1 + 9 * (torch.arange(d) % 17 == 3))
    g = torch.Generator().manual_seed(seed)
    x = x * 2.0 ** torch.randint(-6, 7, (T, Hkv, 1), generator=g).float()
    x[::5, :, 1:] = 0.0
    x[3::7] = 0.0
    x[4::9] = (torch.arange(d) % 32) / 2.0 - 8          # ties of either format
    if dtype == BF16:
        x[5::11, :, 2] = 3e38
        x[6::11] = x[6::11] * 1e-30
    else:
        x[5::11, :, 2] = 65504.0
        x[6::11] = 2.0 ** -24
    return x.to(dtype)


def same(dev_cache, host):
    for got, want in zip(dev_cache, host):
        off = got.cpu().numpy().view(np.uint8) != want.view(np.uint8)
        assert not off.any(), np.argwhere(off)[:5].tolist()


def both(fmt, kn, vn, slots, on_gpu, host):
    APPEND[fmt](kn.cuda(), vn.cuda(), torch.as_tensor(np.asarray(slots, np.int64)).cuda(), *on_gpu)
    o.append(kn.float().numpy(), slots, host[0], host[2], fmt)
    o.append(vn.float().numpy(), slots, host[1], host[3], fmt)


def empty(N, Hkv, bs, d):
    return ([np.full((N, Hkv, bs, d), 0x5A, np.uint8) for _ in "kv"]
            + [np.full((N, Hkv), 3.0, np.float32) for _ in "kv"])


def runs(lens, starts, bs, N, seed):
    """Slots of sequences that append lens[i] tokens behind starts[i] in scattered blocks."""
    rng = np.random.default_rng(seed)
    order, at, out = rng.permutation(N), 0, []
    for n, s in zip(lens, starts):
        pos = np.arange(s, s + n)
        nb = (s + n + bs - 1) // bs
        out.append(order[at: at + nb][pos // bs] * bs + pos % bs)
        at += nb
    return np.concatenate(out).astype(np.int64)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("T,seqs,bs,Hkv,d,dtype,pad", [
    (1, 1, 8, 1, 64, F16, 0), (1, 1, 32, 1, 128, BF16, 0), (7, 1, 8, 3, 64, F16, 0), (33, 1, 32, 2, 128, BF16, 5),
    (64, 64, 16, 5, 128, F16, 7), (250, 5, 16, 3, 64, BF16, 60), (1023, 3, 8, 4, 128, BF16, 0),
    (1024, 1, 32, 1, 64, F16, 500), (100, 25, 32, 40, 128, F16, 10)])
def test_append_bit_exact(fmt, T, seqs, bs, Hkv, d, dtype, pad):
    rng = np.random.default_rng(T + seqs)
    lens = [T // seqs + (i < T % seqs) for i in range(seqs)]
    starts = rng.integers(0, bs, seqs)
    starts[::3] = 0
    N = sum((s + n + bs - 1) // bs for s, n in zip(starts, lens)) + 2
    slots = runs(lens, starts, bs, N, T)
    slots[rng.permutation(T)[:pad]] = -1
    host = empty(N, Hkv, bs, d)
    for x in host[:2]:
        x[:] = rng.integers(0, 255, x.shape, dtype=np.uint8)
        x[x == 0x80] = 0x81 if fmt == "int8" else 0x80
    for x in host[2:]:
        x[:] = np.float32(2.0) ** rng.integers(-9, 6, x.shape)
        x[::4] = 0.0
    on = dev(*host)
    kn, vn = rows(T, Hkv, d, dtype, 5), rows(T, Hkv, d, dtype, 6)
    both(fmt, kn, vn, slots, on, host)
    same(on, host)
    assert binding.pa_check_device_errors() == 0
    # the same rows again, then others a token at a time
    both(fmt, kn, vn, slots, on, host)
    top = float(torch.finfo(dtype).max)
    four = (kn.float() * 4).clamp(-top, top).to(dtype)      # finite: others are outside the contract
    for t in range(min(T, 9)):
        both(fmt, four[t: t + 1], vn[t: t + 1], slots[t: t + 1], on, host)
    same(on, host)


@pytest.mark.parametrize("fmt", FMTS)
def test_a_sequence_grows_token_by_token(fmt):
    """Eight sequences over 70 steps: blocks filled row by row, scales growing on the way."""
    Hkv, bs, d, B, N = 2, 16, 64, 8, 8 * 5
    order = np.random.default_rng(3).permutation(N).reshape(B, 5)
    host = empty(N, Hkv, bs, d)
    on = dev(*host)
    for t in range(70):
        kn, vn = rows(B, Hkv, d, F16, 100 + t), rows(B, Hkv, d, F16, 300 + t)
        slots = order[:, t // bs] * bs + t % bs
        both(fmt, kn, vn, slots, on, host)
    same(on, host)


@pytest.mark.parametrize("fmt", FMTS)
def test_padding_and_bad_slots_between_the_tokens_of_a_block(fmt):
    """A block's tokens with up to 200 padding entries, and slots outside the pool, between them."""
    Hkv, bs, d, N = 2, 16, 64, 6
    slots = np.full(900, -1, np.int64)
    for at, s in ((3, 18), (4, 19), (40, 20), (240, 21), (299, 22), (300, 80), (301, 81), (333, 82), (600, 0),
                  (640, 1), (899, 2)):
        slots[at] = s
    slots[120] = N * bs
    slots[298] = 1 << 40
    slots[620] = N * bs + 5
    host = empty(N, Hkv, bs, d)
    on = dev(*host)
    kn, vn = rows(900, Hkv, d, BF16, 1), rows(900, Hkv, d, BF16, 2)
    both(fmt, kn, vn, slots, on, host)
    same(on, host)
    assert binding.pa_check_device_errors() == binding.DEVERR["SLOT"]


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("d,dtype", [(64, F16), (128, BF16)])
def test_padded_batches(fmt, d, dtype):
    """Sequences padded to a common length, thousands of entries between the tokens of two of them and,
    twice, between two tokens of one block."""
    Hkv, bs, wide, lens = 3, 16, 2500, [40, 1, 0, 2500, 17, 16]
    starts = [5, 0, 0, 9, 15, 0]
    N = sum((s + n + bs - 1) // bs for s, n in zip(starts, lens)) + 1
    flat, at = runs(lens, starts, bs, N, 4), 0
    slots = np.full((len(lens), wide), -1, np.int64)
    for i, n in enumerate(lens):
        slots[i, :n] = flat[at: at + n]
        at += n
    slots[0, 2400] = slots[0, 39]                       # the last token far behind the one before
    slots[0, 39] = -1
    slots[4, [600, 1200, 1800]] = slots[4, [3, 4, 5]]   # tokens 3, 4, 5 of the second block, and no other
    slots[4, 3: 17] = -1
    slots = slots.reshape(-1)
    host = empty(N, Hkv, bs, d)
    on = dev(*host)
    T = len(slots)
    kn, vn = rows(T, Hkv, d, dtype, 1), rows(T, Hkv, d, dtype, 2)
    both(fmt, kn, vn, slots, on, host)
    same(on, host)
    assert binding.pa_check_device_errors() == 0


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("T,bs,Hkv,d", [(1, 8, 1, 64), (77, 16, 3, 128), (1001, 32, 4, 64), (6000, 16, 8, 128)])
def test_read_back_bit_exact(fmt, T, bs, Hkv, d):
    N = T // bs + 5
    c = cache(N, Hkv, bs, d, fmt, T, spread=5)
    rng = np.random.default_rng(T)
    slots = rng.integers(0, N * bs, T)
    slots[2::9] = -1
    on = dev(*c)
    for dtype in (F16, BF16):
        ko, vo = (torch.full((T, Hkv, d), 0.5, dtype=dtype, device="cuda") for _ in "kv")
        GATHER[fmt](*on, torch.from_numpy(slots).cuda(), ko, vo)
        live = slots >= 0
        for out, codes, scale in ((ko, c[0], c[2]), (vo, c[1], c[3])):
            want = torch.full((T, Hkv, d), 0.5, dtype=dtype)
            # fl32(code scale), then one rounding to 16 bits: a code has 8 bits, a scale 24
            val = o.gather(codes, scale, slots[live], fmt).astype(np.float32)
            want[torch.from_numpy(live)] = torch.from_numpy(val).to(dtype)
            assert torch.equal(out.cpu().view(torch.int16), want.view(torch.int16))
    assert binding.pa_check_device_errors() == 0
    slots[0] = N * bs
    GATHER[fmt](*on, torch.from_numpy(slots).cuda(), ko, vo)
    assert binding.pa_check_device_errors() == binding.DEVERR["SLOT"]


def check_decode(fmt, lens, H, Hkv, d, bs, dtype, c=None, seed=0, mag=1.0, shift=0.0, spread=0, scale=None,
                 q=None, tbl=None):
    B = len(lens)
    if tbl is None:
        tbl, N = rand_tables(lens, bs, seed)
    else:
        N = int(tbl.max()) + 1
    c = cache(N, Hkv, bs, d, fmt, seed + 1, mag, shift, spread) if c is None else c
    behind(c, lens, tbl, bs)
    q = wl.normal_tensor((B, H, d), dtype, seed + 2) if q is None else q
    scale = d ** -0.5 if scale is None else scale
    out = torch.full((B, H, d), 7.0, dtype=dtype, device="cuda")
    ws = workspace(B, H, d)
    on = dev(*c)
    dt, dl = dev(tbl, np.asarray(lens, np.int32))
    for _ in range(2):
        DECODE[fmt](q.cuda(), *on, dt, dl, max([*lens, 1]), scale, out, ws)
    assert binding.pa_check_device_errors() == 0
    qn = q.double().numpy()
    ref = o.decode(qn, *c, tbl, lens, scale, fmt)
    got = out.double().cpu().numpy()
    bound = decode_bound(qn, c, tbl, lens, scale, dtype, ref, fmt)
    bad = ~(np.abs(got - ref) <= bound)
    assert not bad.any(), (bad.sum(), (np.abs(got - ref) / bound)[bad][:5], got[bad][:5], ref[bad][:5])


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("lens,H,Hkv,d,bs,dtype", [
    ([1], 1, 1, 64, 8, F16), ([1], 1, 1, 128, 32, BF16), ([5, 0, 33], 4, 2, 64, 16, F16),
    ([0, 0], 4, 4, 128, 16, BF16), ([32, 31, 64, 65], 3, 3, 128, 8, F16), ([100, 7, 300], 14, 2, 128, 16, BF16),
    ([257, 1], 8, 1, 64, 32, F16), ([513], 16, 1, 128, 16, F16), ([130, 300, 2, 511], 24, 2, 64, 8, BF16),
    ([777, 12], 32, 2, 128, 32, F16), ([1500], 64, 2, 64, 16, BF16), ([40] * 60, 5, 5, 128, 16, F16)])
def test_decode(fmt, lens, H, Hkv, d, bs, dtype):
    check_decode(fmt, lens, H, Hkv, d, bs, dtype)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("d,bs,G,dtype", [(128, 16, 1, F16), (128, 16, 4, BF16), (64, 8, 7, F16), (128, 32, 16, BF16),
                                          (64, 16, 2, BF16)])
def test_decode_long(fmt, d, bs, G, dtype):
    check_decode(fmt, [5003, 9000, 1, 2048], 2 * G, 2, d, bs, dtype, shift=0.5)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("bs", [8, 16, 32])
def test_decode_scales_far_apart(fmt, bs):
    """Blocks 2^-12 .. 2^12 apart; softmax rows from flat to nearly one-hot."""
    check_decode(fmt, [400, 900], 8, 2, 128, bs, F16, spread=6, scale=0.02)
    check_decode(fmt, [400, 900], 8, 2, 64, bs, BF16, spread=12, scale=1e-4)
    check_decode(fmt, [400, 900], 2, 2, 64, bs, BF16, scale=3.0)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("G", [1, 4, 8])
@pytest.mark.parametrize("order", [1, -1])
def test_decode_v_scales_from_tiny_to_huge(fmt, G, order):
    """V scales rise (or fall) from 2^-60 to 2^60 along the context; the heavy keys are those of the
    smallest scale in one half of the heads, spread over all in the other."""
    n, d, bs, Hkv = 512, 64, 16, 2
    tbl = np.random.default_rng(0).permutation(n // bs)[None].astype(np.int32)
    c = cache(n // bs, Hkv, bs, d, fmt, 5)
    e = np.linspace(-60, 60, n // bs)[::order].round()
    for j, b in enumerate(tbl[0]):
        c[3][b] = np.float32(2.0 ** e[j])
    q = wl.normal_tensor((1, G * Hkv, d), BF16, 6)
    check_decode(fmt, [n], G * Hkv, Hkv, d, bs, BF16, c=c, q=q, tbl=tbl)
    small = tbl[0, 0 if order == 1 else -1]
    c[2][:] = np.float32(2.0) ** -12                     # keys that say nothing but in the small block
    c[0][small] = c[0][small, :, :1]
    c[2][small] = 1.0
    k = o.values(c[0], c[2], fmt)[small, :, 0]
    q = torch.from_numpy(np.repeat(k, G, 0)[None] * 0.05).to(BF16)
    check_decode(fmt, [n], G * Hkv, Hkv, d, bs, BF16, c=c, q=q, tbl=tbl, scale=1.0)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("G", [1, 4, 8, 16])
@pytest.mark.parametrize("e", [-60, -20, 30])
def test_decode_small_v_scale_with_all_the_weight(fmt, G, e):
    """One block of each context has all the weight (the others' logits are 512 lower: their weights are
    0 in fp32) and a V scale 2^e times theirs: the result is as exact as if it stood alone."""
    B, Hkv, bs, d, n = 150, 2, 16, 64, 272
    nb = n // bs
    rng = np.random.default_rng(G)
    c = cache(B * nb, Hkv, bs, d, fmt, 5)
    one = o.encode(np.float32(1), fmt)
    c[0][:] = o.encode(np.float32(-1), fmt)
    c[2][:] = 4.0
    c[3][:] = 2.0 ** -5
    tbl = rng.permutation(B * nb).reshape(B, nb).astype(np.int32)
    heavy = rng.integers(0, nb, B)
    at = tbl[np.arange(B), heavy]
    c[0][at] = one
    c[3][at] = np.float32(2.0 ** (e - 5))
    q = torch.ones(B, G * Hkv, d, dtype=BF16)
    out = torch.empty(B, G * Hkv, d, dtype=BF16, device="cuda")
    DECODE[fmt](q.cuda(), *dev(*c), *dev(tbl, np.full(B, n, np.int32)), n, 1.0, out, workspace(B, G * Hkv, d))
    assert binding.pa_check_device_errors() == 0
    v = o.values(c[1], c[3], fmt)[at]                    # [B, Hkv, bs, d], equal weights
    ref, mag = (np.repeat(x, G, 1) for x in (v.mean(2), np.abs(v).mean(2)))
    # the output's rounding, P's two parts (2^-16), sums of a few dozen steps (2^-22 each) of codes from 128 on
    bound = 2.0 ** -8 * np.abs(ref) + 2.0 ** -16 * mag + 64 * 2.0 ** -22 * (mag + 128 * 2.0 ** (e - 5) * (fmt == "int8"))
    assert (np.abs(out.double().cpu().numpy() - ref) <= bound).all()


@pytest.mark.parametrize("fmt", FMTS)
def test_decode_zero_scales_and_all_codes(fmt):
    c = cache(12, 2, 16, 64, fmt, 3)
    c[3][::2] = 0.0
    c[2][::3] = 0.0
    b = np.arange(256, dtype=np.uint8)
    if fmt == "fp8":
        b[b & 127 == 127] = 0
    c[0][5, 0].reshape(-1)[:256] = b
    c[1][5, 1].reshape(-1)[:256] = b
    check_decode(fmt, [180], 4, 2, 64, 16, F16, c=c, tbl=np.arange(12, dtype=np.int32)[None])
    c[3][:] = 0.0
    check_decode(fmt, [180], 4, 2, 64, 16, BF16, c=c, tbl=np.arange(12, dtype=np.int32)[None])


@pytest.mark.parametrize("fmt", FMTS)
def test_decode_reports_bad_tables(fmt):
    lens, bs, Hkv, H, d = [40, 33, -3, 100], 16, 2, 4, 64
    tbl = np.array([[0, 99, 2], [3, -7, 5], [0, 0, 0], [1, 4, 6]], np.int32)     # 100 tokens need 7 blocks
    c = cache(8, Hkv, bs, d, fmt, 1)
    q = wl.normal_tensor((4, H, d), F16, 2)
    out = torch.empty(4, H, d, dtype=F16, device="cuda")
    DECODE[fmt](q.cuda(), *dev(*c), *dev(tbl, np.asarray(lens, np.int32)), 100, 0.125, out, workspace(4, H, d))
    e = binding.DEVERR
    assert binding.pa_check_device_errors() == e["BLOCK_ID"] | e["CONTEXT"] | e["TABLE_WIDTH"]
    cut = [40, 33, 0, 48]
    ref = o.decode(q.double().numpy(), *c, tbl, cut, 0.125, fmt)
    bound = decode_bound(q.double().numpy(), c, tbl, cut, 0.125, F16, ref, fmt)
    assert (np.abs(out.double().cpu().numpy() - ref) <= bound).all()
