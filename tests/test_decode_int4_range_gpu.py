"""pa_decode_int4 over caches whose V steps differ by many powers of two.

K rows are constant (step 0), so a key's base-2 logit is exactly what the test asks for and every
weight is known; V's steps are set per group, per token and per head's weight.  The bound is taken
group by group and head by head: what a token of negligible weight, another group or another query
head holds must not cost a group its codes."""
import numpy as np
import pytest
import torch

from oracle import cache4 as o
from paged_kv_cache_103_gb300 import binding

from _cache4 import dev, workspace

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from paged_kv_cache_103_gb300 import build
    build.build()
    binding.load()


def make_case(logits, steps, H, d, bs, seed):
    """One sequence of one KV head.  logits: base-2 logits [n, c], one column per set of heads (at
    most one set per group of 64 channels: set c's heads have ones in group c and zeros elsewhere,
    one column: ones everywhere); steps [n, d / 64] of V.  Codes are random and V's minimum is -8
    steps, so values lie around zero.  -> q, cache, table, scale."""
    rng = np.random.default_rng(seed)
    n, sets = logits.shape
    nb, NG = -(-n // bs), d // 64
    N = nb + 2
    tbl = rng.permutation(N)[:nb].astype(np.int32)[None]
    kc, vc = (rng.integers(0, 256, (N, 1, bs, d // 2)).astype(np.uint8) for _ in "kv")
    ks, vs = (np.zeros((N, 1, bs, NG, 2), np.float16) for _ in "kv")
    q = np.zeros((1, H, d), np.float32)
    if sets == 1:
        q[:] = 1
    else:
        for h in range(H):
            c = h * sets // H
            q[0, h, 64 * c: 64 * c + 64] = 1
    per = d if sets == 1 else 64                  # ones in q
    for t in range(n):
        b, r = tbl[0, t // bs], t % bs
        for g in range(NG):
            ks[b, 0, r, g, 1] = logits[t, 0 if sets == 1 else g]
            vs[b, 0, r, g] = steps[t, g], -8 * steps[t, g]
    return q, [kc, vc, ks, vs], tbl, float(np.log(2) / per)


def group_bound(q, cache, tbl, n, scale, dtype, ref):
    """Largest |gpu - ref| per output element, from each head's and group's own weights.

    With w the exact weights and a_j = 15 s_j + |m_j| of the element's group:
    * one rounding of the output: eps / 2 of |ref|, or half the smallest subnormal;
    * P in two bf16 parts, the first toward zero: 2^-16 of sum_j w_j s_j |c_j - 8|;
    * a weight is a sum of at most 8 fp32 roundings of a logit of size x (2^-24 |x| each, times
      ln 2, both in w and in the sum that divides), exp2 (2^-22) and three fp32 products: below
      2^-19 + 2^-20 |x|;
    * the sums over the keys, on the tensor cores (16 keys at a time, the two parts one after the
      other, each sum cut off 2^-23 of the largest partial sum at worst, which the weight of the
      chunks between two subtractions of the codes' middle bounds, eight at most): 32 of them for P's
      codes and 32 for the eights, and one rounding of what is left per subtraction; the
      minima in fp32, each lane every eighth key, n / 8 roundings of 2^-24; the joins, 64 of 2^-24:
      (64 + 32 + n / 16) 2^-23 of sum_j w_j a_j.
    """
    kc, vc, ks, vs = cache
    _, H, d = q.shape
    t = np.arange(n)
    bs = kc.shape[2]
    at = tbl[0][t // bs].astype(np.int64) * bs + t % bs
    k = o.gather_int4(kc, ks, at)[:, 0]
    v = o.gather_int4(vc, vs, at)[:, 0]
    s = np.repeat(vs[at // bs, 0, at % bs, :, 0].astype(np.float64), 64, -1)
    m = np.repeat(vs[at // bs, 0, at % bs, :, 1].astype(np.float64), 64, -1)
    off, amp = np.abs(v - m - 8 * s), 15 * s + np.abs(m)
    fin = torch.finfo(dtype)
    bound = np.maximum(fin.eps / 2 * np.abs(ref), fin.smallest_normal * fin.eps / 2)
    for h in range(H):
        x = (k @ q[0, h].astype(np.float64)) * scale
        w = np.exp(x - x.max())
        w /= w.sum()
        size = np.abs(x / np.log(2)).max()
        rel = 2.0 ** -19 + 2.0 ** -20 * size + (96 + n / 16) * 2.0 ** -23
        bound[0, h] += 2.0 ** -16 * (w @ off) + rel * (w @ amp)
    return bound


def run(q, cache, tbl, n, scale, dtype, B):
    """B sequences, all of them the same one: a long list, so that a warp walks many chunks."""
    _, H, d = q.shape
    out = torch.full((B, H, d), float("nan"), dtype=dtype, device="cuda")
    binding.pa_decode_int4(torch.from_numpy(q).to(dtype).cuda().repeat(B, 1, 1), *dev(*cache),
                           *dev(tbl.repeat(B, 0), np.full(B, n, np.int32)), n, scale, out, workspace(B, H, d))
    assert binding.pa_check_device_errors() == 0
    return out.cpu().double().numpy()


def flat(n, x=0.0):
    return np.full((n, 1), x)


def scenario(name, d, rng):
    """(logits, steps): n tokens, most of them of weight 2^-12 and step 0.01."""
    n, NG = 4097, d // 64
    steps = np.full((n, NG), 0.01)
    logits = flat(n, -12.0)
    if name == "groups":               # the top key's step, in one group only
        logits[40], steps[40, 0] = 0, 4000
    elif name == "first":              # a huge step of no weight, before and behind all others
        logits[0], steps[0], logits[2000] = -40, 4000, 0
    elif name == "last":
        logits[-1], steps[-1], logits[2000] = -40, 4000, 0
    elif name == "heads":              # half of the heads see the huge step, the others do not
        logits = np.concatenate([flat(n, -12.0), flat(n, -12.0)], 1)
        logits[7], steps[7] = (0, -60), 4000
        logits[2000, 1] = 0
    elif name == "rising":             # every chunk raises the maximum, steps fall by the way
        logits = (np.arange(n)[:, None] // 32 * 9).astype(np.float64) - 600
        steps = np.exp2(11 - np.arange(n)[:, None] // 32 * 0.25).repeat(NG, 1)
    elif name == "falling":
        logits = 500 - (np.arange(n)[:, None] // 32 * 9).astype(np.float64)
        steps = np.exp2(-20 + np.arange(n)[:, None] // 32 * 0.25).repeat(NG, 1)
    elif name == "zero":               # the top key's step is 0: only the small weights have codes
        logits[9], steps[9] = 0, 0
        steps[10:] = 2.0 ** -20
    elif name == "mixed":
        logits = rng.integers(-30, 1, (n, 1)).astype(np.float64)
        steps = np.exp2(rng.uniform(-20, 11, (n, NG)))
    elif name == "jump":               # one raise of the maximum by more than fp32's exponents
        logits[:], logits[2000:] = -300, 100
        steps[2000:] = 0.5
    return logits, steps


SCENARIOS = ["groups", "first", "last", "heads", "rising", "falling", "zero", "mixed", "jump"]


SHAPES = [(1, 128, 16, torch.float16), (4, 128, 16, torch.bfloat16), (7, 128, 32, torch.float16),
          (16, 128, 8, torch.float16), (2, 64, 16, torch.float16), (12, 64, 32, torch.bfloat16)]


# (two sets of heads need two heads and two groups)
@pytest.mark.parametrize("name,H,d,bs,dtype", [(name, *shape) for name in SCENARIOS for shape in SHAPES
                                               if name != "heads" or shape[0] > 1 and shape[1] == 128])
def test_steps_of_very_different_size(name, H, d, bs, dtype):
    logits, steps = scenario(name, d, np.random.default_rng(H))
    n = len(logits)
    q, cache, tbl, scale = make_case(logits, steps, H, d, bs, H + d)
    ref = o.decode_int4(q.astype(np.float64), *cache, tbl, [n], scale)
    bound = group_bound(q, cache, tbl, n, scale, dtype, ref)
    for B in (1, 2500):
        err = np.abs(run(q, cache, tbl, n, scale, dtype, B) - ref)
        assert (err <= bound).all(), "%d: worst %.3g of its bound" % (B, (err / bound).max())


def rms(x):
    return float(np.sqrt(np.mean(np.square(x))))


@pytest.mark.parametrize("H,Hkv,d", [(1, 1, 128), (3, 1, 128), (7, 1, 64), (8, 1, 128), (13, 1, 128)])
@pytest.mark.parametrize("n,B,limit", [(60, 40, 1.05), (32769, 2500, 1.25)])
def test_an_f16_result_is_off_by_little_but_its_own_rounding(n, B, limit, H, Hkv, d):
    """Weights that f16 does not hold, and runs of 1000 chunks a warp.  Root mean squares, r that of
    the output's rounding (known from the reference; some 2^-12.3 of the result):
    * short contexts: with x = sum_j (w_j s_j (c_j - 8))^2 the result is of size sqrt(x), and P's
      second part is off by 2^-17.8 of each product, together 2^-17.8 sqrt(x): r / 45, and the
      fp32 steps less: 5% is ample;
    * long ones: with a = sum_j w_j 8 s_j, the result is some a / 300 and r 2^-20.5 a; of the 32 sums at
      most between two subtractions, of the codes and of the eights, each cuts half a unit of 2^-23 on
      average, alike but where one of the two lies beyond a power of two: (1/2) 32 / 2 of 2^-24 a
      = 2^-21 a where it does, and its deviation, 2^-23 a, averages out over the subtractions:
      at most sqrt(1 + (3/4)^2) = 1.25 r.
    """
    rng = np.random.default_rng(n + H)
    logits = -rng.integers(0, 24, (n, 1)) / 32 if n < 100 else np.zeros((n, 1))
    steps = rng.uniform(0.2, 0.3, (n, d // 64))
    q, cache, tbl, scale = make_case(logits, steps, H, d, 16, H)
    ref = o.decode_int4(q.astype(np.float64), *cache, tbl, [n], scale)
    got = run(q, cache, tbl, n, scale, torch.float16, B)
    r = rms(ref.astype(np.float16).astype(np.float64) - ref)
    assert rms(got - ref) <= limit * r, "%.3f" % (rms(got - ref) / r)
