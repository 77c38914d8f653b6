"""Operators of the block-scaled 8-bit KV cache and of eviction, as cases that can be timed.

Five operators over the paged cache:

* ``write``   append new tokens' K/V to a cache of 8-bit codes with one scale per (block, KV head),
  which rescales the block's earlier rows where its scale grows, and read the blocks back;
* ``read``    read tokens of such a cache back into 16 bits;
* ``decode``  one query token per sequence over such a cache;
* ``weigh``   one query token per sequence over the 16-bit cache, each token's softmax weights added
  to an accumulator per (sequence, KV head);
* ``evict``   keep the first, the last and the heaviest tokens of each (sequence, KV head) and move
  them together.

``run`` computes a case with elementary torch operations in 32 bits, or, where ``own`` is true,
with the library's kernels.  A code is an INT8 integer (``TOP`` 127) or an E4M3 number (448) and stands
for ``code * scale``.  An append to a block takes ``a``, the largest magnitude of the rows that it
writes there; the scale becomes ``s = max(s_old, a / TOP)``, with ``s_old`` as 0 if row 0 is among the
rows written; the new rows' codes are ``round(x / s)``, and if ``0 < s_old < s`` the other rows' become
``round(code * (s_old / s))``.
"""
import math
import random

import torch

own = False

DTYPES = {"f16": torch.float16, "bf16": torch.bfloat16}
TOP = {"int8": 127.0, "fp8": 448.0}


# ------------------------------------------------------------------------------------ cases
def listed():
    return [
        # one decode step's append: 64 sequences of a 40-head (MHA) model, one token each
        dict(name="write_step", kind="write", fmt="int8", T=64, seqs=64, Hkv=40, d=128, bs=16, dtype="f16",
             pad=0),
        # a prefill step's append: four chunks of about 2048 tokens that begin inside a block, 8 KV
        # heads, some padding
        dict(name="write_prompt", kind="write", fmt="fp8", T=8192, seqs=4, Hkv=8, d=128, bs=16, dtype="bf16",
             pad=100),
        # an odd number of tokens in large blocks, a small head: a short chunk's context
        dict(name="read_chunk", kind="read", fmt="fp8", T=1001, Hkv=4, d=64, bs=32, dtype="f16", pad=37),
        # the context of a chunked prefill (4 x 8192 tokens) read back for the 16-bit kernels
        dict(name="read_context", kind="read", fmt="int8", T=32768, Hkv=8, d=128, bs=16, dtype="bf16", pad=0),
        # the smallest batch: latency
        dict(name="decode_tiny", kind="decode", fmt="fp8", B=4, H=4, Hkv=2, d=64, bs=16, dtype="f16",
             lens="uniform", lo=1, n=64, empty=0),
        # 64 sequences of a 40-head (MHA) model, U[128, 2048] tokens
        dict(name="decode_mha_64", kind="decode", fmt="int8", B=64, H=40, Hkv=40, d=128, bs=16, dtype="f16",
             lens="uniform", lo=128, n=2048, empty=0),
        # the largest: 16 sequences of 32768 tokens, 32 / 8 heads
        dict(name="decode_gqa4_32k", kind="decode", fmt="fp8", B=16, H=32, Hkv=8, d=128, bs=16, dtype="bf16",
             lens="full", lo=0, n=32768, empty=0),
        # long-tailed lengths, 7 query heads a KV head, large blocks, two empty sequences
        dict(name="weigh_gqa7_tail", kind="weigh", B=32, H=28, Hkv=4, d=128, bs=32, dtype="bf16",
             lens="tail", lo=1, n=24576, empty=2),
        # 64 sequences of a 40-head (MHA) model, U[128, 2048] tokens
        dict(name="weigh_mha_64", kind="weigh", B=64, H=40, Hkv=40, d=128, bs=16, dtype="f16",
             lens="uniform", lo=128, n=2048, empty=0),
        # 16 sequences of 16384 tokens, 32 / 8 heads
        dict(name="weigh_gqa4_16k", kind="weigh", B=16, H=32, Hkv=8, d=128, bs=16, dtype="bf16",
             lens="full", lo=0, n=16384, empty=0),
        # a few conversations cut to an odd budget, some within it, shared blocks replaced by new ones
        dict(name="evict_few", kind="evict", B=5, Hkv=4, d=64, bs=8, dtype="f16", lens="uniform", lo=100,
             n=1000, empty=1, keep=301, first=4, last=60, fresh=3),
        # 32 contexts of 8192 tokens cut in half, in place
        dict(name="evict_half", kind="evict", B=32, Hkv=8, d=128, bs=16, dtype="bf16", lens="full", lo=0,
             n=8192, empty=0, keep=4096, first=4, last=512, fresh=0),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    """One more case over the ranges of the listed ones."""
    kind = rng.choice(["write", "write", "read", "decode", "decode", "decode", "weigh", "weigh", "evict", "evict"])
    d = rng.choice([64, 128, 128])
    bs = rng.choice([8, 16, 32])
    dtype = rng.choice(["f16", "bf16"])
    fmt = rng.choice(["int8", "fp8"])
    Hkv = rng.choice([1, 2, 4, 5, 8, 40])
    if kind == "write":
        seqs = _log(rng, 1, 64)
        T = seqs * _log(rng, 1, max(1, 65536 // (Hkv * seqs)))
        return dict(kind=kind, fmt=fmt, T=T, seqs=seqs, Hkv=Hkv, d=d, bs=bs, dtype=dtype,
                    pad=rng.randrange(0, T // 4 + 1))
    if kind == "read":
        T = _log(rng, 1, 262144 // Hkv)
        return dict(kind=kind, fmt=fmt, T=T, Hkv=Hkv, d=d, bs=bs, dtype=dtype, pad=rng.randrange(0, T // 4 + 1))
    Hkv = rng.choice([1, 2, 4, 5, 8])
    most = {"decode": 2000000, "weigh": 1000000, "evict": 1000000}[kind]
    n = _log(rng, 64 if kind == "evict" else 1, 32768 if kind == "decode" else 16384)
    B = _log(rng, 1, max(1, min(128, most // (n * Hkv))))
    c = dict(kind=kind, B=B, Hkv=Hkv, d=d, bs=bs, dtype=dtype, lens=rng.choice(["full", "uniform", "tail"]),
             lo=rng.randrange(1, n + 1), n=n, empty=rng.randrange(0, B // 8 + 1))
    if kind == "evict":
        first, last = rng.randrange(0, 8), rng.randrange(0, n // 8 + 1)
        c.update(first=first, last=last, keep=rng.randrange(max(1, first + last), n + 1), fresh=rng.randrange(0, 5))
        return c
    c["H"] = Hkv * rng.choice([1, 2, 3, 4, 7, 8, 12, 16])
    if kind == "decode":
        c["fmt"] = fmt
    return c


# ----------------------------------------------------------------------------------- inputs
def _lens(case, gen):
    """Context lengths (host): all n, uniform in [lo, n], or lognormal (median n / 16) with one
    sequence in sixteen at two thirds of n or more; ``empty`` of them are 0."""
    B, n, lo = case["B"], case["n"], case["lo"]
    u = torch.rand(B, generator=gen, dtype=torch.float64)
    if case["lens"] == "full":
        lens = torch.full((B,), n)
    elif case["lens"] == "uniform":
        lens = lo + (u * (n - lo + 1)).long()
    else:
        z = torch.randn(B, generator=gen, dtype=torch.float64)
        lens = ((z + math.log(max(n / 16, 1))).exp().round().long()).clamp(1, max(n // 3, 1))
        lens[::16] = (2 * n // 3) + (u[::16] * (n - 2 * n // 3 + 1)).long()
    lens = lens.clamp(max=n)
    if case["empty"]:
        lens[torch.randperm(B, generator=gen)[: case["empty"]]] = 0
    return lens


def _normal(shape, dtype, gen, channels=False):
    """N(0, 1) values; with ``channels`` a few head-dim channels are shifted and widened, as keys
    have them."""
    x = torch.empty(shape, dtype=dtype, device="cuda")
    flat = x.view(-1, shape[-1])
    step = 1 << 20
    d = shape[-1]
    wide = 1 + 3 * (torch.rand(d, generator=gen, device="cuda") < 0.06).float()
    shift = 2 * torch.randn(d, generator=gen, device="cuda") * (wide > 1)
    for a in range(0, flat.shape[0], step):
        y = torch.randn(flat[a: a + step].shape, generator=gen, device="cuda")
        flat[a: a + step] = (y * wide + shift if channels else y).to(dtype)
    return x


def _paged(lens, bs, hgen, spare=0, most=0):
    """A pool of 1.25 x the blocks that the lengths need (that ``len(lens)`` sequences of ``most``
    tokens need) and ``spare`` more, handed out in random order."""
    nb = (lens + bs - 1) // bs
    N = max(1, math.ceil(1.25 * (len(lens) * ((most + bs - 1) // bs) if most else int(nb.sum())))) + spare
    width = max(1, int(nb.max()))
    order = torch.randperm(N, generator=hgen)
    col = torch.arange(width)
    idx = (nb.cumsum(0) - nb)[:, None] + col
    tables = torch.where(col < nb[:, None], order[idx.clamp(max=N - 1)], torch.tensor(-1)).int()
    # (block, row) of the slots behind each sequence's last token
    seq, r = torch.meshgrid(torch.arange(len(lens)), torch.arange(bs), indexing="ij")
    last = tables.gather(1, (nb - 1).clamp(min=0)[:, None]).expand(-1, bs)
    behind = (lens[:, None] > 0) & (r >= ((lens - 1) % bs + 1)[:, None])
    return dict(lens=lens.int().cuda(), tables=tables.cuda(), N=N, max_len=int(lens.max()), tokens=int(lens.sum()),
                free=order[int(nb.sum()):], behind=(last[behind].cuda().long(), r[behind].cuda()))


def _const(v):
    """A divisor on the GPU: dividing by a host number multiplies by its rounded reciprocal."""
    return torch.full((), v, device="cuda")


def _codes(x, fmt):
    """fp32 quotients -> the nearest codes (uint8 bytes)."""
    if fmt == "int8":
        return x.round().clamp(-127, 127).to(torch.int8).view(torch.uint8)
    return x.clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)


def _numbers(codes, fmt):
    """Code bytes -> the fp32 numbers that they are."""
    return codes.view(torch.int8 if fmt == "int8" else torch.float8_e4m3fn).float()


def _divide(x, s):
    """x / s, 0 where s is 0."""
    return torch.where(s > 0, x / torch.where(s > 0, s, torch.ones_like(s)), torch.zeros_like(x))


def _cache8(N, Hkv, bs, d, fmt, dtype, gen, channels):
    """A cache whose blocks were quantised whole: codes [N, Hkv, bs, d], scales [N, Hkv]."""
    codes = torch.empty(N, Hkv, bs, d, dtype=torch.uint8, device="cuda")
    scale = torch.empty(N, Hkv, dtype=torch.float32, device="cuda")
    step = max(1, (1 << 26) // (Hkv * bs * d))
    for a in range(0, N, step):
        n = min(step, N - a)
        x = _normal((n, Hkv, bs, d), dtype, gen, channels).float()
        s = x.abs().amax((-1, -2)) / _const(TOP[fmt])
        codes[a: a + n], scale[a: a + n] = _codes(_divide(x, s[..., None, None]), fmt), s
    return codes, scale


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(int(seed))
    hgen = torch.Generator().manual_seed(int(seed))
    kind, dt = case["kind"], DTYPES[case["dtype"]]
    Hkv, d, bs = case["Hkv"], case["d"], case["bs"]
    st = dict(case=dict(case), scale=d ** -0.5)
    if kind in ("write", "read"):
        T, fmt = case["T"], case["fmt"]
        if kind == "write":
            # each sequence appends T / seqs tokens behind 0 .. bs - 1 that its last block holds
            seqs = case["seqs"]
            held = torch.randint(0, bs, (seqs,), generator=hgen)
            p = _paged(held + T // seqs, bs, hgen, spare=1, most=bs - 1 + T // seqs)
            pos = held[:, None] + torch.arange(T // seqs)
            table = p["tables"].cpu().long()
            slots = (table.gather(1, pos // bs) * bs + pos % bs).flatten()
            N = p["N"]
            if case["pad"]:
                slots[torch.randperm(T, generator=hgen)[: case["pad"]]] = -1
            st.update(k_new=_normal((T, Hkv, d), dt, gen, True), v_new=_normal((T, Hkv, d), dt, gen),
                      spare=int(p["free"][0]))
            # read back: every row up to the last appended one
            pos = torch.arange(bs - 1 + T // seqs)
            back = table.gather(1, (pos // bs).clamp(max=table.shape[1] - 1).expand(seqs, -1)) * bs + pos % bs
            st["back"] = torch.where(pos < (held + T // seqs)[:, None], back, torch.tensor(-1)).flatten().cuda()
        else:
            # a context's blocks lie all over the pool, the tokens of a block one behind the other
            N = math.ceil(1.25 * T / bs) + 1
            pos = torch.arange(T)
            slots = torch.randperm(N, generator=hgen)[pos // bs] * bs + pos % bs
            if case["pad"]:
                slots[torch.randperm(T, generator=hgen)[: case["pad"]]] = -1
        st["slots"] = slots.cuda()
        for x in "kv":
            st[x + "_cache"], st[x + "_scale"] = _cache8(N, Hkv, bs, d, fmt, dt, gen, x == "k")
            rows = st["back" if kind == "write" else "slots"].numel()
            st[x + "_out"] = torch.full((rows, Hkv, d), 0.5, dtype=dt, device="cuda")
        return st
    B = case["B"]
    lens = _lens(case, hgen)
    st.update(_paged(lens, bs, hgen, spare=1 + B * case.get("fresh", 0), most=case["n"] if kind == "evict" else 0))
    blk, row = st.pop("behind")
    free = st.pop("free")
    N = st["N"]
    if kind == "decode":
        for x in "kv":
            st[x + "_cache"], st[x + "_scale"] = _cache8(N, Hkv, bs, d, case["fmt"], dt, gen, x == "k")
            st[x + "_cache"][blk, :, row] = 0x7F          # slots that nothing was written to (an E4M3 NaN)
            st[x + "_scale"][free.cuda()] = float("nan")  # blocks that nothing was written to
    else:
        for x in "kv":
            st[x + "_cache"] = _normal((N, bs, Hkv, d), dt, gen, x == "k")
            if kind == "weigh":
                st[x + "_cache"][blk, row] = float("nan")
        # the accumulators of a server's sequences, B of them in this batch
        R, W = B + 3, case["n"] + 17
        at = torch.arange(W, device="cuda")
        u = torch.rand(R, Hkv, W, generator=gen, device="cuda")
        w = -u.clamp(min=1e-6).log() * (32.0 / max(case["n"], 1))
        # a token's weight falls with its age, a few tokens draw most of it
        w = w * torch.where(u < 0.02, 40.0, 1.0) * (1 - 0.5 * at / W)
        rows = torch.randperm(R, generator=hgen)[:B]
        st["rows"] = rows.int().cuda()
        full = torch.zeros(R, dtype=torch.long)
        full[rows] = lens
        w[at >= full.cuda()[:, None, None].expand_as(w)] = 0
        st["weights"] = w
    if kind in ("decode", "weigh"):
        st["q"] = _normal((B, case["H"], d), dt, gen)
        st["out"] = torch.empty_like(st["q"])
        return st
    # the table that the kept tokens go to: the same blocks, but for new ones in the place of the
    # first ``fresh``, which other sequences share
    keep = case["keep"]
    width = (keep + bs - 1) // bs
    dst = torch.full((B, width), -1, dtype=torch.int32)
    old = st["tables"].cpu()[:, :width]
    dst[:, : old.shape[1]] = old
    new = min(case["fresh"], width, old.shape[1])
    nb = (lens.clamp(max=keep) + bs - 1) // bs
    dst[:, :new] = torch.where(torch.arange(new) < nb[:, None], free[1: 1 + B * new].view(B, new).int(), dst[:, :new])
    st.update(new_tables=dst.cuda(), spare=int(free[0]),
              kept=torch.empty(B, Hkv, keep, dtype=torch.int32, device="cuda"),
              kept_lens=torch.empty(B, dtype=torch.int32, device="cuda"),
              new_weights=torch.zeros_like(st["weights"]))
    return st


# ------------------------------------------------------------------------------ plain forms
def _plain_gather(st, slots):
    c = st["case"]
    bs, ok, at = c["bs"], slots >= 0, slots.clamp(min=0)
    outs = []
    for x in "kv":
        val = _numbers(st[x + "_cache"][at // bs, :, at % bs], c["fmt"]) * st[x + "_scale"][at // bs][..., None]
        outs.append(torch.where(ok[:, None, None], val.to(st[x + "_out"].dtype), st[x + "_out"]))
    return outs


def _plain_write(st):
    c = st["case"]
    bs, fmt, slots = c["bs"], c["fmt"], st["slots"]
    ok = slots >= 0
    # padding tokens go to a block that nothing holds
    at = torch.where(ok, slots, torch.full_like(slots, st["spare"] * bs))
    blk, row = at // bs, at % bs
    live = ok[:, None].float()
    N = st["k_cache"].shape[0]
    zero = torch.zeros(N, device="cuda")
    touched = zero.index_reduce(0, blk, ok.float(), "amax")[:, None] > 0
    fresh = zero.index_reduce(0, blk, (ok & (row == 0)).float(), "amax")[:, None] > 0
    for x in "kv":
        new, cache, scale = st[x + "_new"].float(), st[x + "_cache"], st[x + "_scale"]
        a = torch.zeros_like(scale).index_reduce(0, blk, new.abs().amax(-1) * live, "amax")
        old = torch.where(fresh, torch.zeros_like(scale), scale)
        s = torch.where(touched, torch.maximum(old, a / _const(TOP[fmt])), scale)
        grows = touched & (old > 0) & (s > old)
        again = _codes(_numbers(cache, fmt) * _divide(old, s)[..., None, None], fmt)
        cache.copy_(torch.where(grows[..., None, None], again, cache))
        codes = _codes(_divide(new, s[blk][..., None]), fmt)
        cache[blk, :, row] = torch.where(ok[:, None, None], codes, torch.zeros_like(codes))
        scale.copy_(s)
    return [*_plain_gather(st, st["back"]), st["k_scale"], st["v_scale"]]


def _plain_read(st):
    return _plain_gather(st, st["slots"])


def _attend(q, k, v, mask, scale):
    """q [B, Hkv, G, d], k / v [B, L, Hkv, d] fp32, mask [B, L] -> [B, Hkv, G, d] and the softmax
    weights' sum over each KV head's query heads [B, Hkv, L]."""
    s = torch.einsum("bhgd,blhd->bhgl", q, k) * scale
    s = torch.where(mask[:, None, None], s, torch.full_like(s, -math.inf))
    p = (s - s.amax(-1, keepdim=True).clamp(min=-1e30)).exp()
    p = p / p.sum(-1, keepdim=True).clamp(min=1e-30)
    v = torch.where(mask[..., None, None], v, torch.zeros_like(v))
    return torch.einsum("bhgl,blhd->bhgd", p, v), p.sum(2)


def _context(st):
    """Block and row of each position of the longest context, and which positions a sequence has."""
    pos = torch.arange(max(st["max_len"], 1), device="cuda")
    blk = st["tables"].long()[:, pos // st["case"]["bs"]].clamp(min=0)
    return blk, (pos % st["case"]["bs"]).expand_as(blk), pos < st["lens"][:, None]


def _plain_decode(st):
    c = st["case"]
    blk, row, mask = _context(st)
    k, v = (_numbers(st[x + "_cache"][blk, :, row], c["fmt"]) * st[x + "_scale"][blk][..., None] for x in "kv")
    q = st["q"].float().view(c["B"], c["Hkv"], -1, c["d"])
    return _attend(q, k, v, mask, st["scale"])[0].view_as(st["q"]).to(st["q"].dtype)


def _plain_weigh(st):
    c = st["case"]
    blk, row, mask = _context(st)
    k, v = (st[x + "_cache"][blk, row].float() for x in "kv")
    q = st["q"].float().view(c["B"], c["Hkv"], -1, c["d"])
    out, p = _attend(q, k, v, mask, st["scale"])
    L = p.shape[-1]
    st["weights"][st["rows"].long(), :, :L] += p
    return out.view_as(st["q"]).to(st["q"].dtype), st["weights"]


def _plain_evict(st):
    c = st["case"]
    B, Hkv, keep, bs = c["B"], c["Hkv"], c["keep"], c["bs"]
    lens, rows = st["lens"].long(), st["rows"].long()
    w = st["weights"][rows]
    n = lens[:, None, None]
    at = torch.arange(w.shape[-1], device="cuda")
    always = (at < c["first"]) | (at >= n - c["last"]) | (n <= keep)
    key = torch.where(always, torch.full_like(w, math.inf), w)
    key = torch.where(at < n, key, torch.full_like(w, -math.inf))
    best = key.sort(dim=-1, descending=True, stable=True).indices[..., :keep]
    best = torch.where(best < n, best, torch.full_like(best, w.shape[-1])).sort(-1).values
    kept = torch.full((B, Hkv, keep), -1, dtype=torch.int32, device="cuda")
    kept[..., : best.shape[-1]] = torch.where(best < n, best, torch.full_like(best, -1)).int()
    some = kept >= 0
    new = torch.zeros_like(w)
    m = min(keep, w.shape[-1])
    new[..., :m] = torch.where(some[..., :m], w.gather(2, kept[..., :m].long().clamp(min=0)),
                               torch.zeros((), device="cuda"))
    new_weights = st["new_weights"]
    new_weights[rows] = new
    # rows that are not kept go from a block that nothing holds to itself
    spare = torch.full((), st["spare"], device="cuda", dtype=torch.long)
    p = kept.long().clamp(min=0)
    b = torch.arange(B, device="cuda")[:, None, None]
    h = torch.arange(Hkv, device="cuda")[None, :, None].expand_as(p)
    r = torch.arange(keep, device="cuda").expand_as(p)
    src, to = st["tables"].long()[b, p // bs], st["new_tables"].long()[b, r // bs]
    src, to = torch.where(some, src, spare), torch.where(some, to, spare)
    for x in "kv":
        cache = st[x + "_cache"]
        cache[to, r % bs, h] = torch.where(some[..., None], cache[src, p % bs, h], cache[to, r % bs, h])
    return kept, some[:, 0].sum(-1).int(), new_weights, st["k_cache"], st["v_cache"]


PLAIN = dict(write=_plain_write, read=_plain_read, decode=_plain_decode, weigh=_plain_weigh, evict=_plain_evict)


# ------------------------------------------------------------------------ the library's calls
def _workspace(st, size, *sizes):
    """A decode's workspace, which a program allocates and zeroes once."""
    if "ws" not in st:
        st["ws"] = torch.zeros(size(*sizes), dtype=torch.uint8, device="cuda")
    return st["ws"]


def _own(st):
    import paged_kv_cache_103_gb300 as pa
    c = st["case"]
    kind = c["kind"]
    cache = [st[x] for x in ("k_cache", "v_cache", "k_scale", "v_scale") if x in st]
    if kind in ("write", "read"):
        append, read = {"int8": (pa.pa_reshape_and_cache_int8_block, pa.pa_gather_cache_int8_block),
                        "fp8": (pa.pa_reshape_and_cache_fp8_block, pa.pa_gather_cache_fp8_block)}[c["fmt"]]
        if kind == "write":
            append(st["k_new"], st["v_new"], st["slots"], *cache)
        read(*cache, st["back" if kind == "write" else "slots"], st["k_out"], st["v_out"])
        return [st["k_out"], st["v_out"]] + ([st["k_scale"], st["v_scale"]] if kind == "write" else [])
    if kind == "decode":
        decode = {"int8": pa.pa_decode_int8_block, "fp8": pa.pa_decode_fp8_block}[c["fmt"]]
        decode(st["q"], *cache, st["tables"], st["lens"], st["max_len"], st["scale"], st["out"],
               _workspace(st, pa.pa_decode_workspace_size, c["B"], c["H"], c["d"]))
        return st["out"]
    if kind == "weigh":
        pa.pa_decode_weights(st["q"], *cache, st["tables"], st["lens"], st["max_len"], st["scale"], st["out"],
                             st["weights"], st["rows"],
                             _workspace(st, pa.pa_decode_weights_workspace_size, c["B"], c["H"], c["Hkv"], c["d"],
                                        st["tokens"]))
        return st["out"], st["weights"]
    pa.pa_select_tokens(st["weights"], st["rows"], st["lens"], c["first"], c["last"], st["kept"], st["kept_lens"],
                        st["new_weights"])
    pa.pa_compact_tokens(*cache, st["kept"], st["kept_lens"], st["tables"], st["new_tables"])
    return st["kept"], st["kept_lens"], st["new_weights"], *cache


def run(state):
    return _own(state) if own else PLAIN[state["case"]["kind"]](state)


# -------------------------------------------------------------------------------------- work
def work(case):
    """Each input read once, each output written once."""
    kind, Hkv, d, bs = case["kind"], case["Hkv"], case["d"], case["bs"]
    if kind in ("write", "read"):
        T, n = case["T"], case["T"] - case["pad"]
        row = d + 4 / bs
        if kind == "read":
            return dict(bytes=2 * n * Hkv * (row + 2 * d) + 8 * T, flops=2.0 * n * Hkv * d)
        # half a block a sequence is there before: rescaled (read and written) or left, and read back
        old = case["seqs"] * (bs - 1) / 2
        return dict(bytes=2 * n * Hkv * (2 * d + row) + 2 * (n + old) * Hkv * (row + 2 * d) + 16 * T,
                    flops=2.0 * n * Hkv * d * 6)
    B = case["B"]
    lens = _lens(case, torch.Generator().manual_seed(1))     # the ragged cases' lengths: one draw's
    tokens, blocks = int(lens.sum()), int(((lens + bs - 1) // bs).sum())
    if kind == "evict":
        kept = int(lens.clamp(max=case["keep"]).sum())
        return dict(bytes=kept * Hkv * (2 * 2 * 2 * d + 4 + 4) + tokens * Hkv * 4 + 8 * blocks,
                    flops=2.0 * tokens * Hkv)
    H = case["H"]
    io = 4 * B * H * d + 4 * B + 4 * blocks
    if kind == "decode":
        return dict(bytes=2 * tokens * Hkv * d + 8 * blocks * Hkv + io, flops=4.0 * tokens * H * d)
    return dict(bytes=4 * tokens * Hkv * d + 8 * tokens * Hkv + io, flops=4.0 * tokens * H * d)


# ------------------------------------------------------------------------------------- exact
_E4M3 = None


def _value(code, fmt):
    """Code bytes -> their numbers in fp64, from the formats' definitions."""
    global _E4M3
    if fmt == "int8":
        c = code.double()
        return torch.where(c < 128, c, c - 256)
    if _E4M3 is None:
        table = []
        for b in range(256):
            e, m = b >> 3 & 15, b & 7
            v = math.nan if b & 127 == 127 else m * 2.0 ** -9 if e == 0 else (8 + m) * 2.0 ** (e - 10)
            table.append(-v if b & 128 else v)
        _E4M3 = torch.tensor(table, dtype=torch.float64, device="cuda")
    return _E4M3[code.long()]


def _nearest(x, fmt):
    """The value of the nearest code (ties to even) to each fp64 number."""
    if fmt == "int8":
        return torch.round(x).clip(-127, 127)
    e = torch.floor(torch.log2(x.abs().clip(min=2.0 ** -6)))
    step = torch.exp2(e - 3)
    return (torch.round(x / step) * step).clip(-448, 448)


def _exact_softmax(q, k, v, scale):
    """q [H, d], k / v [L, Hkv, d], all fp64 -> [H, d] and the weights [H, L]."""
    out = torch.zeros_like(q)
    weight = torch.zeros(q.shape[0], k.shape[0], dtype=torch.float64, device=q.device)
    G = q.shape[0] // k.shape[1]
    for h in range(q.shape[0] if k.shape[0] else 0):
        s = (k[:, h // G] @ q[h]) * scale
        w = torch.exp(s - s.max())
        weight[h] = w / w.sum()
        out[h] = weight[h] @ v[:, h // G]
    return out, weight


def _exact_write(st):
    c = st["case"]
    bs, fmt, slots = c["bs"], c["fmt"], st["slots"].tolist()
    groups = {}
    for t, s in enumerate(slots):
        if s >= 0:
            groups.setdefault(s // bs, []).append(t)
    back = st["back"]
    live = back >= 0
    outs, scales = [], []
    for x in "kv":
        value, scale = _value(st[x + "_cache"], fmt), st[x + "_scale"].double()
        new = st[x + "_new"].double()
        for b, ts in groups.items():
            r = [slots[t] % bs for t in ts]
            a = new[ts].abs().amax((0, 2))
            old = torch.zeros_like(a) if 0 in r else scale[b].clone()
            s = torch.maximum(old, (a / TOP[fmt]).float().double())
            safe = torch.where(s > 0, s, torch.ones_like(s))
            ratio = (old / safe).float().double()[:, None, None]
            again = _nearest((value[b] * ratio).float().double(), fmt)
            value[b] = torch.where(((old > 0) & (s > old))[:, None, None], again, value[b])
            y = _nearest((new[ts] / safe[:, None]).float().double(), fmt)
            value[b, :, r] = torch.where(s[:, None] > 0, y, torch.zeros_like(y)).transpose(0, 1)
            scale[b] = s
        out = st[x + "_out"].double()
        at = back[live]
        out[live] = value[at // bs, :, at % bs] * scale[at // bs][..., None]
        outs.append(out)
        scales.append(scale)
    return outs + scales


def exact(case, seed):
    st = prepare(case, seed)
    kind, bs, Hkv = case["kind"], case["bs"], case["Hkv"]
    if kind == "write":
        return _exact_write(st)
    if kind == "read":
        live = st["slots"] >= 0
        at = st["slots"][live]
        outs = []
        for x in "kv":
            out = st[x + "_out"].double()
            out[live] = (_value(st[x + "_cache"][at // bs, :, at % bs], case["fmt"])
                         * st[x + "_scale"].double()[at // bs][..., None])
            outs.append(out)
        return outs
    lens = st["lens"].tolist()
    if kind in ("decode", "weigh"):
        out = torch.zeros_like(st["q"], dtype=torch.float64)
        weights = st["weights"].double() if kind == "weigh" else None
        G = case["H"] // Hkv
        for i, n in enumerate(lens):
            pos = torch.arange(n, device="cuda")
            b, r = st["tables"][i].long()[pos // bs], pos % bs
            if kind == "decode":
                k, v = (_value(st[x + "_cache"][b, :, r], case["fmt"]) * st[x + "_scale"].double()[b][..., None]
                        for x in "kv")
            else:
                k, v = (st[x + "_cache"][b, r].double() for x in "kv")
            out[i], w = _exact_softmax(st["q"][i].double(), k, v, st["scale"])
            if kind == "weigh":
                weights[int(st["rows"][i]), :, :n] += w.view(Hkv, G, n).sum(1)
        return out if kind == "decode" else (out, weights)
    keep, first, last = case["keep"], case["first"], case["last"]
    kept = torch.full_like(st["kept"], -1)
    kept_lens = torch.zeros_like(st["kept_lens"])
    new_weights = st["new_weights"].double()
    caches = [st["k_cache"].double(), st["v_cache"].double()]
    from_ = [x.clone() for x in caches]
    for i, n in enumerate(lens):
        m = min(n, keep)
        kept_lens[i] = m
        row = int(st["rows"][i])
        new_weights[row] = 0
        for h in range(Hkv):
            w = st["weights"][row, h, :n].tolist()
            if n <= keep:
                chosen = list(range(n))
            else:
                middle = sorted(range(first, n - last), key=lambda j: (-w[j], j))[: keep - first - last]
                chosen = sorted([*range(first), *middle, *range(n - last, n)])
            p = torch.tensor(chosen, device="cuda", dtype=torch.long)
            r = torch.arange(m, device="cuda")
            kept[i, h, :m] = p.int()
            new_weights[row, h, :m] = st["weights"][row, h][p].double()
            src, to = st["tables"][i].long()[p // bs], st["new_tables"][i].long()[r // bs]
            for was, now in zip(from_, caches):
                now[to, r % bs, h] = was[src, p % bs, h]
    return kept, kept_lens, new_weights, *caches
