"""Operators of the 4-bit KV cache and of block-sparse decode, as cases that can be timed.

Five operators over the paged cache:

* ``write``     quantise new tokens' K/V into the 4-bit cache and read the written tokens back;
* ``read``      read tokens of a quantised cache (4-bit, INT8 or E4M3) back into 16 bits;
* ``decode``    one query token per sequence over a 4-bit cache;
* ``summarise`` one INT8 box (smallest and largest key) per block and KV head;
* ``sparse``    choose the blocks whose boxes promise the largest scores, attend over those only.

``run`` computes a case with elementary torch operations in 32 bits, or, where ``own`` is
true, with the library's kernels.  A 4-bit row is cut into groups of 64 values; a group holds
``m = f16(min)``, ``s = f16((max - min) / 15)`` and codes ``rint((x - m) / s)`` in 0 .. 15, and a
code stands for ``s * code + m``.
"""
import math
import random

import torch

own = False

GROUP = 64
F16_MAX = 65504.0
DTYPES = {"f16": torch.float16, "bf16": torch.bfloat16}


# ------------------------------------------------------------------------------------ cases
def listed():
    return [
        # one decode step's append: 64 sequences of a 40-head (MHA) model, one token each
        dict(name="write_step", kind="write", T=64, Hkv=40, d=128, bs=16, dtype="f16", pad=0),
        # a prefill step's append: four 2048-token chunks, 8 KV heads
        dict(name="write_prompt", kind="write", T=8192, Hkv=8, d=128, bs=16, dtype="bf16", pad=0),
        # an odd number of E4M3 tokens, some of them padding: a short chunk's context
        dict(name="read_fp8_chunk", kind="read", fmt="fp8", T=1001, Hkv=4, d=128, bs=32, dtype="f16",
             pad=37),
        # the context of a chunked prefill (4 x 8192 tokens) read back for the 16-bit kernels
        dict(name="read_int4_context", kind="read", fmt="int4", T=32768, Hkv=8, d=128, bs=16,
             dtype="bf16", pad=0),
        # the smallest batch: latency
        dict(name="decode_tiny", kind="decode", B=4, H=4, Hkv=2, d=64, bs=16, dtype="f16",
             lens="uniform", lo=1, n=64, empty=0),
        # 64 sequences of a 40-head (MHA) model, U[128, 2048] tokens
        dict(name="decode_mha_64", kind="decode", B=64, H=40, Hkv=40, d=128, bs=16, dtype="f16",
             lens="uniform", lo=128, n=2048, empty=0),
        # long-tailed lengths, 7 query heads a KV head, large blocks, two empty sequences
        dict(name="decode_gqa7_tail", kind="decode", B=32, H=28, Hkv=4, d=128, bs=32, dtype="bf16",
             lens="tail", lo=1, n=24576, empty=2),
        # the largest: 16 sequences of 32768 tokens, 32 / 8 heads
        dict(name="decode_gqa4_32k", kind="decode", B=16, H=32, Hkv=8, d=128, bs=16, dtype="bf16",
             lens="full", lo=0, n=32768, empty=0),
        # blocks that one decode step filled
        dict(name="boxes_step", kind="summarise", nblk=13, Hkv=4, d=128, bs=8, dtype="bf16",
             partial=1),
        # the blocks of a prefill step: 4 x 8192 tokens
        dict(name="boxes_prompt", kind="summarise", nblk=2048, Hkv=8, d=128, bs=16, dtype="bf16",
             partial=0),
        # ragged contexts of up to 8192 tokens, 64 blocks kept of up to 512
        dict(name="sparse_8k", kind="sparse", B=8, H=32, Hkv=8, d=128, bs=16, dtype="bf16",
             lens="uniform", lo=512, n=8192, empty=1, keep=64, first=1, last=2),
        # 16 sequences of 32768 tokens, 128 blocks kept of 2048
        dict(name="sparse_32k", kind="sparse", B=16, H=32, Hkv=8, d=128, bs=16, dtype="bf16",
             lens="full", lo=0, n=32768, empty=0, keep=128, first=1, last=4),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    """One more case over the ranges of the listed ones."""
    kind = rng.choice(["write", "read", "decode", "decode", "summarise", "sparse", "sparse"])
    d = rng.choice([64, 128, 128])
    bs = rng.choice([8, 16, 32])
    dtype = rng.choice(["f16", "bf16"])
    Hkv = rng.choice([1, 2, 4, 5, 8, 40])
    if kind == "write":
        T = _log(rng, 1, 65536 // Hkv)
        return dict(kind=kind, T=T, Hkv=Hkv, d=d, bs=bs, dtype=dtype, pad=rng.randrange(0, T // 4 + 1))
    if kind == "read":
        fmt = rng.choice(["int4", "int4", "int8", "fp8"])
        T = _log(rng, 1, 262144 // Hkv)
        return dict(kind=kind, fmt=fmt, T=T, Hkv=Hkv, d=d if fmt == "int4" else 128, bs=bs, dtype=dtype,
                    pad=rng.randrange(0, T // 4 + 1))
    if kind == "summarise":
        nblk = _log(rng, 1, 65536 // (Hkv * bs) * 4)
        return dict(kind=kind, nblk=nblk, Hkv=Hkv, d=d, bs=bs, dtype=dtype,
                    partial=rng.randrange(0, nblk + 1))
    Hkv = rng.choice([1, 2, 4, 5, 8])
    G = rng.choice([1, 2, 3, 4, 7, 8, 12, 16])
    n = _log(rng, 1 if kind == "decode" else 256, 32768)
    B = _log(rng, 1, max(1, min(128, 2000000 // (n * Hkv))))
    lens = rng.choice(["full", "uniform", "tail"])
    c = dict(kind=kind, B=B, H=Hkv * G, Hkv=Hkv, d=d, bs=bs, dtype=dtype, lens=lens, lo=rng.randrange(1, n + 1),
             n=n, empty=rng.randrange(0, B // 8 + 1))
    if kind == "sparse":
        c.update(first=rng.randrange(0, 3), last=rng.randrange(1, 5),
                 keep=_log(rng, 8, max(9, n // bs)))
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


def _paged(case, gen, hgen):
    """A pool of 1.25 x the blocks that the lengths need, handed out in random order."""
    bs = case["bs"]
    lens = _lens(case, hgen)
    nb = (lens + bs - 1) // bs
    N = max(1, math.ceil(1.25 * int(nb.sum())))
    width = max(1, int(nb.max()))
    order = torch.randperm(N, generator=hgen)
    col = torch.arange(width)
    idx = (nb.cumsum(0) - nb)[:, None] + col
    used = col < nb[:, None]
    tables = torch.where(used, order[idx.clamp(max=N - 1)], torch.tensor(-1)).int()
    # (block, row) of the slots behind each sequence's last token
    seq, r = torch.meshgrid(torch.arange(len(lens)), torch.arange(bs), indexing="ij")
    last = tables.gather(1, (nb - 1).clamp(min=0)[:, None]).expand(-1, bs)
    behind = (lens[:, None] > 0) & (r >= ((lens - 1) % bs + 1)[:, None])
    return dict(lens=lens.int().cuda(), tables=tables.cuda(), N=N, max_len=int(lens.max()),
                behind=(last[behind].cuda().long(), r[behind].cuda()))


def _const(v):
    """A divisor on the GPU: dividing by a host number multiplies by its rounded reciprocal."""
    return torch.full((), v, device="cuda")


def _quantise(x):
    """x [..., d] (16-bit) -> packed codes [..., d / 2] uint8 and (s, m) [..., d / 64, 2] f16."""
    g = x.float().unflatten(-1, (x.shape[-1] // GROUP, GROUP))
    lo, hi = g.amin(-1), g.amax(-1)
    m = lo.clamp(-F16_MAX, F16_MAX).half()
    s = ((hi - lo) / _const(15.0)).clamp(max=F16_MAX).half()
    sf, mf = s.float()[..., None], m.float()[..., None]
    c = torch.where(sf > 0, (g - mf) / sf, torch.zeros_like(g))
    c = c.round().clamp(0, 15).to(torch.uint8).flatten(-2)
    return c[..., 0::2] | (c[..., 1::2] << 4), torch.stack((s, m), -1)


def _values4(codes, scale):
    """Packed codes and (s, m) -> the fp32 values that they stand for."""
    c = torch.stack((codes & 15, codes >> 4), -1).flatten(-2)
    g = c.unflatten(-1, (c.shape[-1] // GROUP, GROUP)).float()
    sm = scale.float()
    return (g * sm[..., 0:1] + sm[..., 1:2]).flatten(-2)


def _cache4(N, Hkv, bs, d, dtype, gen, channels):
    codes = torch.empty(N, Hkv, bs, d // 2, dtype=torch.uint8, device="cuda")
    scale = torch.empty(N, Hkv, bs, d // GROUP, 2, dtype=torch.float16, device="cuda")
    step = max(1, (1 << 26) // (Hkv * bs * d))
    for a in range(0, N, step):
        n = min(step, N - a)
        codes[a: a + n], scale[a: a + n] = _quantise(_normal((n, Hkv, bs, d), dtype, gen, channels))
    return codes, scale


def _slots(case, hgen, N):
    """Distinct slots of the pool, its last block left free; ``pad`` of them are padding (-1)."""
    T = case["T"]
    slots = torch.randperm((N - 1) * case["bs"], generator=hgen)[:T]
    # a prompt's tokens take neighbouring slots, a decode step's lie all over the pool
    slots = slots.sort().values if T > 256 else slots
    if case["pad"]:
        slots[torch.randperm(T, generator=hgen)[: case["pad"]]] = -1
    return slots.cuda()


def _boxes(k):
    """k [..., bs, d] -> INT8 (smallest, largest) codes [..., 2, d] and their fp32 scale [...]."""
    lo, hi = k.float().amin(-2), k.float().amax(-2)
    s = torch.maximum(lo.abs(), hi.abs()).amax(-1) / _const(127.0)
    box = torch.stack((lo, hi), -2)
    div = torch.where(s > 0, s, torch.ones_like(s))[..., None, None]
    return (box / div).round().clamp(-127, 127).to(torch.int8), s


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(int(seed))
    hgen = torch.Generator().manual_seed(int(seed))
    kind, dt = case["kind"], DTYPES[case["dtype"]]
    Hkv, d, bs = case["Hkv"], case["d"], case["bs"]
    st = dict(case=dict(case), scale=d ** -0.5)
    if kind == "write":
        T = case["T"]
        N = math.ceil(1.25 * T / bs) + 1
        st.update(k_new=_normal((T, Hkv, d), dt, gen, True), v_new=_normal((T, Hkv, d), dt, gen),
                  slots=_slots(case, hgen, N), N=N)
        for x in "kv":
            st[x + "_cache"] = torch.zeros(N, Hkv, bs, d // 2, dtype=torch.uint8, device="cuda")
            st[x + "_scale"] = torch.zeros(N, Hkv, bs, d // GROUP, 2, dtype=torch.float16, device="cuda")
            st[x + "_out"] = torch.zeros(T, Hkv, d, dtype=dt, device="cuda")
    elif kind == "read":
        T = case["T"]
        N = math.ceil(1.25 * T / bs) + 1
        for x in "kv":
            if case["fmt"] == "int4":
                st[x + "_cache"], st[x + "_scale"] = _cache4(N, Hkv, bs, d, dt, gen, x == "k")
            else:
                r = _normal((N, bs, Hkv, d), dt, gen, x == "k").float()
                top = 127.0 if case["fmt"] == "int8" else 448.0
                s = r.abs().amax(-1) / top
                y = r / torch.where(s > 0, s, torch.ones_like(s))[..., None]
                st[x + "_cache"] = (y.round().to(torch.int8) if case["fmt"] == "int8"
                                    else y.to(torch.float8_e4m3fn)).view(torch.uint8)
                st[x + "_scale"] = s.transpose(1, 2).contiguous()
            st[x + "_out"] = torch.full((T, Hkv, d), 0.5, dtype=dt, device="cuda")
        st["slots"] = _slots(case, hgen, N)
    elif kind == "summarise":
        N = math.ceil(1.25 * case["nblk"]) + 1
        fills = torch.full((case["nblk"],), bs, dtype=torch.int32)
        fills[: case["partial"]] = torch.randint(0, bs + 1, (case["partial"],), generator=hgen,
                                                 dtype=torch.int32)
        st.update(k_cache=_normal((N, bs, Hkv, d), dt, gen, True),
                  ids=torch.randperm(N, generator=hgen)[: case["nblk"]].int().cuda(),
                  fills=fills.cuda(),
                  boxes=torch.zeros(N, Hkv, 2, d, dtype=torch.int8, device="cuda"),
                  box_scale=torch.zeros(N, Hkv, dtype=torch.float32, device="cuda"))
    else:
        st.update(_paged(case, gen, hgen))
        st["q"] = _normal((case["B"], case["H"], d), dt, gen)
        st["out"] = torch.empty_like(st["q"])
        blk, row = st.pop("behind")
        if kind == "decode":
            for x in "kv":
                st[x + "_cache"], st[x + "_scale"] = _cache4(st["N"], Hkv, bs, d, dt, gen, x == "k")
                st[x + "_scale"][blk, :, row] = float("nan")      # slots that nothing was written to
        else:
            st["k_cache"] = _normal((st["N"], bs, Hkv, d), dt, gen, True)
            st["v_cache"] = _normal((st["N"], bs, Hkv, d), dt, gen)
            st["boxes"], st["box_scale"] = _boxes(st["k_cache"].transpose(1, 2))
            for x in "kv":
                st[x + "_cache"][blk, row] = float("nan")
            B, keep = case["B"], case["keep"]
            st["sel"] = torch.empty(B, Hkv, keep, dtype=torch.int32, device="cuda")
            st["sel_lens"] = torch.empty(B, Hkv, dtype=torch.int32, device="cuda")
    return st


# ------------------------------------------------------------------------------ plain forms
def _plain_write(st):
    c = st["case"]
    bs, slots = c["bs"], st["slots"]
    ok = slots >= 0
    # padding tokens go to the pool's last block, which holds nothing
    at = torch.where(ok, slots, torch.full_like(slots, (st["N"] - 1) * bs))
    outs = []
    for x in "kv":
        codes, scale = _quantise(st[x + "_new"])
        cache, scales = st[x + "_cache"], st[x + "_scale"]
        cache[at // bs, :, at % bs] = codes
        scales[at // bs, :, at % bs] = scale
        val = _values4(cache[at // bs, :, at % bs], scales[at // bs, :, at % bs])
        outs.append(torch.where(ok[:, None, None], val.to(st[x + "_out"].dtype), st[x + "_out"]))
    return outs


def _plain_read(st):
    c = st["case"]
    bs, slots = c["bs"], st["slots"]
    ok = slots >= 0
    at = slots.clamp(min=0)
    outs = []
    for x in "kv":
        if c["fmt"] == "int4":
            val = _values4(st[x + "_cache"][at // bs, :, at % bs], st[x + "_scale"][at // bs, :, at % bs])
        else:
            raw = st[x + "_cache"][at // bs, at % bs]
            raw = raw.view(torch.int8) if c["fmt"] == "int8" else raw.view(torch.float8_e4m3fn)
            val = raw.float() * st[x + "_scale"][at // bs, :, at % bs][..., None]
        outs.append(torch.where(ok[:, None, None], val.to(st[x + "_out"].dtype), st[x + "_out"]))
    return outs


def _attend(q, k, v, mask, scale):
    """q [B, Hkv, G, d], k / v [B, L, Hkv, d] fp32, mask [B, L, Hkv] -> [B, Hkv, G, d]."""
    s = torch.einsum("bhgd,blhd->bhgl", q, k) * scale
    live = mask.transpose(1, 2)[:, :, None]
    s = torch.where(live, s, torch.full_like(s, -math.inf))
    p = (s - s.amax(-1, keepdim=True).clamp(min=-1e30)).exp()
    v = torch.where(mask[..., None], v, torch.zeros_like(v))
    return torch.einsum("bhgl,blhd->bhgd", p, v) / p.sum(-1, keepdim=True).clamp(min=1e-30)


def _plain_decode(st):
    c = st["case"]
    bs = c["bs"]
    pos = torch.arange(max(st["max_len"], 1), device="cuda")
    blk = st["tables"].long()[:, pos // bs].clamp(min=0)
    row = (pos % bs).expand_as(blk)
    k = _values4(st["k_cache"][blk, :, row], st["k_scale"][blk, :, row])
    v = _values4(st["v_cache"][blk, :, row], st["v_scale"][blk, :, row])
    mask = (pos < st["lens"][:, None])[..., None].expand(k.shape[:3])
    q = st["q"].float().view(c["B"], c["Hkv"], -1, c["d"])
    return _attend(q, k, v, mask, st["scale"]).view_as(st["q"]).to(st["q"].dtype)


def _plain_summarise(st):
    k = st["k_cache"][st["ids"].long()].transpose(1, 2).float()      # [n, Hkv, bs, d]
    live = torch.arange(k.shape[2], device="cuda") < st["fills"][:, None]
    live = live[:, None, :, None]
    lo = torch.where(live, k, torch.full_like(k, math.inf)).amin(2)
    hi = torch.where(live, k, torch.full_like(k, -math.inf)).amax(2)
    some = (st["fills"] > 0)[:, None, None]
    lo, hi = torch.where(some, lo, torch.zeros_like(lo)), torch.where(some, hi, torch.zeros_like(hi))
    code, s = _boxes(torch.stack((lo, hi), -2))
    boxes, scales = st["boxes"].clone(), st["box_scale"].clone()
    boxes[st["ids"].long()] = code
    scales[st["ids"].long()] = s
    return boxes, scales


def _plain_select(st):
    """(physical blocks [B, Hkv, keep], their tokens [B, Hkv]); scores in the defined roundings."""
    c = st["case"]
    B, Hkv, keep, bs = c["B"], c["Hkv"], c["keep"], c["bs"]
    tables, lens = st["tables"].long(), st["lens"].long()
    q = st["q"].float().view(B, Hkv, -1, c["d"])
    sq = q.abs().amax(-1) / _const(127.0)
    qc = (q / torch.where(sq > 0, sq, torch.ones_like(sq))[..., None]).round().clamp(-127, 127)
    box = st["boxes"][tables.clamp(min=0)].float()                   # [B, W, Hkv, 2, d]
    # integers below 2^24: exact in fp32 in any order
    dot = (torch.einsum("bwhd,bhgd->bhwg", box[..., 1, :], qc.clamp(min=0)) +
           torch.einsum("bwhd,bhgd->bhwg", box[..., 0, :], qc.clamp(max=0)))
    sb = st["box_scale"][tables.clamp(min=0)].transpose(1, 2)        # [B, Hkv, W]
    score = (dot * sq[:, :, None]).mul(sb[..., None]).amax(-1)
    nb = ((lens + bs - 1) // bs)[:, None, None]
    w = torch.arange(tables.shape[1], device="cuda")
    kept = (w < c["first"]) | (w >= nb - c["last"])
    score = torch.where(kept, torch.full_like(score, math.inf), score)
    score = torch.where(w < nb, score, torch.full_like(score, -math.inf))
    best = score.sort(dim=-1, descending=True, stable=True).indices[..., :keep]
    best = torch.where(best < nb, best, torch.full_like(best, tables.shape[1])).sort(-1).values
    some = best < tables.shape[1]
    ids = tables[:, None].expand(B, Hkv, -1).gather(2, best.clamp(max=tables.shape[1] - 1))
    sel = torch.full((B, Hkv, keep), -1, dtype=torch.int32, device="cuda")
    sel[..., : best.shape[-1]] = torch.where(some, ids, torch.full_like(ids, -1)).int()
    n = some.sum(-1)
    tail = (lens - (nb[:, 0, 0] - 1) * bs)[:, None]
    return sel, torch.where(n > 0, (n - 1) * bs + tail, torch.zeros_like(n)).int()


def _plain_sparse(st):
    c = st["case"]
    B, Hkv, d, bs = c["B"], c["Hkv"], c["d"], c["bs"]
    sel, n = _plain_select(st)
    h = torch.arange(Hkv, device="cuda")[None, :, None, None]
    r = torch.arange(bs, device="cuda")
    at = sel.long().clamp(min=0)[..., None]
    k = st["k_cache"][at, r, h].float().view(B, Hkv, -1, d).transpose(1, 2)
    v = st["v_cache"][at, r, h].float().view(B, Hkv, -1, d).transpose(1, 2)
    mask = (torch.arange(k.shape[1], device="cuda")[:, None] < n[:, None])
    q = st["q"].float().view(B, Hkv, -1, d)
    return sel, n, _attend(q, k, v, mask, st["scale"]).view_as(st["q"]).to(st["q"].dtype)


PLAIN = dict(write=_plain_write, read=_plain_read, decode=_plain_decode, summarise=_plain_summarise,
             sparse=_plain_sparse)


# ------------------------------------------------------------------------ the library's calls
def _decode_workspace(pa, st):
    """The decode's workspace, which a program allocates and zeroes once."""
    if "ws" not in st:
        c = st["case"]
        st["ws"] = torch.zeros(pa.pa_decode_workspace_size(c["B"], c["H"], c["d"]), dtype=torch.uint8,
                               device="cuda")
    return st["ws"]


def _own(st):
    import paged_kv_cache_103_gb300 as pa
    c = st["case"]
    kind = c["kind"]
    cache = [st[x] for x in ("k_cache", "v_cache", "k_scale", "v_scale") if x in st]
    if kind == "write":
        pa.pa_reshape_and_cache_int4(st["k_new"], st["v_new"], st["slots"], *cache)
        pa.pa_gather_cache_int4(*cache, st["slots"], st["k_out"], st["v_out"])
        return [st["k_out"], st["v_out"]]
    if kind == "read":
        read = dict(int4=pa.pa_gather_cache_int4, int8=pa.pa_gather_cache_int8,
                    fp8=pa.pa_gather_cache_fp8)[c["fmt"]]
        read(*cache, st["slots"], st["k_out"], st["v_out"])
        return [st["k_out"], st["v_out"]]
    if kind == "decode":
        pa.pa_decode_int4(st["q"], *cache, st["tables"], st["lens"], st["max_len"], st["scale"],
                          st["out"], _decode_workspace(pa, st))
        return st["out"]
    if kind == "summarise":
        pa.pa_summarize_blocks(st["k_cache"], st["ids"], st["boxes"], st["box_scale"], st["fills"])
        return st["boxes"], st["box_scale"]
    if "sel_ws" not in st:
        st["sel_ws"] = torch.zeros(pa.pa_select_blocks_workspace_size(c["B"], c["Hkv"],
                                                                      st["tables"].shape[1]),
                                   dtype=torch.uint8, device="cuda")
    pa.pa_select_blocks(st["q"], st["boxes"], st["box_scale"], st["tables"], st["lens"], c["bs"],
                        c["first"], c["last"], st["sel"], st["sel_lens"], st["sel_ws"])
    pa.pa_decode_selected(st["q"], st["k_cache"], st["v_cache"], st["sel"], st["sel_lens"],
                          c["keep"] * c["bs"], st["scale"], st["out"], _decode_workspace(pa, st))
    return st["sel"], st["sel_lens"], st["out"]


def run(state):
    return _own(state) if own else PLAIN[state["case"]["kind"]](state)


# -------------------------------------------------------------------------------------- work
def work(case):
    """Each input read once, each output written once."""
    kind, Hkv, d = case["kind"], case["Hkv"], case["d"]
    row4 = d // 2 + d // GROUP * 4
    if kind in ("write", "read"):
        n = case["T"] - case["pad"]
        row = row4 if kind == "write" or case["fmt"] == "int4" else d + 4
        wide = 2 if kind == "write" else 1          # new rows in as well as values out
        return dict(bytes=2 * n * Hkv * (row + wide * 2 * d) + 8 * case["T"],
                    flops=2 * n * Hkv * d * (6 if kind == "write" else 2))
    if kind == "summarise":
        n = case["nblk"] * Hkv
        return dict(bytes=n * (case["bs"] * d * 2 + 2 * d + 4) + 8 * case["nblk"],
                    flops=2.0 * n * case["bs"] * d)
    B, H, bs = case["B"], case["H"], case["bs"]
    lens = _lens(case, torch.Generator().manual_seed(1))     # the ragged cases' lengths: one draw's
    tokens, blocks = int(lens.sum()), int(((lens + bs - 1) // bs).sum())
    io = 4 * B * H * d + 4 * B + 4 * blocks
    if kind == "decode":
        return dict(bytes=2 * tokens * Hkv * row4 + io, flops=4.0 * tokens * H * d)
    kept = int(lens.clamp(max=case["keep"] * bs).sum())
    return dict(bytes=2 * kept * Hkv * d * 2 + blocks * Hkv * (2 * d + 4) + io,
                flops=4.0 * kept * H * d + 2.0 * blocks * H * 2 * d)


# ------------------------------------------------------------------------------------- exact
def _exact4(codes, scale):
    low, high = (codes % 16).double(), (codes // 16).double()
    x = torch.empty(*codes.shape[:-1], 2 * codes.shape[-1], dtype=torch.float64, device=codes.device)
    x[..., 0::2], x[..., 1::2] = low, high
    sm = scale.double().repeat_interleave(GROUP, dim=-2)
    return x * sm[..., 0] + sm[..., 1]


def _exact_rows(st, x, at):
    c = st["case"]
    b, r = at // c["bs"], at % c["bs"]
    if c["fmt"] == "int4":
        return _exact4(st[x + "_cache"][b, :, r], st[x + "_scale"][b, :, r])
    raw = st[x + "_cache"][b, r].view(torch.int8 if c["fmt"] == "int8" else torch.float8_e4m3fn)
    return raw.to(torch.float32).double() * st[x + "_scale"][b, :, r].double().unsqueeze(-1)


def _exact_softmax(q, k, v, scale):
    """q [H, d], k / v [L, Hkv, d], all fp64."""
    out = torch.zeros_like(q)
    G = q.shape[0] // k.shape[1]
    for h in range(q.shape[0] if k.shape[0] else 0):
        s = (k[:, h // G] @ q[h]) * scale
        w = torch.exp(s - s.max())
        out[h] = (w @ v[:, h // G]) / w.sum()
    return out


def exact(case, seed):
    st = prepare(case, seed)
    kind, bs = case["kind"], case["bs"]
    if kind in ("write", "read"):
        outs = []
        live = st["slots"] >= 0
        for x in "kv":
            out = st[x + "_out"].double()
            if kind == "read":
                out[live] = _exact_rows(st, x, st["slots"][live])
            else:
                new = st[x + "_new"].double()[live]
                for g in range(case["d"] // GROUP):
                    y = new[..., g * GROUP: (g + 1) * GROUP]
                    m = y.min(-1, keepdim=True).values.half().double()
                    s = ((y.max(-1, keepdim=True).values - y.min(-1, keepdim=True).values) / 15).half().double()
                    code = torch.where(s > 0, torch.round((y - m) / s), torch.zeros_like(y)).clip(0, 15)
                    new[..., g * GROUP: (g + 1) * GROUP] = s * code + m
                out[live] = new
            outs.append(out)
        return outs
    if kind == "summarise":
        boxes, scales = st["boxes"].clone(), st["box_scale"].double()
        for i, (b, f) in enumerate(zip(st["ids"].tolist(), st["fills"].tolist())):
            k = st["k_cache"][b, :f].double()
            box = (torch.stack((k.min(0).values, k.max(0).values), 1) if f
                   else torch.zeros(case["Hkv"], 2, case["d"], dtype=torch.float64, device="cuda"))
            top = box.abs().flatten(1).max(1).values
            s = (top / 127).float().double()
            box = torch.where(s[:, None, None] > 0, box / s[:, None, None], torch.zeros_like(box))
            boxes[b] = torch.round(box.float()).clip(-127, 127).to(torch.int8)
            scales[b] = top / 127
        return boxes, scales
    out = torch.zeros_like(st["q"], dtype=torch.float64)
    lens = st["lens"].tolist()
    if kind == "decode":
        for i, n in enumerate(lens):
            pos = torch.arange(n, device="cuda")
            at = st["tables"][i].long()[pos // bs] * bs + pos % bs
            k, v = (_exact4(st[x + "_cache"][at // bs, :, at % bs], st[x + "_scale"][at // bs, :, at % bs])
                    for x in "kv")
            out[i] = _exact_softmax(st["q"][i].double(), k, v, st["scale"])
        return out
    sel = torch.full_like(st["sel"], -1)
    sel_lens = torch.zeros_like(st["sel_lens"])
    G = case["H"] // case["Hkv"]
    for i, n in enumerate(lens):
        nb = (n + bs - 1) // bs
        ids = st["tables"][i, :nb].long()
        q = st["q"][i].float()
        sq = (q.abs().max(-1).values.double() / 127).float()
        qc = torch.round(q / torch.where(sq > 0, sq, torch.ones_like(sq))[:, None]).clip(-127, 127).double()
        for h in range(case["Hkv"] if n else 0):
            lo, hi = st["boxes"][ids, h, 0].double(), st["boxes"][ids, h, 1].double()
            score = None
            for j in range(h * G, h * G + G):
                dot = torch.where(qc[j] > 0, hi * qc[j], lo * qc[j]).sum(-1)
                one = (dot.float() * sq[j]) * st["box_scale"][ids, h]
                score = one if score is None else torch.maximum(score, one)
            if nb > case["keep"]:
                middle = score[case["first"]: nb - case["last"]].tolist()
                order = sorted(range(len(middle)), key=lambda t: (-middle[t], t))
                order = [t + case["first"] for t in order[: max(0, case["keep"] - case["first"] - case["last"])]]
                chosen = sorted(set(range(case["first"])) | set(range(nb - case["last"], nb)) | set(order))
            else:
                chosen = list(range(nb))
            pick = ids[torch.tensor(chosen, device="cuda")]
            sel[i, h, : len(chosen)] = pick.int()
            m = (len(chosen) - 1) * bs + n - (nb - 1) * bs
            sel_lens[i, h] = m
            t = torch.arange(m, device="cuda")
            k, v = (st[x + "_cache"][pick[t // bs], t % bs, h].double()[:, None] for x in "kv")
            out[i, h * G: h * G + G] = _exact_softmax(st["q"][i, h * G: h * G + G].double(), k, v, st["scale"])
    return sel, sel_lens, out
