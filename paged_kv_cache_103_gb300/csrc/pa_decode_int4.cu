// Paged decode attention over the 4-bit cache (pa_decode_int4): what pa_decode
// computes, with K and V the rows that the codes of pa_reshape_and_cache_int4
// stand for (format: pa_cache_int4.cu).
//
// With x = s c + m per group g of 64 head-dim values, step and minimum leave the
// sums over the codes:
//     q . K_j       = sum_g  s_jg (sum_c q_c c_jc) + m_jg (sum_c q_c)
//     sum_j p_j V_j = sum_j (p_j s_jg) c_jc  +  sum_j p_j m_jg      (c in g)
// so the tensor cores multiply bare codes, K's step and minimum meet each score
// once per key and group, V's step is folded into P, and the minima are one number
// per (head, group).
//
// A code needs no conversion.  As the low bits of an f16 whose other bits are zero
// it is the subnormal c 2^-24 (c 2^-20 in the nibble above), exactly; tensor cores
// take subnormals at full speed, and the powers of two leave through q (K's upper
// nibbles) and the output (V's).  Eight codes become four f16 pairs with four ANDs
// and a shift, against one conversion and more per pair for the 8-bit caches,
// whose conversions bound those kernels.
//
// What bounds it is HBM: 144 bytes a token and KV head at d = 128.  The decode of
// the 16-bit cache keeps four math warps and two loading warps per CTA; at a third
// of the bytes per token the loading warps' hand-offs and the math would both be in
// the way, so here every warp is on its own.  The list of (sequence, KV head,
// 32-token chunk) triples is cut evenly over the CTAs and, inside each, over its
// warps; a warp streams its run of chunks through a ring of its own in shared
// memory with bulk copies that its lanes issue (one per tile of codes or scales: a
// tile is contiguous) and that it alone waits for.  No two warps meet before the
// end, when the pairs that cross from warp to warp are merged in shared memory and
// those that cross from CTA to CTA through the workspace, by the CTA that arrives
// last:
//     M = max m_p,  out = sum_p 2^(m_p - M) o_p / sum_p 2^(m_p - M) l_p.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cmath>
#include <cstring>
#include <mutex>

#include "pa.h"
#include "pa_common.cuh"

namespace {

constexpr int kWarps = 8;
constexpr int kThreads = kWarps * 32;
constexpr int kChunk = 32;              // tokens per stage
constexpr int kTiles = kChunk / 16;     // 16-key MMA tiles per chunk
constexpr int kMaxG = 16;
constexpr int kMaxBatch = 4096;
constexpr int kMaxCtas = 512;
constexpr int kMaxStages = 8;
// A CTA in use has at least one chunk per warp: smaller batches take fewer CTAs
// rather than more partial results.
constexpr int kMinChunksPerCta = kWarps;
constexpr uint64_t kWaitLimitNs = 1ull << 30;   // about one second
constexpr float kLog2e = 1.4426950408889634f;

struct Int4Params {
    const uint16_t* q;
    uint16_t* out;
    const uint8_t *k_cache, *v_cache, *k_scale, *v_scale;
    const int32_t* block_tables;
    const int32_t* context_lens;
    int32_t* counters;   // [B * Hkv] arrival tickets of pairs split between CTAs
    float* partials;     // [2 * CTAs][2 * kMaxG + kMaxG * D]
    unsigned int* err;
    // A KV head with more than kMaxG query heads is `subs` pairs of kMaxG heads.
    int32_t max_blocks, B, H, Hkv, G, bs_shift, num_blocks, stages, subs;
    float scale_log2;
};

// ctas per SM: two, or one where 9 .. 16 heads need two 8-wide MMA tiles and the
// accumulators with them.
__host__ __device__ constexpr int ctas_per_sm(int NT) { return NT == 1 ? 2 : 1; }

// One partial result: row maxima [kMaxG], row sums [kMaxG], outputs [G][D].
__host__ __device__ constexpr int slot_floats(int G, int D) { return 2 * kMaxG + G * D; }

// A run of chunks [c0, end) of one pair that a warp left in shared memory.
struct Run {
    int32_t a;    // flattened index of the pair's first chunk; -1: none
    int32_t i, g, c0, end, nc;
    uint32_t at;  // byte offset of its slot
    int32_t pad;
};

struct Layout {
    uint32_t stage, slots, runs, bars, open, scan, prefix, total;
};

__host__ __device__ inline Layout make_layout(int D, int G, int B, int stages) {
    Layout L;
    L.stage = 2u * kChunk * (D / 2 + D / 64 * 4);            // K, V codes, K, V scales
    L.slots = kWarps * stages * L.stage;                     // a slot per warp
    L.runs = L.slots + kWarps * slot_floats(G, D) * 4;       // [2 * kWarps]
    L.bars = L.runs + 2 * kWarps * (uint32_t)sizeof(Run);    // [kWarps][stages]
    L.open = L.bars + kWarps * kMaxStages * 8;               // runs left to other CTAs
    L.scan = L.open + 16;
    L.prefix = L.scan + kWarps * 4;                          // [B + 1]
    L.total = L.prefix + (uint32_t)(B + 1) * 4;
    return L;
}

__device__ __forceinline__ int32_t clamp_len(int32_t n, int32_t cap) {
    return n < 0 ? 0 : (n > cap ? cap : n);
}

// First chunk of part x when W chunks are cut into n parts.
__device__ __forceinline__ int32_t share(int64_t x, int64_t W, int64_t n) {
    return (int32_t)(x * W / n);
}

// A position in the flattened list: chunk c of pair (i, g), whose nc chunks start at a.
struct Cursor {
    int32_t i, g, c, nc, a;
};

__device__ __forceinline__ Cursor find(const int32_t* prefix, int32_t B, int32_t Hkv, int32_t pos) {
    int32_t lo = 0, hi = B;   // largest i with prefix[i] <= pos
    while (hi - lo > 1) {
        const int32_t mid = (lo + hi) >> 1;
        if (prefix[mid] <= pos) lo = mid; else hi = mid;
    }
    Cursor s;
    s.i = lo;
    s.nc = (prefix[lo + 1] - prefix[lo]) / Hkv;
    const int32_t local = pos - prefix[lo];
    s.g = local / s.nc;
    s.c = local - s.g * s.nc;
    s.a = prefix[lo] + s.g * s.nc;
    return s;
}

// The pair after s (there is one).
__device__ __forceinline__ Cursor next_pair(const int32_t* prefix, int32_t Hkv, Cursor s) {
    s.a += s.nc;
    s.c = 0;
    if (++s.g == Hkv) {
        s.g = 0;
        do ++s.i; while (prefix[s.i + 1] == prefix[s.i]);
        s.nc = (prefix[s.i + 1] - prefix[s.i]) / Hkv;
    }
    return s;
}

__device__ __forceinline__ uint32_t lds32(uint32_t addr) {
    uint32_t v;
    asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(addr));
    return v;
}

__device__ __forceinline__ float2 half2_floats(uint32_t v) {
    __half2 h;
    memcpy(&h, &v, 4);
    return __half22float2(h);
}

template <bool kBF16>
__device__ __forceinline__ float2 widen2(uint32_t v) {
    if constexpr (kBF16)
        return make_float2(__uint_as_float(v << 16), __uint_as_float(v & 0xFFFF0000u));
    else
        return half2_floats(v);
}

// (step, minimum) of the NG groups of one row.
template <int NG>
__device__ __forceinline__ void load_scales(uint32_t addr, float (&s)[NG], float (&m)[NG]) {
    uint32_t w[NG];
    if constexpr (NG == 2) {
        const uint2 v = pa::lds64(addr);
        w[0] = v.x;
        w[1] = v.y;
    } else {
        w[0] = lds32(addr);
    }
#pragma unroll
    for (int g = 0; g < NG; ++g) {
        const float2 f = half2_floats(w[g]);
        s[g] = f.x;
        m[g] = f.y;
    }
}

constexpr uint32_t kLowNibbles = 0x000F000Fu;    // c 2^-24 each
constexpr uint32_t kHighNibbles = 0x00F000F0u;   // c 2^-20 each

template <int D, bool kBF16, int NT>
__global__ void __launch_bounds__(kThreads, ctas_per_sm(NT)) decode_int4_kernel(const Int4Params p) {
    constexpr int NG = D / 64;
    constexpr uint32_t kRow = D / 2, kSRow = NG * 4;         // bytes of a row's codes and scales
    constexpr uint32_t kCodes = kChunk * kRow, kScales = kChunk * kSRow;
    const int32_t B = p.B, Hkv = p.Hkv, G = p.G, S = p.stages, bs_shift = p.bs_shift;
    const Layout L = make_layout(D, G, B, S);
    extern __shared__ __align__(128) unsigned char smem[];
    const uint32_t sbase = pa::smem_addr(smem);
    Run* runs = reinterpret_cast<Run*>(smem + L.runs);
    int32_t* open_run = reinterpret_cast<int32_t*>(smem + L.open);
    int32_t* scan = reinterpret_cast<int32_t*>(smem + L.scan);
    int32_t* prefix = reinterpret_cast<int32_t*>(smem + L.prefix);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int32_t max_len = p.max_blocks << bs_shift;

    // ---- prefix[i] = Hkv * chunks of the sequences before i
    {
        const int per = (B + kThreads - 1) / kThreads;
        const int beg = min(tid * per, B), end = min(beg + per, B);
        int32_t local = 0;
        for (int i = beg; i < end; ++i) {
            const int32_t raw = __ldg(p.context_lens + i);
            if (blockIdx.x == 0) {
                if (raw < 0) pa::raise_error(p.err, PA_DEVERR_CONTEXT);
                if (raw > max_len) pa::raise_error(p.err, PA_DEVERR_TABLE_WIDTH);
            }
            local += (clamp_len(raw, max_len) + kChunk - 1) / kChunk;
        }
        int32_t x = local;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int32_t y = __shfl_up_sync(0xffffffffu, x, o);
            if (lane >= o) x += y;
        }
        if (lane == 31) scan[warp] = x;
        if (tid < 2 * kWarps) runs[tid].a = -1;
        if (tid < 2) open_run[tid] = -1;
        if (lane == 0) {
            for (int s = 0; s < S; ++s)
                pa::mbar_init(reinterpret_cast<uint64_t*>(smem + L.bars) + warp * S + s, 1);
            pa::fence_barrier_init();
        }
        __syncthreads();
        int32_t run = x - local;
        for (int w = 0; w < warp; ++w) run += scan[w];
        for (int i = beg; i < end; ++i) {
            prefix[i] = run * Hkv;
            run += (clamp_len(__ldg(p.context_lens + i), max_len) + kChunk - 1) / kChunk;
        }
        if (tid == 0) {
            int32_t total = 0;
            for (int w = 0; w < kWarps; ++w) total += scan[w];
            prefix[B] = total * Hkv;
        }
        __syncthreads();
    }

    // ---- zero rows of empty contexts
    for (int32_t i = blockIdx.x; i < B; i += gridDim.x) {
        if (prefix[i + 1] != prefix[i]) continue;
        uint4* row = reinterpret_cast<uint4*>(p.out + (int64_t)i * p.H * D);
        for (int v = tid; v < p.H * D / 8; v += kThreads) row[v] = make_uint4(0, 0, 0, 0);
    }

    const int64_t W = prefix[B];
    int64_t C = (W + kMinChunksPerCta - 1) / kMinChunksPerCta;
    if (C > (int64_t)gridDim.x) C = gridDim.x;
    if ((int64_t)blockIdx.x >= C) return;
    const int32_t cta_lo = share(blockIdx.x, W, C), cta_hi = share(blockIdx.x + 1, W, C);
    const int32_t lo = cta_lo + share(warp, cta_hi - cta_lo, kWarps);
    const int32_t hi = cta_lo + share(warp + 1, cta_hi - cta_lo, kWarps);

    const uint32_t ring = sbase + (uint32_t)warp * S * L.stage;
    const uint32_t bars = sbase + L.bars + (uint32_t)(warp * S) * 8;
    uint64_t* bars_p = reinterpret_cast<uint64_t*>(smem + L.bars) + warp * S;
    bool dead = false;

    if (lo < hi) {
        // ================= loading: this warp's chunks, in order =================
        // Lane 4 b + w issues copy w (K codes, V codes, K scales, V scales) of the
        // chunk's block b.
        const int which = lane & 3;
        const int bpc = kChunk >> bs_shift;     // blocks per chunk: 4, 2 or 1
        const uint8_t* src = which == 0 ? p.k_cache : which == 1 ? p.v_cache
                                        : which == 2 ? p.k_scale : p.v_scale;
        const uint32_t unit = (which < 2 ? kRow : kSRow) << bs_shift;   // bytes of a tile
        const uint32_t dst = (which == 0 ? 0 : which == 1 ? kCodes
                              : which == 2 ? 2 * kCodes : 2 * kCodes + kScales) +
                             (uint32_t)(lane >> 2) * unit;
        const uint32_t block_bytes = (2 * (kRow + kSRow)) << bs_shift;
        const uint64_t policy = pa::l2_policy_evict_first();
        const int32_t real_heads = Hkv / p.subs;
        // A pair's table entries, 32 at a time (lane l holds entry wbase + l), with
        // the window after it and the next pair's first one loaded a step ahead.
        struct Walk {
            Cursor s;
            int32_t n, wbase, went, wnext;
            const int32_t* row;
        };
        auto open = [&](const Cursor& s) {
            Walk w;
            w.s = s;
            w.n = __ldg(p.context_lens + s.i);
            w.row = p.block_tables + (int64_t)s.i * p.max_blocks;
            w.wbase = (s.c * kChunk) >> bs_shift;
            const int32_t j = w.wbase + lane;
            w.went = j < p.max_blocks ? __ldg(w.row + j) : -1;
            w.wnext = j + 32 < p.max_blocks ? __ldg(w.row + j + 32) : -1;
            return w;
        };
        int32_t ipos = lo;              // next chunk to issue
        int istage = 0;
        Walk cur = open(find(prefix, B, Hkv, lo)), nxt = cur;
        const Cursor start = cur.s;
        if (start.a + start.nc < hi) nxt = open(next_pair(prefix, Hkv, start));
        auto issue = [&]() {
            const int32_t j0 = (cur.s.c * kChunk) >> bs_shift;
            if (j0 + bpc > cur.wbase + 32) {
                cur.wbase += 32;
                cur.went = cur.wnext;
                const int32_t j = cur.wbase + 32 + lane;
                cur.wnext = j < p.max_blocks ? __ldg(cur.row + j) : -1;
            }
            const int32_t b = lane >> 2;
            const int32_t blk = __shfl_sync(0xffffffffu, cur.went, (j0 - cur.wbase + b) & 31);
            const int32_t nb = (clamp_len(cur.n, max_len) + (1 << bs_shift) - 1) >> bs_shift;
            const bool want = b < bpc && j0 + b < nb;
            const bool ok = want && blk >= 0 && blk < p.num_blocks;
            const uint32_t good = __ballot_sync(0xffffffffu, ok && which == 0);
            const uint32_t to = ring + (uint32_t)istage * L.stage + dst;
            if (__any_sync(0xffffffffu, want && !ok)) {
                // A block outside the pool stands for rows of zeros: steps and
                // minima of zero (its stale codes are finite).
                if (want && !ok && which >= 2) {
                    if (which == 2) pa::raise_error(p.err, PA_DEVERR_BLOCK_ID);
                    for (uint32_t x = 0; x < unit; x += 16)
                        asm volatile("st.shared.v4.u32 [%0], {%1, %1, %1, %1};" ::"r"(to + x), "r"(0)
                                     : "memory");
                }
                pa::fence_proxy_async_smem();
            }
            if (lane == 0)
                pa::mbar_arrive_expect_tx(bars_p + istage, (uint32_t)__popc(good) * block_bytes);
            __syncwarp();
            if (ok)
                pa::bulk_load(to, src + ((int64_t)blk * real_heads + cur.s.g / p.subs) * unit, unit,
                              bars + 8 * istage, policy);
            if (++istage == S) istage = 0;
            ++ipos;
            if (++cur.s.c == cur.s.nc && ipos < hi) {
                cur = nxt;
                if (cur.s.a + cur.s.nc < hi) nxt = open(next_pair(prefix, Hkv, cur.s));
            }
        };

        // ============================ attention ============================
        const int cr = lane >> 2, c4 = lane & 3;
        uint32_t qb[NT][NG][4][2];      // Q^T fragments: lane holds query head 8 nt + cr
        float qsum[NT][NG][2];          // sum of q times scale, heads 8 nt + 2 c4 + {0, 1}
        float qsc = 0.f;                // from an MMA score over a step to a base-2 logit
        auto load_q = [&](const Cursor& s) {
            // In k-step ks of a group the lane's fragment pairs values v0 + {0, 4} (b0) and
            // v0 + {1, 5} (b1), v0 = 16 c4 + 8 (ks / 2) + 2 (ks % 2): the nibbles that the
            // masks leave.  q is scaled by 2^e so that its largest value lies in
            // [2^14, 2^15), and by 1/16 more where it meets upper nibbles.
            float amax = 0.f;
            uint32_t raw[NT][NG][8];
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                const int h = 8 * nt + cr;
                const uint4* row = reinterpret_cast<const uint4*>(
                    p.q + ((int64_t)s.i * p.H + s.g * G + h) * D + 16 * c4);
#pragma unroll
                for (int g = 0; g < NG; ++g) {
                    const uint4 z = make_uint4(0, 0, 0, 0);
                    const uint4 a = h < G ? __ldg(row + 8 * g) : z;
                    const uint4 b = h < G ? __ldg(row + 8 * g + 1) : z;
                    raw[nt][g][0] = a.x, raw[nt][g][1] = a.y, raw[nt][g][2] = a.z, raw[nt][g][3] = a.w;
                    raw[nt][g][4] = b.x, raw[nt][g][5] = b.y, raw[nt][g][6] = b.z, raw[nt][g][7] = b.w;
                }
            }
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int g = 0; g < NG; ++g) {
                    float sum = 0.f;
#pragma unroll
                    for (int w = 0; w < 8; ++w) {
                        const float2 f = widen2<kBF16>(raw[nt][g][w]);
                        sum += f.x + f.y;
                        amax = fmaxf(amax, fmaxf(fabsf(f.x), fabsf(f.y)));
                    }
                    sum += __shfl_xor_sync(0xffffffffu, sum, 1);
                    sum += __shfl_xor_sync(0xffffffffu, sum, 2);
                    qsum[nt][g][0] = p.scale_log2 * __shfl_sync(0xffffffffu, sum, 8 * c4);
                    qsum[nt][g][1] = p.scale_log2 * __shfl_sync(0xffffffffu, sum, 8 * c4 + 4);
                }
            amax = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(amax)));
            const int e = min(141 - pa::biased_exponent(amax), 126);
            const float up = pa::exp2_int(e), up16 = up * 0.0625f;   // e >= -113
            qsc = p.scale_log2 * pa::exp2_int(max(-126, min(24 - e, 127)));
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int g = 0; g < NG; ++g)
#pragma unroll
                    for (int ks = 0; ks < 4; ++ks) {
                        // words 4 (ks / 2) + (ks % 2) and + 2: values v0, v0 + 1 and v0 + 4, v0 + 5
                        const float2 a = widen2<kBF16>(raw[nt][g][4 * (ks >> 1) + (ks & 1)]);
                        const float2 b = widen2<kBF16>(raw[nt][g][4 * (ks >> 1) + (ks & 1) + 2]);
                        qb[nt][g][ks][0] = pa::pack2<false>(a.x * up, b.x * up);
                        qb[nt][g][ks][1] = pa::pack2<false>(a.y * up16, b.y * up16);
                    }
        };

        Cursor s = start;
        load_q(s);
        while (ipos < hi && ipos - lo < S) issue();
        int stage = 0;
        uint32_t phase = 0;
        int segn = 0;
        for (int32_t pos = lo; pos < hi;) {
            const int32_t c0 = s.c, c_end = min(s.nc, s.c + hi - pos);
            const int32_t n = clamp_len(__ldg(p.context_lens + s.i), max_len);
            // Running state for heads 8 nt + 2 c4 + {0, 1}: maximum, sum, sums of P times
            // V's minima; o: rows are values 64 g + 8 cr + u (e < 2) and + 4 + u.
            float m_run[NT][2], l_run[NT][2], lowv[NT][NG][2], o[NG][4][NT][4];
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    m_run[nt][j] = -INFINITY;
                    l_run[nt][j] = 0.f;
#pragma unroll
                    for (int g = 0; g < NG; ++g) {
                        lowv[nt][g][j] = 0.f;
#pragma unroll
                        for (int u = 0; u < 4; ++u) o[g][u][nt][j] = o[g][u][nt][2 + j] = 0.f;
                    }
                }
            // P times V's step is kept in f16 range by 2^vexp, which o carries.
            int vexp = 126;
            for (int32_t c = c0; c < c_end; ++c) {
                const bool ready = dead || pa::mbar_wait(bars_p + stage, phase, kWaitLimitNs);
                if (!__all_sync(0xffffffffu, ready)) {
                    dead = true;
                    if (lane == 0) pa::raise_error(p.err, PA_DEVERR_TIMEOUT);
                }
                if (!dead) {
                    const int32_t valid = n - c * kChunk;   // tokens of the chunk in the context
                    const uint32_t kt = ring + (uint32_t)stage * L.stage;
                    const uint32_t vt = kt + kCodes, kst = vt + kCodes, vst = kst + kScales;
                    // ---- S^T = K Q^T per group, then base-2 logits
                    float x[kTiles][NT][4];
#pragma unroll
                    for (int mt = 0; mt < kTiles; ++mt) {
                        float st[NG][NT][4];
#pragma unroll
                        for (int g = 0; g < NG; ++g)
#pragma unroll
                            for (int nt = 0; nt < NT; ++nt)
                                st[g][nt][0] = st[g][nt][1] = st[g][nt][2] = st[g][nt][3] = 0.f;
                        const uint32_t row0 = 16 * mt + cr;
#pragma unroll
                        for (int g = 0; g < NG; ++g) {
                            const uint2 w0 = pa::lds64(kt + row0 * kRow + 32 * g + 8 * c4);
                            const uint2 w1 = pa::lds64(kt + (row0 + 8) * kRow + 32 * g + 8 * c4);
#pragma unroll
                            for (int ks = 0; ks < 4; ++ks) {
                                const uint32_t y0 = (ks < 2 ? w0.x : w0.y) >> (8 * (ks & 1));
                                const uint32_t y1 = (ks < 2 ? w1.x : w1.y) >> (8 * (ks & 1));
                                const uint32_t a[4] = {y0 & kLowNibbles, y1 & kLowNibbles,
                                                       y0 & kHighNibbles, y1 & kHighNibbles};
#pragma unroll
                                for (int nt = 0; nt < NT; ++nt)
                                    pa::mma_16816<false>(st[g][nt], a, qb[nt][g][ks][0], qb[nt][g][ks][1]);
                            }
                        }
#pragma unroll
                        for (int r = 0; r < 2; ++r) {
                            float ks[NG], km[NG];
                            load_scales<NG>(kst + (row0 + 8 * r) * kSRow, ks, km);
#pragma unroll
                            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                                for (int j = 0; j < 2; ++j) {
                                    float v = 0.f;
#pragma unroll
                                    for (int g = 0; g < NG; ++g)
                                        v += km[g] * qsum[nt][g][j] + ks[g] * qsc * st[g][nt][2 * r + j];
                                    x[mt][nt][2 * r + j] =
                                        (int)row0 + 8 * r < valid ? v : -INFINITY;
                                }
                        }
                    }
                    // ---- V's steps and minima of this lane's rows; steps in f16 range
                    float vs[kTiles][2][NG], vm[kTiles][2][NG], vmax = 0.f, rs = 1.f;
#pragma unroll
                    for (int mt = 0; mt < kTiles; ++mt)
#pragma unroll
                        for (int r = 0; r < 2; ++r) {
                            const int row = 16 * mt + cr + 8 * r;
                            load_scales<NG>(vst + row * kSRow, vs[mt][r], vm[mt][r]);
#pragma unroll
                            for (int g = 0; g < NG; ++g) {
                                // rows past the context may hold anything: weightless
                                vs[mt][r][g] = row < valid ? vs[mt][r][g] : 0.f;
                                vm[mt][r][g] = row < valid ? vm[mt][r][g] : 0.f;
                                vmax = fmaxf(vmax, vs[mt][r][g]);
                            }
                        }
                    vmax = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(vmax)));
                    if (vmax > 0.f) {
                        const int e = min(vexp, 141 - pa::biased_exponent(vmax));
                        if (e < vexp) {
                            rs = e - vexp >= -126 ? pa::exp2_int(e - vexp) : 0.f;
                            vexp = e;
                        }
                    }
                    const float vup = pa::exp2_int(vexp);
                    // ---- online softmax per head
                    bool grew = false;
                    float alpha[NT][2];
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                        for (int j = 0; j < 2; ++j) {
                            float v = x[0][nt][j];
#pragma unroll
                            for (int mt = 0; mt < kTiles; ++mt)
                                v = fmaxf(v, fmaxf(x[mt][nt][j], x[mt][nt][2 + j]));
                            v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 4));
                            v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 8));
                            v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 16));
                            const float m_new = fmaxf(m_run[nt][j], v);
                            grew |= m_new > m_run[nt][j];
                            alpha[nt][j] = pa::fast_exp2(m_run[nt][j] - m_new);
                            m_run[nt][j] = m_new;
                        }
                    if (__any_sync(0xffffffffu, grew) || rs != 1.f) {
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                            for (int j = 0; j < 2; ++j) {
                                l_run[nt][j] *= alpha[nt][j];
                                const float f = alpha[nt][j] * rs;
#pragma unroll
                                for (int g = 0; g < NG; ++g) {
                                    lowv[nt][g][j] *= alpha[nt][j];
#pragma unroll
                                    for (int u = 0; u < 4; ++u) {
                                        o[g][u][nt][j] *= f;
                                        o[g][u][nt][2 + j] *= f;
                                    }
                                }
                            }
                    }
                    // ---- P, and O^T += V^T P^T
#pragma unroll
                    for (int mt = 0; mt < kTiles; ++mt) {
                        uint32_t pb[NG][NT][2];
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt) {
                            float e[4];
#pragma unroll
                            for (int q = 0; q < 4; ++q) {
                                e[q] = pa::fast_exp2(x[mt][nt][q] - m_run[nt][q & 1]);
                                l_run[nt][q & 1] += e[q];
                            }
#pragma unroll
                            for (int g = 0; g < NG; ++g)
#pragma unroll
                                for (int r = 0; r < 2; ++r) {
                                    // rounded to f16: P's only rounding
                                    const float f = vs[mt][r][g] * vup;
                                    pb[g][nt][r] = pa::movmatrix_trans(
                                        pa::pack2<false>(e[2 * r] * f, e[2 * r + 1] * f));
                                    lowv[nt][g][0] += e[2 * r] * vm[mt][r][g];
                                    lowv[nt][g][1] += e[2 * r + 1] * vm[mt][r][g];
                                }
                        }
                        // The fragment's key pairs: 16 mt + 8 r + 2 c4 + {0, 1}; odd c4 read
                        // the pair's second row first, so that the four rows of a load lie in
                        // both halves of the 128 bytes, and swap in the byte permutation.
                        const uint32_t odd = c4 & 1;
                        const uint32_t row = 16 * mt + 2 * c4;
#pragma unroll
                        for (int g = 0; g < NG; ++g) {
                            uint32_t z[2][2];   // [key half][values 0..3 | 4..7]
#pragma unroll
                            for (int r = 0; r < 2; ++r) {
                                const uint32_t at = vt + (row + 8 * r) * kRow + 32 * g + 4 * cr;
                                const uint32_t w0 = lds32(at + odd * kRow), w1 = lds32(at + (odd ^ 1) * kRow);
                                z[r][0] = __byte_perm(w0, w1, odd ? 0x1054 : 0x5410);
                                z[r][1] = __byte_perm(w0, w1, odd ? 0x3276 : 0x7632);
                            }
#pragma unroll
                            for (int u = 0; u < 4; ++u) {
                                const uint32_t mask = u & 1 ? kHighNibbles : kLowNibbles;
                                const int sh = 8 * (u >> 1);
                                const uint32_t a[4] = {(z[0][0] >> sh) & mask, (z[0][1] >> sh) & mask,
                                                       (z[1][0] >> sh) & mask, (z[1][1] >> sh) & mask};
#pragma unroll
                                for (int nt = 0; nt < NT; ++nt)
                                    pa::mma_16816<false>(o[g][u][nt], a, pb[g][nt][0], pb[g][nt][1]);
                            }
                        }
                    }
                }
                __syncwarp();   // every lane has read the stage: it may be filled again
                if (++stage == S) {
                    stage = 0;
                    phase ^= 1u;
                }
                if (ipos < hi && !dead) issue();
            }
            pos += c_end - c0;

            // ---- the pair's chunks of this warp are done
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int j = 0; j < 2; ++j) {
#pragma unroll
                    for (int off = 4; off < 32; off <<= 1) {
                        l_run[nt][j] += __shfl_xor_sync(0xffffffffu, l_run[nt][j], off);
#pragma unroll
                        for (int g = 0; g < NG; ++g)
                            lowv[nt][g][j] += __shfl_xor_sync(0xffffffffu, lowv[nt][g][j], off);
                    }
                }
            const bool whole = c0 == 0 && c_end == s.nc;
            // The warp's first run may end while its ring is in use: a slot of its own.
            // A later unfinished run is its last: the ring is free.
            const uint32_t at = segn == 0 ? L.slots + (uint32_t)warp * slot_floats(G, D) * 4
                                          : (uint32_t)warp * S * L.stage;
            float* slot = reinterpret_cast<float*>(smem + at);
            const float low = pa::exp2_int(min(24 - vexp, 127)), high = low * 0.0625f;
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    const int h = 8 * nt + 2 * c4 + j;
                    if (h >= G) continue;
                    const float inv = whole ? 1.f / l_run[nt][j] : 1.f;
                    if (!whole && cr == 0) {
                        slot[h] = m_run[nt][j];
                        slot[kMaxG + h] = l_run[nt][j];
                    }
#pragma unroll
                    for (int g = 0; g < NG; ++g) {
                        float v[8];
#pragma unroll
                        for (int u = 0; u < 8; ++u)
                            v[u] = (o[g][u & 3][nt][2 * (u >> 2) + j] * (u & 1 ? high : low) +
                                    lowv[nt][g][j]) * inv;
                        const int at_d = 64 * g + 8 * cr;
                        if (whole) {
                            *reinterpret_cast<uint4*>(p.out + ((int64_t)s.i * p.H + s.g * G + h) * D + at_d) =
                                make_uint4(pa::pack2<kBF16>(v[0], v[1]), pa::pack2<kBF16>(v[2], v[3]),
                                           pa::pack2<kBF16>(v[4], v[5]), pa::pack2<kBF16>(v[6], v[7]));
                        } else {
                            float4* to = reinterpret_cast<float4*>(slot + 2 * kMaxG + h * D + at_d);
                            to[0] = make_float4(v[0], v[1], v[2], v[3]);
                            to[1] = make_float4(v[4], v[5], v[6], v[7]);
                        }
                    }
                }
            if (!whole && lane == 0) {
                Run& r = runs[2 * warp + (segn ? 1 : 0)];
                r.i = s.i;
                r.g = s.g;
                r.c0 = c0;
                r.end = c_end;
                r.nc = s.nc;
                r.at = at;
                r.a = s.a;
            }
            ++segn;
            if (pos < hi) {
                s = next_pair(prefix, Hkv, s);
                load_q(s);
            }
        }
        if (dead)   // copies still in flight land before the CTA may exit
            for (int st = 0; st < S && st < ipos - lo; ++st)
                pa::mbar_wait(bars_p + st, (uint32_t)((ipos - lo - 1 - st) / S) & 1u, kWaitLimitNs);
    }
    __syncthreads();

    // ====================== runs of one pair in several warps ======================
    // Runs lie in list order, so a pair's runs are neighbours.  The warp that holds a
    // pair's first run merges it if the pair lies in this CTA, and leaves it to the
    // whole CTA if other CTAs share it (at most the CTA's first and last pair).
    auto merged4 = [&](int first, int count, int h, int d4, float& M, float& l) -> float4 {
        M = -INFINITY;
        for (int k = 0; k < count; ++k)
            if (runs[first + k].a == runs[first].a)
                M = fmaxf(M, reinterpret_cast<const float*>(smem + runs[first + k].at)[h]);
        float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
        l = 0.f;
        for (int k = 0; k < count; ++k) {
            if (runs[first + k].a != runs[first].a) continue;
            const float* slot = reinterpret_cast<const float*>(smem + runs[first + k].at);
            const float f = pa::fast_exp2(slot[h] - M);
            const float4 x = *reinterpret_cast<const float4*>(slot + 2 * kMaxG + h * D + d4);
            l += f * slot[kMaxG + h];
            v.x += f * x.x;
            v.y += f * x.y;
            v.z += f * x.z;
            v.w += f * x.w;
        }
        return v;
    };
    auto store4 = [&](int32_t i, int32_t h, int d4, float4 v, float inv) {
        *reinterpret_cast<uint2*>(p.out + ((int64_t)i * p.H + h) * D + d4) =
            make_uint2(pa::pack2<kBF16>(v.x * inv, v.y * inv), pa::pack2<kBF16>(v.z * inv, v.w * inv));
    };
    auto span = [&](int first) {   // runs from `first` on that may belong to its pair
        int last = first;
        for (int k = first + 1; k < 2 * kWarps; ++k)
            if (runs[k].a == runs[first].a) last = k;
        return last - first + 1;
    };
    for (int k = 2 * warp; k < 2 * warp + 2; ++k) {
        const int32_t a = runs[k].a;
        if (a < 0) continue;
        bool leads = true;
        for (int b = 0; b < k; ++b) leads &= runs[b].a != a;
        if (!leads) continue;
        const int count = span(k);
        if (runs[k].c0 != 0 || runs[k + count - 1].end != runs[k].nc) {
            if (lane == 0) open_run[runs[k].a > cta_lo ? 1 : 0] = k;
            continue;
        }
        for (int e = lane; e < G * D / 4; e += 32) {
            const int h = e / (D / 4), d4 = (e % (D / 4)) * 4;
            float M, l;
            const float4 v = merged4(k, count, h, d4, M, l);
            store4(runs[k].i, runs[k].g * G + h, d4, v, 1.f / l);
        }
    }
    __syncthreads();

    // ================= pairs shared with other CTAs, by the whole CTA =================
    constexpr int kSlot = slot_floats(kMaxG, D);
    int32_t* is_last = open_run + 2;
    for (int which = 0; which < 2; ++which) {
        const int k = open_run[which];
        if (k < 0) continue;
        const Run r = runs[k];
        const int count = span(k);
        const int64_t c_first = ((int64_t)(r.a + 1) * C - 1) / W;
        const int64_t c_last = ((int64_t)(r.a + r.nc) * C - 1) / W;
        // A CTA's first slot holds the pair that its share begins in or with, its
        // second the one that begins later.
        float* mine = p.partials + (2 * (int64_t)blockIdx.x + (cta_lo >= r.a ? 0 : 1)) * kSlot;
        for (int e = tid; e < G * D / 4; e += kThreads) {
            const int h = e / (D / 4), d4 = (e % (D / 4)) * 4;
            float M, l;
            const float4 v = merged4(k, count, h, d4, M, l);
            *reinterpret_cast<float4*>(mine + 2 * kMaxG + h * D + d4) = v;
            if (d4 == 0) {
                mine[h] = M;
                mine[kMaxG + h] = l;
            }
        }
        __syncthreads();
        if (tid == 0) {
            int32_t* ticket = p.counters + (int64_t)r.i * Hkv + r.g;
            const int last = pa::atomic_add_acq_rel_gpu(ticket, 1) == (int)(c_last - c_first);
            if (last) atomicExch(ticket, 0);   // ready for the next launch
            *is_last = last;
        }
        __syncthreads();
        if (*is_last) {
            const int n = (int)(c_last - c_first + 1);
            const int64_t slot0 = 2 * c_first + (share(c_first, W, C) == r.a ? 0 : 1);
            for (int e = tid; e < G * D / 4; e += kThreads) {
                const int h = e / (D / 4), d4 = (e % (D / 4)) * 4;
                float M = -INFINITY, l = 0.f;
                float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
                for (int c0 = 0; c0 < n; c0 += 8) {
                    float pm[8], pl[8];
                    float4 po[8];
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        const int c = c0 + j;
                        if (c < n) {
                            const float* q = p.partials + (c ? 2 * (c_first + c) : slot0) * kSlot;
                            pm[j] = __ldcg(q + h);
                            pl[j] = __ldcg(q + kMaxG + h);
                            po[j] = __ldcg(reinterpret_cast<const float4*>(q + 2 * kMaxG + h * D + d4));
                        } else {
                            pm[j] = -INFINITY;
                            pl[j] = 0.f;
                            po[j] = make_float4(0.f, 0.f, 0.f, 0.f);
                        }
                    }
                    float Mb = M;
#pragma unroll
                    for (int j = 0; j < 8; ++j) Mb = fmaxf(Mb, pm[j]);
                    if (Mb == -INFINITY) continue;
                    const float f0 = pa::fast_exp2(M - Mb);   // 0 while M = -inf
                    l *= f0;
                    acc.x *= f0;
                    acc.y *= f0;
                    acc.z *= f0;
                    acc.w *= f0;
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        const float f = pa::fast_exp2(pm[j] - Mb);
                        l += f * pl[j];
                        acc.x += f * po[j].x;
                        acc.y += f * po[j].y;
                        acc.z += f * po[j].z;
                        acc.w += f * po[j].w;
                    }
                    M = Mb;
                }
                store4(r.i, r.g * G + h, d4, acc, 1.f / l);
            }
        }
    }
}

// ---- host side -----------------------------------------------------------------

// Shared memory per CTA that leaves room for ctas_per_sm(NT) of them on an SM.
uint32_t smem_budget(int NT) { return (NT == 1 ? 113 : 226) * 1024; }

int choose_stages(int D, int G, int B) {
    const int NT = G <= 8 ? 1 : 2;
    const Layout L = make_layout(D, G, B, 0);
    if (L.total >= smem_budget(NT)) return 0;
    const int s = (int)((smem_budget(NT) - L.total) / (kWarps * L.stage));
    return s > kMaxStages ? kMaxStages : s;
}

template <int D, bool kBF16, int NT>
pa_status launch(const Int4Params& p, cudaStream_t stream) {
    auto kern = decode_int4_kernel<D, kBF16, NT>;
    // The shared-memory limit is set once per device.
    static std::mutex mu;
    static uint64_t done = 0;
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev >= 64) return PA_ERR_CUDA;
    {
        std::lock_guard<std::mutex> g(mu);
        if (!(done >> dev & 1)) {
            if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                     (int)smem_budget(NT)) != cudaSuccess)
                return PA_ERR_CUDA;
            done |= 1ull << dev;
        }
    }
    int ctas = pa::device_sm_count() * ctas_per_sm(NT);
    if (ctas <= 0) return PA_ERR_CUDA;
    if (ctas > kMaxCtas) ctas = kMaxCtas;
    const Layout L = make_layout(D, p.G, p.B, p.stages);
    kern<<<ctas, kThreads, L.total, stream>>>(p);
    return pa::cuda_status(cudaGetLastError());
}

}  // namespace

extern "C" {

PA_API pa_status pa_decode_int4(const void* q, const void* k_cache, const void* v_cache,
                                const void* k_scale, const void* v_scale,
                                const int32_t* block_tables, int32_t max_blocks,
                                const int32_t* context_lens, int32_t max_context_len, int32_t B,
                                int32_t H, int32_t Hkv, int32_t d, int32_t block_size,
                                int32_t num_blocks, float scale, pa_dtype dtype, void* out,
                                void* workspace, size_t ws_bytes, void* stream) {
    if (B < 0 || H <= 0 || Hkv <= 0 || max_blocks <= 0 || num_blocks <= 0 ||
        max_context_len < 0 || !std::isfinite(scale))
        return PA_ERR_INVALID;
    if (dtype != PA_F16 && dtype != PA_BF16) return PA_ERR_UNSUPPORTED;
    if (H % Hkv != 0) return PA_ERR_UNSUPPORTED;
    int G = H / Hkv, subs = 1;
    if (G > kMaxG) {
        if (G % kMaxG != 0) return PA_ERR_UNSUPPORTED;
        subs = G / kMaxG;
        G = kMaxG;
    }
    if (d != 64 && d != 128) return PA_ERR_UNSUPPORTED;
    if (block_size != 8 && block_size != 16 && block_size != 32) return PA_ERR_UNSUPPORTED;
    if (B > kMaxBatch || (int64_t)num_blocks * block_size > INT32_MAX ||
        (int64_t)max_blocks * block_size > INT32_MAX)
        return PA_ERR_UNSUPPORTED;
    // Flattened chunk indices are int32.
    const int64_t max_chunks = ((int64_t)max_blocks * block_size + kChunk - 1) / kChunk;
    if ((int64_t)B * Hkv * subs * max_chunks >= ((int64_t)1 << 30)) return PA_ERR_UNSUPPORTED;
    if (B > 0 && ws_bytes < pa_decode_workspace_size(B, H, d)) return PA_ERR_INVALID;
    if (B == 0) return PA_OK;
    if (!q || !k_cache || !v_cache || !k_scale || !v_scale || !block_tables || !context_lens ||
        !out || !workspace)
        return PA_ERR_INVALID;
    if ((reinterpret_cast<uintptr_t>(k_cache) | reinterpret_cast<uintptr_t>(v_cache) |
         reinterpret_cast<uintptr_t>(k_scale) | reinterpret_cast<uintptr_t>(v_scale) |
         reinterpret_cast<uintptr_t>(q) | reinterpret_cast<uintptr_t>(out)) & 15u)
        return PA_ERR_INVALID;
    Int4Params p;
    p.stages = choose_stages(d, G, B);
    if (p.stages < 2) return PA_ERR_UNSUPPORTED;
    p.err = pa::device_error_word();
    if (!p.err) return PA_ERR_CUDA;
    p.q = static_cast<const uint16_t*>(q);
    p.out = static_cast<uint16_t*>(out);
    p.k_cache = static_cast<const uint8_t*>(k_cache);
    p.v_cache = static_cast<const uint8_t*>(v_cache);
    p.k_scale = static_cast<const uint8_t*>(k_scale);
    p.v_scale = static_cast<const uint8_t*>(v_scale);
    p.block_tables = block_tables;
    p.context_lens = context_lens;
    p.counters = static_cast<int32_t*>(workspace);
    const size_t tickets = (((size_t)B * H * sizeof(int32_t)) + 255) & ~size_t(255);
    p.partials = reinterpret_cast<float*>(static_cast<unsigned char*>(workspace) + tickets);
    p.max_blocks = max_blocks;
    p.B = B;
    p.H = H;
    p.Hkv = Hkv * subs;
    p.G = G;
    p.subs = subs;
    p.bs_shift = block_size == 8 ? 3 : block_size == 16 ? 4 : 5;
    p.num_blocks = num_blocks;
    p.scale_log2 = scale * kLog2e;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (G <= 8) {
        if (d == 128)
            return dtype == PA_BF16 ? launch<128, true, 1>(p, st) : launch<128, false, 1>(p, st);
        return dtype == PA_BF16 ? launch<64, true, 1>(p, st) : launch<64, false, 1>(p, st);
    }
    if (d == 128)
        return dtype == PA_BF16 ? launch<128, true, 2>(p, st) : launch<128, false, 2>(p, st);
    return dtype == PA_BF16 ? launch<64, true, 2>(p, st) : launch<64, false, 2>(p, st);
}

}  // extern "C"
