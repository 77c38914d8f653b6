// Paged decode attention over the 4-bit cache (pa_decode_int4): what pa_decode
// computes, with K and V the rows that the codes of pa_reshape_and_cache_int4
// stand for (format: pa_cache_int4.cu).
//
// With x = s c + m per group g of 64 head-dim values, step and minimum leave the
// sums over the codes:
//     q . K_j       = sum_g  s_jg (sum_c q_c c_jc) + m_jg (sum_c q_c)
//     sum_j p_j V_j = sum_j (p_j s_jg) (c_jc - 8)  +  sum_j p_j (m_jg + 8 s_jg)   (c in g)
// so the tensor cores multiply bare codes, K's step and minimum meet each score
// once per key and group, V's step is folded into P, and the values of code 8 are one
// number per (head, group).  The 8 that the codes are taken from is a product of its
// own, P times a tile of eights, subtracted every four chunks: what the tensor cores'
// truncating sums do to the codes' mean (2.5 times their spread, and 100 times the result of
// a long flat context) they do to the eights as well, and between two subtractions the sums
// stay small.  (Subtracted once, at the end of a run, an f16 result of 16 contexts of 32768
// tokens, G = 4, was off 1.6 times as far as an fp32 computation's; every eight chunks it is
// 1.002 times in 107.2 us, every four 1.0004 in 107.7, every two 1.0004 in 108.9.)
//
// P times V's step goes to the tensor cores as two bf16 numbers, its upper half and what
// that leaves, rounded: 16 bits of it (off by 2^-16 of it at most) at every size that fp32
// holds, whatever the steps of other tokens, groups and heads are.  (One f16 number under a
// power of two for each warp, as it was, lost the codes of small steps beside a step 2^17
// times theirs, and gave an f16 result 1.4 times an fp32 computation's error.)  Up to four
// query heads the second part takes columns of the products that are free, above that
// products of its own.  Against the single number 16 x 32768 tokens of 8 KV heads take 107.7
// instead of 106 us with G = 4, 124 instead of 108 with G = 8, 197 instead of 159 with G = 16.
//
// A code needs no conversion.  As the low bits of an f16 whose other bits are zero
// it is the subnormal c 2^-24 (c 2^-20 in the nibble above), exactly, and as a bf16's a
// byte of two codes is c 2^-133 + c' 2^-129; tensor cores take subnormals at full speed, and the
// powers of two leave through q (K's upper nibbles) and the output (V's).  Eight codes
// become four pairs with four ANDs and a shift, against one conversion and more per pair
// for the 8-bit caches, whose conversions bound those kernels.
//
// What bounds it is HBM: 144 bytes a token and KV head at d = 128.  The decode of
// the 16-bit cache keeps four math warps and two loading warps per CTA; at a third
// of the bytes per token the loading warps' hand-offs and the math would both be in
// the way, so here every warp is on its own.  The list of (sequence, KV head,
// 32-token chunk) triples is cut into parts of equal cost for the CTAs and, inside each,
// for its warps; a warp streams its run of chunks through a ring of its own in shared
// memory by asynchronous 16-byte copies, 512 contiguous bytes an instruction, that it
// alone waits for.  No two warps meet before the end, when the pairs that cross from
// warp to warp are merged in shared memory and those that cross from CTA to CTA
// through the workspace, by the CTA that arrives last:
//     M = max m_p,  out = sum_p 2^(m_p - M) o_p / sum_p 2^(m_p - M) l_p.
//
// Measured (d = 128, device time): 16 x 32768 tokens of 8 KV heads, G = 4: 107.8 us, 5.6
// TB/s, DRAM traffic 1.000 times the bytes above, 53 % of the ALU's and 28 % of the tensor
// pipe's cycles, 57 % of the issue slots; 64 sequences of 128 .. 2048 tokens, 40 heads, G =
// 1: 70 us, 5.7 TB/s; 32 long-tailed contexts, 4 heads of G = 7, 70 MB: 24 us, of which
// the start is some 4 (lengths, table, first copies) and the joining of pairs at the end as
// much; 4 sequences of up to 64 tokens: 6.6 us, all latency.  Asynchronous copies took the
// place of bulk copies (one per tile, each a turn of a loop over the lanes), and one CTA
// that of two CTAs of 8 warps, whose pairs crossed CTAs twice as often.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cmath>
#include <cstring>

#include "pa.h"
#include "pa_common.cuh"
#include "pa_runs.cuh"

namespace {

using namespace pa::runs;

constexpr int kTiles = kChunk / 16;     // 16-key MMA tiles per chunk
// Stages of a warp's ring: it computes on one while the others fill.
__host__ __device__ constexpr int ring_stages(int D) { return D == 128 ? 2 : 4; }
constexpr float kLog2e = 1.4426950408889634f;

struct Int4Params {
    const uint16_t* q;
    uint16_t* out;
    const uint8_t *k_cache, *v_cache, *k_scale, *v_scale;
    const int32_t* block_tables;
    const int32_t* context_lens;
    int32_t* counters;
    float* partials;
    unsigned int* err;
    // A KV head with more than kMaxG query heads is `subs` pairs of kMaxG heads.
    int32_t max_blocks, B, H, Hkv, G, bs_shift, num_blocks, subs, warps;
    float scale_log2;
};

// The forms of the kernel by query heads of a KV head: one; up to 4; up to 8; up to 16.
enum Form { kG1, kG4, kG8, kG16 };
constexpr Form form_of(int G) { return G == 1 ? kG1 : G <= 4 ? kG4 : G <= 8 ? kG8 : kG16; }
// One CTA per SM.  Warps by the registers a chunk takes: at d = 128 twelve of 168, which
// keeps more than 128 in use (with sixteen of 128, which spill, 16 x 32768 tokens take 111.4 us
// with G = 4 instead of 107.3, the 40-head batch 71.7 instead of 69.8, the long-tailed one of
// G = 7 27.1 instead of 24.2; fourteen leave the four schedulers uneven: 120 us); at d = 64
// sixteen (64.2 us against 65.7 with twelve); eight where 9 .. 16 heads need two 8-wide
// MMA tiles and twice the accumulators.
__host__ __device__ constexpr int max_warps(int D, int form) {
    return form == kG16 ? 8 : D == 128 ? 12 : 16;
}
constexpr uint32_t kSmemBudget = 227 * 1024;

// Bytes of the warps' rings: K, V codes, K, V scales a stage; and of all that lies before the
// runs' slots, per warp K and V scales of 32 rows more.
__host__ __device__ constexpr uint32_t ring_bytes(int D) {
    return ring_stages(D) * 2u * kChunk * (D / 2 + D / 64 * 4);
}
__host__ __device__ constexpr uint32_t rows_bytes(int D) { return 2 * kChunk * (D / 64) * 8; }
__host__ __device__ inline Layout layout_of(int D, int G, int B, int warps) {
    return make_layout(warps * (ring_bytes(D) + rows_bytes(D)), D, G, B, warps);
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

// (step, minimum) of the NG groups of one row, as they lie in the cache (f16) and as
// the rows' scratch holds them (fp32).
template <int NG>
__device__ __forceinline__ void load_f16_scales(uint32_t addr, float (&v)[2 * NG]) {
    uint32_t w[NG];
    if constexpr (NG == 2) {
        const uint2 x = pa::lds64(addr);
        w[0] = x.x;
        w[1] = x.y;
    } else {
        w[0] = lds32(addr);
    }
#pragma unroll
    for (int g = 0; g < NG; ++g) {
        const float2 f = half2_floats(w[g]);
        v[2 * g] = f.x;
        v[2 * g + 1] = f.y;
    }
}
template <int NG>
__device__ __forceinline__ void load_row(uint32_t addr, float (&v)[2 * NG]) {
    if constexpr (NG == 2) {
        const uint4 x = pa::lds128(addr);
        v[0] = __uint_as_float(x.x);
        v[1] = __uint_as_float(x.y);
        v[2] = __uint_as_float(x.z);
        v[3] = __uint_as_float(x.w);
    } else {
        const uint2 x = pa::lds64(addr);
        v[0] = __uint_as_float(x.x);
        v[1] = __uint_as_float(x.y);
    }
}
template <int NG>
__device__ __forceinline__ void store_row(uint32_t addr, const float (&v)[2 * NG]) {
    if constexpr (NG == 2)
        asm volatile("st.shared.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "f"(v[0]), "f"(v[1]),
                     "f"(v[2]), "f"(v[3]) : "memory");
    else
        asm volatile("st.shared.v2.f32 [%0], {%1, %2};" ::"r"(addr), "f"(v[0]), "f"(v[1]) : "memory");
}

constexpr uint32_t kLowNibbles = 0x000F000Fu;    // c 2^-24 each
constexpr uint32_t kHighNibbles = 0x00F000F0u;   // c 2^-20 each
constexpr uint32_t kBytes = 0x00FF00FFu;         // of a bf16: (c + 16 c') 2^-133 each

// A head's running maximum is raised only when a logit exceeds it by more than this
// (base 2): probabilities reach 2^8, which fp32 sums bear, and most chunks need neither the
// maximum across lanes nor a rescale.
constexpr float kLazy = 8.f;
constexpr int kSettle = 4;   // chunks between two subtractions of the codes' middle
// V's steps are held 2^64 times as large, so that what they and P are multiplied by, codes
// 2^-133 times theirs, leaves normal numbers down to a P of 2^-33 at f16's smallest step, and
// sums over any context stay far below fp32's largest.
constexpr int kUp = 64;

// A float's upper half as a float: a bf16 number, toward zero.
__device__ __forceinline__ float upper_half(float x) {
    return __uint_as_float(__float_as_uint(x) & 0xFFFF0000u);
}

// kG1: a lane tracks one column, head 0, instead of two; the next one is the second part of P.
// kG4: columns h and h + 4 are both head h, the latter with the second part of P and the
// former with minus the first.
template <int D, bool kBF16, int kForm, int kShift>
__global__ void __launch_bounds__(max_warps(D, kForm) * 32, 1) decode_int4_kernel(const Int4Params p) {
    constexpr bool kOne = kForm == kG1, kDup = kForm == kG4;
    constexpr int NG = D / 64, NT = kForm == kG16 ? 2 : 1, NJ = kOne ? 1 : 2;
    constexpr uint32_t kRow = D / 2, kSRow = NG * 4;         // bytes of a row's codes and scales
    constexpr uint32_t kCodes = kChunk * kRow, kScales = kChunk * kSRow;
    constexpr uint32_t kStage = 2 * (kCodes + kScales);   // K, V codes, K, V scales
    constexpr int S = ring_stages(D);
    const int32_t B = p.B, Hkv = p.Hkv, G = p.G;
    constexpr int bs_shift = kShift, bmask = (1 << kShift) - 1;
    const int nw = p.warps, threads = nw * 32;
    const Layout L = layout_of(D, G, B, nw);
    extern __shared__ __align__(128) unsigned char smem[];
    const uint32_t sbase = pa::smem_addr(smem);
    Run* runs = reinterpret_cast<Run*>(smem + L.runs);
    int32_t* is_last = reinterpret_cast<int32_t*>(smem + L.last);
    int32_t* scan = reinterpret_cast<int32_t*>(smem + L.scan);
    int32_t* prefix = reinterpret_cast<int32_t*>(smem + L.prefix);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int32_t max_len = p.max_blocks << bs_shift;

    asm volatile("griddepcontrol.wait;" ::: "memory");   // launched while the kernel before may run

    // The tables and queries are read a dependent load or two from now: into L2 with
    // them, a line per thread (what they cover is shared by all CTAs).
    {
        const int64_t line = ((int64_t)blockIdx.x * threads + tid) * 128;
        if (line < (int64_t)B * p.max_blocks * 4)
            prefetch_l2(reinterpret_cast<const char*>(p.block_tables) + line);
        if (line < (int64_t)B * p.H * D * 2) prefetch_l2(reinterpret_cast<const char*>(p.q) + line);
    }

    const int32_t W = list_prefix(p.context_lens, B, Hkv, max_len, p.err, nw, prefix, scan, is_last, runs);

    // ---- zero rows of empty contexts
#pragma unroll 1
    for (int32_t i = blockIdx.x; i < B; i += gridDim.x) {
        if (prefix[i + 1] != prefix[i]) continue;
        uint4* row = reinterpret_cast<uint4*>(p.out + (int64_t)i * p.H * D);
#pragma unroll 1
        for (int v = tid; v < p.H * D / 8; v += threads) row[v] = make_uint4(0, 0, 0, 0);
    }

    // CTAs in use have a chunk per warp at least: smaller batches take fewer CTAs
    // rather than more partial results.
    const int32_t C = min((W + nw - 1) / nw, (int32_t)gridDim.x);
    if ((int32_t)blockIdx.x >= C) return;
    const Cut cut(prefix[B], C);
    const int32_t cta_lo = cut.begin(blockIdx.x), cta_hi = cut.begin(blockIdx.x + 1);
    const Cut mine(cta_hi - cta_lo, nw);
    const int32_t lo = cta_lo + mine.begin(warp), hi = cta_lo + mine.begin(warp + 1);

    const uint32_t ring = sbase + (uint32_t)warp * S * kStage;
    const uint32_t krows = sbase + nw * ring_bytes(D) + (uint32_t)warp * rows_bytes(D);
    const uint32_t vrows = krows + kChunk * NG * 8;

    Cursor start{};
    int32_t ipos = hi;              // next chunk to issue
    if (lo < hi) {
        start = find(prefix, B, Hkv, lo);
        ipos = start.a + kPairCost + start.c;
    }
    if (ipos < hi) {
        // ================= loading: this warp's chunks, in order =================
        // A copy instruction moves 512 bytes: kPass rows of codes.  The lane's row and
        // 16-byte column in a pass, and in the chunk's scales (K's by the lower lanes,
        // V's by the upper ones).
        constexpr int kPass = 512 / kRow, kScaleLanes = kScales / 16;
        const int lrow = lane / (kRow / 16), srow = lane % kScaleLanes * (16 / kSRow);
        const uint32_t lcol = lane % (kRow / 16) * 16;
        constexpr uint32_t kTile = kRow << bs_shift, kSTile = kSRow << bs_shift;
        const uint32_t heads = (uint32_t)(Hkv / p.subs);
        // Bytes between blocks; a pass lies in one block unless blocks are shorter than it.
        const uint32_t stride = heads * kTile, sstride = heads * kSTile;
        constexpr bool kOneBlock = kPass <= bmask + 1;
        const uint32_t lane_bytes = kOneBlock ? lane * 16 : (lrow & bmask) * kRow + lcol;
        const uint8_t* scales = lane % (2 * kScaleLanes) < kScaleLanes ? p.k_scale : p.v_scale;
        const uint64_t policy = pa::l2_policy_evict_first();
        constexpr int bpc = kChunk >> bs_shift;     // blocks per chunk: 4, 2 or 1
        // A pair's table entries, 32 at a time (lane l holds the window's entry l), with
        // the window after it loaded a step ahead; an entry past the context is -1, as is
        // an id outside the pool.  (The next pair's first window is not loaded ahead: its
        // registers cost more than the wait, which other warps fill.)
        struct Walk {
            Cursor s;
            int32_t at;              // the chunk's first block in the window
            int32_t went, wnext;
            int32_t next, nb;        // this lane's entry after wnext's; blocks of the context
            const uint8_t *k, *v, *sc;   // the pair's KV head in each tensor, at this lane's bytes
        };
        auto entry = [&](int32_t i, int32_t j, int32_t nb) {
            if (j >= nb) return -1;
            const int32_t blk = pa::ld_behind_wait(p.block_tables + (int64_t)i * p.max_blocks + j);
            if ((uint32_t)blk < (uint32_t)p.num_blocks) return blk;
            pa::raise_error(p.err, PA_DEVERR_BLOCK_ID);
            return -1;
        };
        auto open = [&](const Cursor& s) {
            Walk w;
            w.s = s;
            const int32_t j0 = (s.c * kChunk) >> bs_shift, j = j0 + lane;
            const int32_t n = clamp_len(pa::ld_behind_wait(p.context_lens + s.i), max_len);
            const uint32_t head = (uint32_t)(s.g / p.subs);
            w.at = 0;
            w.nb = (n + bmask) >> bs_shift;
            w.went = entry(s.i, j, w.nb);
            w.wnext = entry(s.i, j + 32, w.nb);
            w.next = j + 64;
            w.k = p.k_cache + (uint64_t)head * kTile + lane_bytes;
            w.v = p.v_cache + (uint64_t)head * kTile + lane_bytes;
            w.sc = scales + (uint64_t)head * kSTile + (srow & bmask) * kSRow;
            return w;
        };
        uint32_t ito = ring;            // its stage
        Walk cur = open(start);
        // One chunk's copies, as one group.  Blocks past the context and ids outside the
        // pool are not read: zeros take their place (a step and a minimum of zero: rows of
        // zeros).
        auto issue = [&]() {
            auto block = [&](int b) { return __shfl_sync(0xffffffffu, cur.went, cur.at + b); };
            if constexpr (kOneBlock) {
                constexpr int kPasses = kChunk / kPass / bpc;
#pragma unroll
                for (int b = 0; b < bpc; ++b) {
                    const int32_t blk = block(b);
                    const uint64_t at = (uint64_t)(uint32_t)max(blk, 0) * stride;
                    const uint32_t to = ito + b * kTile + lane * 16;
#pragma unroll
                    for (int t = 0; t < kPasses; ++t) {
                        copy16(to + t * 512, cur.k + at + t * 512, blk >= 0, policy);
                        copy16(to + t * 512 + kCodes, cur.v + at + t * 512, blk >= 0, policy);
                    }
                }
            } else {
#pragma unroll
                for (int t = 0; t < kChunk / kPass; ++t) {
                    const int32_t blk = block((t * kPass + lrow) >> bs_shift);
                    const uint64_t at = (uint64_t)(uint32_t)max(blk, 0) * stride;
                    const uint32_t to = ito + t * 512 + lane * 16;
                    copy16(to, cur.k + at, blk >= 0, policy);
                    copy16(to + kCodes, cur.v + at, blk >= 0, policy);
                }
            }
            const int32_t sblk = block(srow >> bs_shift);
            if (lane < 2 * kScaleLanes)
                copy16(ito + 2 * kCodes + lane * 16, cur.sc + (uint64_t)(uint32_t)max(sblk, 0) * sstride,
                       sblk >= 0, policy);
            ito = ito + kStage == ring + S * kStage ? ring : ito + kStage;
            ++ipos;
            if (++cur.s.c < cur.s.nc) {
                cur.at += bpc;
                if (cur.at == 32) {     // a window is a whole number of chunks
                    cur.at = 0;
                    cur.went = cur.wnext;
                    cur.wnext = entry(cur.s.i, cur.next, cur.nb);
                    cur.next += 32;
                }
            } else if ((ipos += kPairCost) < hi) {
                cur = open(next_pair(prefix, Hkv, cur.s));
            }
        };

        // ============================ attention ============================
        const int cr = lane >> 2, c4 = lane & 3;
        uint32_t qb[NT][NG][4][2];      // Q^T fragments: lane holds query head 8 nt + cr
        float qsum[NT][NG][2];          // sum of q times scale, heads 8 nt + 2 c4 + {0, 1}
        float qsc = 0.f;                // from an MMA score over a step to a base-2 logit
        // In k-step ks of a group the lane's fragment pairs values v0 + {0, 4} (b0) and
        // v0 + {1, 5} (b1), v0 = 16 c4 + 8 (ks / 2) + 2 (ks % 2): the nibbles that the
        // masks leave.  q is scaled by 2^e so that its largest value lies in [2^14, 2^15),
        // and by 1/16 more where it meets upper nibbles.
        uint32_t raw[NT][NG][8];
        auto fetch_q = [&](const Cursor& s) {
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                const int h = kDup ? cr & 3 : 8 * nt + cr;
                const uint4* row = reinterpret_cast<const uint4*>(
                    p.q + ((int64_t)s.i * p.H + s.g * G + h) * D + 16 * c4);
#pragma unroll
                for (int g = 0; g < NG; ++g) {
                    const uint4 z = make_uint4(0, 0, 0, 0);
                    const uint4 a = h < G ? pa::ld_behind_wait(row + 8 * g) : z;
                    const uint4 b = h < G ? pa::ld_behind_wait(row + 8 * g + 1) : z;
                    raw[nt][g][0] = a.x, raw[nt][g][1] = a.y, raw[nt][g][2] = a.z, raw[nt][g][3] = a.w;
                    raw[nt][g][4] = b.x, raw[nt][g][5] = b.y, raw[nt][g][6] = b.z, raw[nt][g][7] = b.w;
                }
            }
        };
        auto convert_q = [&]() {
            float amax = 0.f;
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
        uint32_t stage = ring;   // the chunk to compute
        // Offsets of this lane in a stage: K rows cr, V rows 2 c4 + {0, 1} in its order.
        const uint32_t odd = c4 & 1;
        const uint32_t koff = cr * kRow + 8 * c4;
        const uint32_t voff0 = kCodes + (2 * c4 + odd) * kRow + 4 * cr;
        const uint32_t voff1 = kCodes + (2 * c4 + (odd ^ 1)) * kRow + 4 * cr;
        const uint32_t perm0 = odd ? 0x1054 : 0x5410, perm1 = odd ? 0x3276 : 0x7632;
        const uint32_t krow = krows + cr * NG * 8, vrow = vrows + cr * NG * 8;
        // The tile of eights: rows 0 .. 7 for group 0, 8 .. 15 for group 1, so that one
        // accumulator has P's sums for both.
        constexpr uint32_t kEight = 0x00080008u;
        const uint32_t eights[2][4] = {{kEight, 0, kEight, 0}, {0, kEight, 0, kEight}};
        const float dup = c4 < 2 ? 0.f : 1.f;   // kG4: which part of P this lane's columns have
        int segn = 0;
#pragma unroll 1
        for (int32_t pos = ipos; pos < hi;) {
            // The first chunk is asked for while q is under way, the ring's others after it:
            // they would only delay it.
            fetch_q(s);
#pragma unroll 1
            for (int k = segn == 0 ? 0 : S; k < S; ++k) {   // a group per stage, empty or not
                if (k == 1) convert_q();
                if (ipos < hi) issue();
                commit_group();
            }
            if (segn) convert_q();
            const int32_t c0 = s.c, c_end = min(s.nc, s.c + hi - pos);
            const int32_t n = clamp_len(pa::ld_behind_wait(p.context_lens + s.i), max_len);
            // Running state for heads 8 nt + 2 c4 + {0, 1} (kG4: of that modulo 4): the negative
            // of the maximum (bias; the logits below are relative to it), sum, sums of P times
            // V's minima; o: rows are values 64 g + 8 cr + u (e < 2) and + 4 + u.
            float bias[NT][NJ], l_run[NT][NJ], lowv[NT][NG][NJ], o[NG][4][NT][4], mid[NT][4];
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
                for (int j = 0; j < NJ; ++j) {
                    bias[nt][j] = 0.f;
                    l_run[nt][j] = 0.f;
#pragma unroll
                    for (int g = 0; g < NG; ++g) lowv[nt][g][j] = 0.f;
                }
#pragma unroll
                for (int g = 0; g < NG; ++g)
#pragma unroll
                    for (int u = 0; u < 4; ++u)
                        o[g][u][nt][0] = o[g][u][nt][1] = o[g][u][nt][2] = o[g][u][nt][3] = 0.f;
                mid[nt][0] = mid[nt][1] = mid[nt][2] = mid[nt][3] = 0.f;
            }
            bool fresh = true;   // no maximum yet
            int32_t valid = n - c0 * kChunk;   // tokens of the context from the chunk on
#pragma unroll 1
            for (int32_t c = c0; c < c_end;) {
                const int32_t stop = min(c + kSettle, c_end);
#pragma unroll 1
                for (; c < stop; ++c, valid -= kChunk) {
                    wait_group<S - 1>();
                    __syncwarp();   // every lane's copies have landed
                    {
                        const uint32_t kt = stage + koff, vt0 = stage + voff0, vt1 = stage + voff1;
                        const uint32_t st_at = stage + 2 * kCodes + lane * kSRow;
                        // ---- S^T = K Q^T over the codes, per group
                        float st[kTiles][NG][NT][4];
#pragma unroll
                        for (int mt = 0; mt < kTiles; ++mt)
#pragma unroll
                            for (int g = 0; g < NG; ++g) {
#pragma unroll
                                for (int nt = 0; nt < NT; ++nt)
                                    st[mt][g][nt][0] = st[mt][g][nt][1] = st[mt][g][nt][2] = st[mt][g][nt][3] = 0.f;
                                const uint2 w0 = pa::lds64(kt + 16 * mt * kRow + 32 * g);
                                const uint2 w1 = pa::lds64(kt + (16 * mt + 8) * kRow + 32 * g);
#pragma unroll
                                for (int ks = 0; ks < 4; ++ks) {
                                    const uint32_t y0 = (ks < 2 ? w0.x : w0.y) >> (8 * (ks & 1));
                                    const uint32_t y1 = (ks < 2 ? w1.x : w1.y) >> (8 * (ks & 1));
                                    const uint32_t a[4] = {y0 & kLowNibbles, y1 & kLowNibbles,
                                                           y0 & kHighNibbles, y1 & kHighNibbles};
#pragma unroll
                                    for (int nt = 0; nt < NT; ++nt)
                                        pa::mma_16816<false>(st[mt][g][nt], a, qb[nt][g][ks][0], qb[nt][g][ks][1]);
                                }
                            }
                        // ---- steps and minima: lane r takes row r of the chunk to fp32, K's
                        // steps with the score's factor, for all lanes to read
                        {
                            float kv[2 * NG], vv[2 * NG];
                            load_f16_scales<NG>(st_at, kv);
                            load_f16_scales<NG>(st_at + kScales, vv);
                            if (lane >= valid)   // a row past the context may hold anything
#pragma unroll
                                for (int g = 0; g < 2 * NG; ++g) vv[g] = 0.f;
#pragma unroll
                            for (int g = 0; g < NG; ++g) {
                                kv[2 * g] *= qsc;
                                vv[2 * g + 1] += 8.f * vv[2 * g];   // the value of code 8
                                vv[2 * g] *= pa::exp2_int(kUp);
                            }
                            store_row<NG>(krows + lane * NG * 8, kv);
                            store_row<NG>(vrows + lane * NG * 8, vv);
                        }
                        __syncwarp();
                        // ---- base-2 logits, relative to the running maxima
                        float x[kTiles][NT][2][NJ];   // [key half][head]
#pragma unroll
                        for (int mt = 0; mt < kTiles; ++mt)
#pragma unroll
                            for (int r = 0; r < 2; ++r) {
                                float kv[2 * NG];
                                load_row<NG>(krow + (16 * mt + 8 * r) * NG * 8, kv);
#pragma unroll
                                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                                    for (int j = 0; j < NJ; ++j) {
                                        float v = bias[nt][j];
#pragma unroll
                                        for (int g = 0; g < NG; ++g) v += kv[2 * g + 1] * qsum[nt][g][j];
#pragma unroll
                                        for (int g = 0; g < NG; ++g) v += kv[2 * g] * st[mt][g][nt][2 * r + j];
                                        x[mt][nt][r][j] = v;
                                    }
                            }
                        if (valid < kChunk)   // the context's last chunk
#pragma unroll
                            for (int mt = 0; mt < kTiles; ++mt)
#pragma unroll
                                for (int r = 0; r < 2; ++r)
#pragma unroll
                                    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                                        for (int j = 0; j < NJ; ++j)
                                            if (16 * mt + cr + 8 * r >= valid) x[mt][nt][r][j] = -INFINITY;
                        // ---- online softmax per head
                        float top[NT][NJ];
                        bool above = fresh;
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                            for (int j = 0; j < NJ; ++j) {
                                top[nt][j] = x[0][nt][0][j];
#pragma unroll
                                for (int mt = 0; mt < kTiles; ++mt)
                                    top[nt][j] = fmaxf(top[nt][j], fmaxf(x[mt][nt][0][j], x[mt][nt][1][j]));
                                above |= top[nt][j] > kLazy;
                            }
                        if (__any_sync(0xffffffffu, above)) {
#pragma unroll
                            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                                for (int j = 0; j < NJ; ++j) {
                                    float v = top[nt][j];
                                    v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 4));
                                    v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 8));
                                    v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 16));
                                    const float up = fresh ? v : fmaxf(v, 0.f);
                                    const float a = fresh ? 0.f : pa::fast_exp2(-up);
                                    bias[nt][j] -= up;
#pragma unroll
                                    for (int mt = 0; mt < kTiles; ++mt)
#pragma unroll
                                        for (int r = 0; r < 2; ++r) x[mt][nt][r][j] -= up;
                                    l_run[nt][j] *= a;
#pragma unroll
                                    for (int g = 0; g < NG; ++g) {
                                        lowv[nt][g][j] *= a;
#pragma unroll
                                        for (int i = j; i <= (kOne ? 1 : j); ++i) {
                                            mid[nt][2 * g + i] *= a;
#pragma unroll
                                            for (int u = 0; u < 4; ++u) {
                                                o[g][u][nt][i] *= a;
                                                o[g][u][nt][2 + i] *= a;
                                            }
                                        }
                                    }
                                }
                        }
                        fresh = false;
                        // ---- P, and O^T += V^T P^T
#pragma unroll
                        for (int mt = 0; mt < kTiles; ++mt) {
                            uint32_t pb[NG][NT][2], pl[NG][NT][2];   // the two parts of P times V's step
#pragma unroll
                            for (int r = 0; r < 2; ++r) {
                                float vv[2 * NG];
                                load_row<NG>(vrow + (16 * mt + 8 * r) * NG * 8, vv);
#pragma unroll
                                for (int nt = 0; nt < NT; ++nt) {
                                    float e[2] = {0.f, 0.f};
#pragma unroll
                                    for (int j = 0; j < NJ; ++j) {
                                        e[j] = pa::fast_exp2(x[mt][nt][r][j]);
                                        l_run[nt][j] += e[j];
                                    }
#pragma unroll
                                    for (int g = 0; g < NG; ++g) {
                                        const float y0 = e[0] * vv[2 * g], y1 = e[1] * vv[2 * g];
                                        const float h0 = upper_half(y0), h1 = upper_half(y1);
                                        if constexpr (kOne) {
                                            pb[g][nt][r] = pa::movmatrix_trans(pa::pack2<true>(h0, y0 - h0));
                                        } else if constexpr (kDup) {
                                            pb[g][nt][r] = pa::movmatrix_trans(
                                                pa::pack2<true>(fmaf(dup, y0, -h0), fmaf(dup, y1, -h1)));
                                        } else {
                                            pb[g][nt][r] = pa::movmatrix_trans(__byte_perm(
                                                __float_as_uint(y0), __float_as_uint(y1), 0x7632));
                                            pl[g][nt][r] = pa::movmatrix_trans(pa::pack2<true>(y0 - h0, y1 - h1));
                                        }
#pragma unroll
                                        for (int j = 0; j < NJ; ++j) lowv[nt][g][j] += e[j] * vv[2 * g + 1];
                                    }
                                }
                            }
                            // The fragment's key pairs: 16 mt + 8 r + 2 c4 + {0, 1}; odd c4 read
                            // the pair's second row first, so that the four rows of a load lie in
                            // both halves of the 128 bytes, and swap in the byte permutation.
#pragma unroll
                            for (int g = 0; g < NG; ++g) {
                                uint32_t z[2][2];   // [key half][values 0..3 | 4..7]
#pragma unroll
                                for (int r = 0; r < 2; ++r) {
                                    const uint32_t w0 = lds32(vt0 + (16 * mt + 8 * r) * kRow + 32 * g);
                                    const uint32_t w1 = lds32(vt1 + (16 * mt + 8 * r) * kRow + 32 * g);
                                    z[r][0] = __byte_perm(w0, w1, perm0);
                                    z[r][1] = __byte_perm(w0, w1, perm1);
                                }
                                // One product behind, the second parts: no two in a row into one
                                // accumulator.
                                constexpr bool kTwo = !kOne && !kDup;
                                uint32_t a[4] = {}, was[4];
#pragma unroll
                                for (int u = 0; u < 4; ++u) {
                                    // u even: the byte's lower code; u odd: the whole byte, lower
                                    // code plus 16 times the upper one, which the end takes apart
                                    const uint32_t mask = u & 1 ? kBytes : kLowNibbles;
#pragma unroll
                                    for (int q = 0; q < 4; ++q) {
                                        const uint32_t w = z[q >> 1][q & 1];
                                        was[q] = a[q];
                                        // bytes 1 and 3 to the low half of each half
                                        a[q] = (u < 2 ? w : __byte_perm(w, 0, 0x4341)) & mask;
                                    }
#pragma unroll
                                    for (int nt = 0; nt < NT; ++nt) {
                                        pa::mma_16816<true>(o[g][u][nt], a, pb[g][nt][0], pb[g][nt][1]);
                                        if (u == 0) pa::mma_16816<true>(mid[nt], eights[g], pb[g][nt][0], pb[g][nt][1]);
                                    }
                                    if constexpr (kTwo)
#pragma unroll
                                        for (int nt = 0; nt < NT; ++nt) {
                                            if (u > 0) pa::mma_16816<true>(o[g][u - 1][nt], was, pl[g][nt][0], pl[g][nt][1]);
                                            if (u == 3) pa::mma_16816<true>(mid[nt], eights[g], pl[g][nt][0], pl[g][nt][1]);
                                            if (u == 3) pa::mma_16816<true>(o[g][u][nt], a, pl[g][nt][0], pl[g][nt][1]);
                                        }
                                }
                            }
                        }
                    }
                    __syncwarp();   // every lane has read the stage: it may be filled again
                    stage = stage + kStage == ring + S * kStage ? ring : stage + kStage;
                    if (ipos < hi) issue();
                    commit_group();
                }
                // The codes' middle leaves o, while it is small.
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int g = 0; g < NG; ++g)
#pragma unroll
                        for (int j = 0; j < (kOne ? 2 : NJ); ++j) {
#pragma unroll
                            for (int u = 0; u < 4; ++u)
#pragma unroll
                                for (int e = j; e < 4; e += 2)
                                    o[g][u][nt][e] -= (u & 1 ? 17.f : 1.f) * mid[nt][2 * g + j];
                            mid[nt][2 * g + j] = 0.f;
                        }
            }
            pos += c_end - c0 + (c_end == s.nc ? kPairCost : 0);

            // ---- the pair's chunks of this warp are done
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int j = 0; j < NJ; ++j) {
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
                                          : (uint32_t)warp * S * kStage;
            float* slot = reinterpret_cast<float*>(smem + at);
            // Both parts of P in one lane; in kG4 the lanes with the second part have the others'.
            auto both = [&](const float (&acc)[4], int i) { return kOne ? acc[i] + acc[i + 1] : acc[i]; };
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int j = 0; j < NJ; ++j) {
                    const int h = 8 * nt + 2 * c4 + j;
                    if (!kDup && h >= G) continue;
                    const float inv = whole ? 1.f / l_run[nt][j] : 1.f;
                    if (!whole && cr == 0 && h < G) {
                        slot[h] = -bias[nt][j];
                        slot[G + h] = l_run[nt][j];
                    }
#pragma unroll
                    for (int g = 0; g < NG; ++g) {
                        float v[8];
#pragma unroll
                        for (int u = 0; u < 8; ++u) {
                            const int e = 2 * (u >> 2) + j;
                            const float even = both(o[g][u & 2][nt], e);
                            const float code = u & 1 ? (both(o[g][u & 3][nt], e) - even) * 0.0625f : even;
                            const float sum = code * pa::exp2_int(133 - kUp);
                            if constexpr (kDup) {
                                const float part = c4 < 2 ? lowv[nt][g][j] - sum : sum;
                                v[u] = (part + __shfl_xor_sync(0xffffffffu, part, 2)) * inv;
                            } else {
                                v[u] = (sum + lowv[nt][g][j]) * inv;
                            }
                        }
                        const int at_d = 64 * g + 8 * cr;
                        if (kDup && (h >= G || c4 >= 2)) continue;
                        if (whole) {
                            *reinterpret_cast<uint4*>(p.out + ((int64_t)s.i * p.H + s.g * G + h) * D + at_d) =
                                make_uint4(pa::pack2<kBF16>(v[0], v[1]), pa::pack2<kBF16>(v[2], v[3]),
                                           pa::pack2<kBF16>(v[4], v[5]), pa::pack2<kBF16>(v[6], v[7]));
                        } else {
                            float4* to = reinterpret_cast<float4*>(slot + slot_head(G) + h * D + at_d);
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
                r.a = s.a;
            }
            ++segn;
            if (pos < hi) s = next_pair(prefix, Hkv, s);
        }
    }
    asm volatile("griddepcontrol.launch_dependents;");   // a next call may be launched: it waits
    __syncthreads();

    // Plain fields, not an Out among the parameters: with one, registers fall differently, and forms
    // spill that do not as it is (G = 16 in blocks of 32 at d = 64 took 63 us for 59, 8 x 32768 tokens).
    join_runs<D, kBF16>(Out{p.out, p.counters, p.partials, p.H, p.Hkv, p.G}, cut, cta_lo, nw, smem, S * kStage,
                        L.slots, runs, is_last, scan);
}

// ---- host side -----------------------------------------------------------------

// As many warps as shared memory holds rings and slots for; 0: not even four.
int choose_warps(int D, int G, int B) {
    for (int w = max_warps(D, form_of(G)); w >= 4; --w)
        if (layout_of(D, G, B, w).total <= kSmemBudget) return w;
    return 0;
}

template <int D, bool kBF16, int kForm, int kShift>
pa_status launch(const Int4Params& p, cudaStream_t stream) {
    auto kern = decode_int4_kernel<D, kBF16, kForm, kShift>;
    static pa::DeviceOnce once;
    if (!pa::allow_smem(once, kern, kSmemBudget)) return PA_ERR_CUDA;
    int ctas = pa::device_sm_count();
    if (ctas <= 0) return PA_ERR_CUDA;
    if (ctas > kMaxCtas) ctas = kMaxCtas;
    const Layout L = layout_of(D, p.G, p.B, p.warps);
    // Started early, so that its launch hides behind the append's or another call's end.
    cudaLaunchAttribute attr{};
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)ctas);
    cfg.blockDim = dim3((unsigned)p.warps * 32);
    cfg.dynamicSmemBytes = L.total;
    cfg.stream = stream;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    return pa::cuda_status(cudaLaunchKernelEx(&cfg, kern, p));
}

template <int D, bool kBF16, int kForm>
pa_status launch_b(const Int4Params& p, cudaStream_t stream) {
    if (p.bs_shift == 3) return launch<D, kBF16, kForm, 3>(p, stream);
    if (p.bs_shift == 4) return launch<D, kBF16, kForm, 4>(p, stream);
    return launch<D, kBF16, kForm, 5>(p, stream);
}

template <int D, bool kBF16>
pa_status launch_g(const Int4Params& p, cudaStream_t stream) {
    switch (form_of(p.G)) {
        case kG1: return launch_b<D, kBF16, kG1>(p, stream);
        case kG4: return launch_b<D, kBF16, kG4>(p, stream);
        case kG8: return launch_b<D, kBF16, kG8>(p, stream);
        default: return launch_b<D, kBF16, kG16>(p, stream);
    }
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
    if ((int64_t)num_blocks * Hkv > INT32_MAX || B > kMaxBatch || (int64_t)num_blocks * block_size > INT32_MAX ||
        (int64_t)max_blocks * block_size > INT32_MAX)
        return PA_ERR_UNSUPPORTED;
    // A block's codes over all KV heads are counted in 32 bits.
    if ((int64_t)Hkv * (d / 2) * block_size > UINT32_MAX) return PA_ERR_UNSUPPORTED;
    // Positions in the list are int32.
    const int64_t max_chunks = ((int64_t)max_blocks * block_size + kChunk - 1) / kChunk;
    if ((int64_t)B * Hkv * subs * (max_chunks + kPairCost) >= ((int64_t)1 << 30)) return PA_ERR_UNSUPPORTED;
    if (B > 0 && ws_bytes < pa_decode_workspace_size(B, H, d)) return PA_ERR_INVALID;
    if (B == 0) return PA_OK;
    if (!q || !k_cache || !v_cache || !k_scale || !v_scale || !block_tables || !context_lens ||
        !out || !workspace)
        return PA_ERR_INVALID;
    if ((reinterpret_cast<uintptr_t>(k_cache) | reinterpret_cast<uintptr_t>(v_cache) |
         reinterpret_cast<uintptr_t>(k_scale) | reinterpret_cast<uintptr_t>(v_scale) |
         reinterpret_cast<uintptr_t>(q) | reinterpret_cast<uintptr_t>(out) |
         reinterpret_cast<uintptr_t>(workspace)) & 15u)
        return PA_ERR_INVALID;
    Int4Params p;
    p.warps = choose_warps(d, G, B);
    if (!p.warps) return PA_ERR_UNSUPPORTED;
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
    p.partials = reinterpret_cast<float*>(static_cast<unsigned char*>(workspace) + ticket_bytes(B, H));
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
    if (d == 128)
        return dtype == PA_BF16 ? launch_g<128, true>(p, st) : launch_g<128, false>(p, st);
    return dtype == PA_BF16 ? launch_g<64, true>(p, st) : launch_g<64, false>(p, st);
}

}  // extern "C"
