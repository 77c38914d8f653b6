// Paged decode attention over the block-scaled 8-bit cache (pa_decode_int8_block /
// pa_decode_fp8_block): what pa_decode computes, with K and V the rows that the codes of
// pa_reshape_and_cache_int8_block / _fp8_block stand for (format: pa_cache_block8.cu).
//
// With x = s c for the codes c of a (block, KV head), the scale leaves both sums over codes:
//     q . K_j = s_b (q . c_j),   sum_j p_j V_j = sum_j (p_j s_b) c_j,
// one factor a block where the 8-bit caches with a scale per token have one a key.
//
// Codes meet the tensor cores with little or no conversion:
//  * an INT8 code plus 128, u, is the f16 subnormal u 2^-24 and the bf16 number u 2^-133 as it
//    stands, a byte under zeros; the xor that adds the 128 is part of the mask's instruction.
//    K's 128 leaves as the sums' first value, -128 sum q; V's as a product of its own, P times
//    a tile of 128s, subtracted every four chunks, so that what the tensor cores cut off
//    their sums they cut off both, and the sums stay small between two subtractions.
//  * an E4M3 code goes to f16 by conversion for K, two an instruction.  V has to be bf16, as P is
//    and both operands of a product have one type, and there is no conversion to it: the code's
//    seven lower bits are put under a bf16's exponent, its sign above, which is the number
//    times 2^-120, exactly, subnormals as subnormals, in 3.5 instructions for two codes.
// P is bf16 in either case: P times the block's V scale goes in two parts, its upper half
// and what that leaves, rounded: 16 bits, whatever the other blocks' scales are.  A power of two,
// from a run's first V scale, keeps the products clear of both ends of fp32's range: a scale 2^40
// times that one moves it, one 2^-64 of it still has all its bits.
//
// What bounds it is HBM: 256 bytes a token and KV head at d = 128.  Every warp streams a run of
// 32-token chunks through a ring of its own in shared memory (pa_runs.cuh), by asynchronous
// 16-byte copies that put each row's 16-byte columns where neither product's reads meet in a
// bank, and by 4-byte copies of the blocks' scales.
//
// Measured (device time): 16 x 32768 tokens of 8 KV heads at d = 128, E4M3: G = 1 169 us, G = 4
// 171 (6.3 TB/s, 94 % of the measured copy; DRAM traffic 1.003 times the bytes, 45 % of the
// ALU's and 15 % of the tensor pipe's cycles, 40 % of the issue slots), G = 8 176, G = 16 185;
// INT8: 172, 173, 174, 195; at d = 64 88 to 95 us up to G = 8; 64 sequences of 128 .. 2048 tokens,
// 40 heads, G = 1: INT8 118 us, E4M3 116; 4 sequences of up to 64 tokens 6.4 us, all latency.
// The caches with a scale per token take 159 us (E4M3) and 175 (INT8) for a 40-head batch of
// nearly this size: a conversion and a factor per key, and loading warps to wait for.
#pragma once

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
__host__ __device__ constexpr int ring_stages(int D) { return D == 128 ? 2 : 3; }
// K and V codes of a chunk; the scales of up to four blocks, K's and V's.
__host__ __device__ constexpr uint32_t stage_bytes(int D) { return 2u * kChunk * D + 32; }
constexpr float kLog2e = 1.4426950408889634f;

struct Block8Params {
    const uint16_t* q;
    const uint8_t *k_cache, *v_cache;
    const float *k_scale, *v_scale;
    const int32_t* block_tables;
    const int32_t* context_lens;
    Out out;
    unsigned int* err;
    // A KV head with more than kMaxG query heads is `subs` pairs of kMaxG heads.
    int32_t max_blocks, B, num_blocks, subs, warps;
    float scale_log2;
};

// The forms of the kernel by query heads of a KV head: one; up to 4; up to 8; up to 16.
enum Form { kG1, kG4, kG8, kG16 };
constexpr Form form_of(int G) { return G == 1 ? kG1 : G <= 4 ? kG4 : G <= 8 ? kG8 : kG16; }
// One CTA per SM, of as many warps as the registers of a chunk leave: at d = 128 twelve of
// 168, at d = 64 sixteen of 128; where 9 .. 16 heads need two 8-wide MMA tiles and twice the
// accumulators eight of 255 at d = 128, and at d = 64 twelve, which spill (16 x 32768 tokens of 8 KV
// heads, G = 16: INT8 120 us, E4M3 108; with eight, which do not, 126 and 116; ten leave the four
// schedulers uneven: 137 and 126).
__host__ __device__ constexpr int max_warps(int D, int form) {
    return form == kG16 ? (D == 128 ? 8 : 12) : D == 128 ? 12 : 16;
}
constexpr uint32_t kSmemBudget = 227 * 1024;

__device__ __forceinline__ uint32_t lds32(uint32_t addr) {
    uint32_t v;
    asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(addr));
    return v;
}

template <bool kBF16>
__device__ __forceinline__ float2 widen2(uint32_t v) {
    if constexpr (kBF16)
        return make_float2(__uint_as_float(v << 16), __uint_as_float(v & 0xFFFF0000u));
    __half2 h;
    memcpy(&h, &v, 4);
    return __half22float2(h);
}

constexpr uint32_t kBytes = 0x00FF00FFu, kSign = 0x00800080u;

// K's codes of four neighbouring channels as two f16 pairs: INT8 channels (0, 2) and (1, 3),
// each (c + 128) 2^-24; E4M3 channels (0, 1) and (2, 3), c.
template <bool kInt8>
__device__ __forceinline__ void k_pairs(uint32_t w, uint32_t& a, uint32_t& b) {
    if constexpr (kInt8) {
        a = (w & kBytes) ^ kSign;
        b = ((w >> 8) & kBytes) ^ kSign;
    } else {
        pa::e4m3x4_to_f16(w, a, b);
    }
}

// V's codes in the lower (u = 0) or upper (u = 1) bytes of both halves, as a pair of bf16:
// INT8 (c + 128) 2^-133, E4M3 c 2^-120.
template <bool kInt8>
__device__ __forceinline__ uint32_t v_pair(uint32_t w, int u) {
    if constexpr (kInt8) return ((u ? w >> 8 : w) & kBytes) ^ kSign;
    return ((u ? w >> 4 : w << 4) & 0x07F007F0u) | ((u ? w : w << 8) & 0x80008000u);
}
template <bool kInt8>
constexpr float kVUnit = kInt8 ? 8589934592.f : 1048576.f;   // 2^33, 2^20: over 2^100

// A head's running maximum is raised only when a logit exceeds it by more than this
// (base 2): probabilities reach 2^8, which fp32 sums bear, and most chunks need neither the
// maximum across lanes nor a rescale.
constexpr float kLazy = 8.f;
constexpr int kSettle = 4;   // chunks between two subtractions of the codes' middle
// The V scales' power of two takes a run's first (largest of a chunk) scale to 2^64, from where
// the products with codes 2^-133 of theirs have room to both sides, and is changed once a scale
// passes 2^104.
constexpr int kUp = 64;
constexpr float kTooHigh = 2.028240960365167e31f;   // 2^104

// A float's upper half as a float: a bf16 number, toward zero.
__device__ __forceinline__ float upper_half(float x) {
    return __uint_as_float(__float_as_uint(x) & 0xFFFF0000u);
}

// kG1: a lane tracks one column, head 0, instead of two; the next one is the second part of P.
// kG4: columns h and h + 4 are both head h, the latter with the second part of P and the
// former with minus the first.
template <int D, bool kBF16, bool kInt8, int kForm, int kShift>
__global__ void __launch_bounds__(max_warps(D, kForm) * 32, 1) decode_block8_kernel(const Block8Params p) {
    constexpr bool kOne = kForm == kG1, kDup = kForm == kG4;
    constexpr int NT = kForm == kG16 ? 2 : 1, NJ = kOne ? 1 : 2;
    constexpr int KS = D / 16;                   // k-steps of the scores, and 16-row tiles of O^T
    constexpr int NW = D / 32;                   // words of a key's V row that a lane has
    constexpr uint32_t kCodes = kChunk * D, kStage = stage_bytes(D);
    constexpr int S = ring_stages(D);
    constexpr int bs_shift = kShift, bmask = (1 << kShift) - 1;
    constexpr int bpc = kChunk >> bs_shift;      // blocks per chunk: 4, 2 or 1
    const int32_t B = p.B, Hkv = p.out.Hkv, G = p.out.G;
    const int nw = p.warps;
    const Layout L = make_layout(nw * S * kStage, D, G, B, nw);
    extern __shared__ __align__(128) unsigned char smem[];
    const uint32_t sbase = pa::smem_addr(smem);
    Run* runs = reinterpret_cast<Run*>(smem + L.runs);
    int32_t* is_last = reinterpret_cast<int32_t*>(smem + L.last);
    int32_t* scan = reinterpret_cast<int32_t*>(smem + L.scan);
    int32_t* prefix = reinterpret_cast<int32_t*>(smem + L.prefix);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int32_t max_len = p.max_blocks << bs_shift;

    asm volatile("griddepcontrol.launch_dependents;");   // a next call may be launched: it waits
    asm volatile("griddepcontrol.wait;" ::: "memory");   // launched while the kernel before may run

    // The tables and queries are read a dependent load or two from now: into L2 with
    // them, a line per thread (what they cover is shared by all CTAs).
    {
        const int64_t line = ((int64_t)blockIdx.x * nw * 32 + tid) * 128;
        if (line < (int64_t)B * p.max_blocks * 4)
            prefetch_l2(reinterpret_cast<const char*>(p.block_tables) + line);
        if (line < (int64_t)B * p.out.H * D * 2) prefetch_l2(reinterpret_cast<const char*>(p.q) + line);
    }
    const int32_t W = list_prefix(p.context_lens, B, Hkv, max_len, p.err, nw, prefix, scan, is_last, runs);

    // ---- zero rows of empty contexts
#pragma unroll 1
    for (int32_t i = blockIdx.x; i < B; i += gridDim.x) {
        if (prefix[i + 1] != prefix[i]) continue;
        uint4* row = reinterpret_cast<uint4*>(p.out.out + (int64_t)i * p.out.H * D);
#pragma unroll 1
        for (int v = tid; v < p.out.H * D / 8; v += nw * 32) row[v] = make_uint4(0, 0, 0, 0);
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

    Cursor start{};
    int32_t ipos = hi;              // next chunk to issue
    if (lo < hi) {
        start = find(prefix, B, Hkv, lo);
        ipos = start.a + kPairCost + start.c;
    }
    if (ipos < hi) {
        // ================= loading: this warp's chunks, in order =================
        // A copy instruction moves 512 bytes, kPass rows of codes.  Row r's 16-byte column c
        // goes to column c ^ (r % 8) at d = 128; at d = 64 two rows share 128 bytes, and column
        // 4 (r % 2) + c of them goes to that ^ 2 (r / 2 % 4): then the reads of the scores
        // (eight neighbouring columns of two rows) and of the outputs (one or two columns of
        // every other row) both take each bank once.
        constexpr int kPass = 512 / D, kPasses = (1 << bs_shift) / kPass;
        const uint32_t lrow = lane / (D / 16), lcol = lane % (D / 16);
        const uint32_t to_lane = D == 128 ? lrow * 128 + ((lcol ^ lrow) << 4)
                                          : (lrow >> 1) * 128 + (((4 * (lrow & 1) + lcol) ^ (lrow & 6)) << 4);
        constexpr uint32_t kTile = (uint32_t)D << bs_shift;
        const uint32_t heads = (uint32_t)(Hkv / p.subs), stride = heads * kTile;
        const float* scales = lane & 4 ? p.v_scale : p.k_scale;
        const uint64_t policy = pa::l2_policy_evict_first();
        // A pair's table entries, 32 at a time (lane l holds the window's entry l), with
        // the window after it loaded a step ahead; an entry past the context is -1, as is
        // an id outside the pool.
        struct Walk {
            Cursor s;
            int32_t at;              // the chunk's first block in the window
            int32_t went, wnext;
            int32_t next, nb;        // this lane's entry after wnext's; blocks of the context
            const uint8_t *k, *v;    // the pair's KV head in each tensor, at this lane's bytes
            const float* sc;
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
            w.k = p.k_cache + (uint64_t)head * kTile + lane * 16;
            w.v = p.v_cache + (uint64_t)head * kTile + lane * 16;
            w.sc = scales + head;
            return w;
        };
        uint32_t ito = ring;            // its stage
        Walk cur = open(start);
        // One chunk's copies, as one group.  Blocks past the context and ids outside the
        // pool are not read: zeros take their place, scales of zero among them.
        auto issue = [&]() {
#pragma unroll
            for (int b = 0; b < bpc; ++b) {
                const int32_t blk = __shfl_sync(0xffffffffu, cur.went, cur.at + b);
                const uint64_t at = (uint64_t)(uint32_t)max(blk, 0) * stride;
                const uint32_t to = ito + b * kTile;
#pragma unroll
                for (int t = 0; t < kPasses; ++t) {
                    const uint32_t off = t * 512;
                    const uint32_t x = D == 128 && t & 1 ? to_lane ^ 64 : to_lane;   // rows 4 .. 7 of eight
                    copy16(to + off + x, cur.k + at + off, blk >= 0, policy);
                    copy16(to + off + x + kCodes, cur.v + at + off, blk >= 0, policy);
                }
            }
            const int32_t sblk = __shfl_sync(0xffffffffu, cur.went, cur.at + (lane & 3));
            if (lane < 8 && (lane & 3) < bpc)
                copy4(ito + 2 * kCodes + lane * 4, cur.sc + (uint64_t)(uint32_t)max(sblk, 0) * heads, sblk >= 0);
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
        uint32_t qb[NT][KS][2];         // Q^T fragments: lane holds query head 8 nt + cr
        float qoff[NT][2];              // INT8: -128 sum q, heads 8 nt + 2 c4 + {0, 1}
        float qsc = 0.f;                // from an MMA score over a scale to a base-2 logit
        // In k-step ks the lane's fragment holds channels v0 + {0, 1, 2, 3} with v0 =
        // D / 4 c4 + 4 ks, paired as k_pairs pairs the codes.  q is scaled by 2^e so that its
        // largest value lies in [2^14, 2^15).
        uint32_t raw[NT][D / 8];
        auto fetch_q = [&](const Cursor& s) {
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                const int h = kDup ? cr & 3 : 8 * nt + cr;
                const uint4* row = reinterpret_cast<const uint4*>(
                    p.q + ((int64_t)s.i * p.out.H + s.g * G + h) * D + D / 4 * c4);
#pragma unroll
                for (int x = 0; x < D / 32; ++x) {
                    const uint4 a = h < G ? pa::ld_behind_wait(row + x) : make_uint4(0, 0, 0, 0);
                    raw[nt][4 * x] = a.x, raw[nt][4 * x + 1] = a.y;
                    raw[nt][4 * x + 2] = a.z, raw[nt][4 * x + 3] = a.w;
                }
            }
        };
        auto convert_q = [&]() {
            float amax = 0.f;
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int w = 0; w < D / 8; ++w) {
                    const float2 f = widen2<kBF16>(raw[nt][w]);
                    amax = fmaxf(amax, fmaxf(fabsf(f.x), fabsf(f.y)));
                }
            amax = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(amax)));
            const int e = min(141 - pa::biased_exponent(amax), 126);
            const float up = pa::exp2_int(e);   // e >= -113
            qsc = p.scale_log2 * pa::exp2_int(max(-126, min((kInt8 ? 24 : 0) - e, 127)));
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                float sum = 0.f;
#pragma unroll
                for (int ks = 0; ks < KS; ++ks) {
                    const float2 a = widen2<kBF16>(raw[nt][2 * ks]), b = widen2<kBF16>(raw[nt][2 * ks + 1]);
                    qb[nt][ks][0] = pa::pack2<false>(a.x * up, (kInt8 ? b.x : a.y) * up);
                    qb[nt][ks][1] = pa::pack2<false>((kInt8 ? a.y : b.x) * up, b.y * up);
                    if constexpr (kInt8) {
                        const float2 x = widen2<false>(qb[nt][ks][0]), y = widen2<false>(qb[nt][ks][1]);
                        sum += (x.x + x.y) + (y.x + y.y);
                    }
                }
                if constexpr (kInt8) {
                    sum *= -128.f * 5.9604644775390625e-8f;   // 2^-24, the codes' unit
                    sum += __shfl_xor_sync(0xffffffffu, sum, 1);
                    sum += __shfl_xor_sync(0xffffffffu, sum, 2);
                    qoff[nt][0] = __shfl_sync(0xffffffffu, sum, 8 * c4);
                    qoff[nt][1] = __shfl_sync(0xffffffffu, sum, 8 * c4 + 4);
                }
            }
        };

        Cursor s = start;
        uint32_t stage = ring;   // the chunk to compute
        // Offsets of this lane in a stage: its columns of K rows cr, and of V rows 2 c4 + {0, 1}.
        uint32_t koff[D / 64], voff[2];
#pragma unroll
        for (int x = 0; x < D / 64; ++x)
            koff[x] = D == 128 ? cr * 128 + (((2 * c4 + x) ^ cr) << 4)
                               : (cr >> 1) * 128 + (((4 * (cr & 1) + c4) ^ (cr & 6)) << 4);
#pragma unroll
        for (int i = 0; i < 2; ++i)
            voff[i] = kCodes + (D == 128 ? (2 * c4 + i) * 128 + ((cr ^ (2 * c4 + i)) << 4)
                                         : c4 * 128 + (((4 * i + (cr >> 1)) ^ (2 * c4)) << 4) + 8 * (cr & 1));
        constexpr uint32_t k128 = 0x00800080u;
        const uint32_t all128[4] = {k128, k128, k128, k128};
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
            // of the maximum (bias; the logits below are relative to it), sum; o: rows are channels
            // D / 8 cr + mt (e < 2) and + D / 16; vref: the V scales' power of two, 0 before any.
            float bias[NT][NJ], l_run[NT][NJ], o[KS][NT][4], mid[NT][4], vref = 0.f;
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
                for (int j = 0; j < NJ; ++j) {
                    bias[nt][j] = 0.f;
                    l_run[nt][j] = 0.f;
                }
#pragma unroll
                for (int mt = 0; mt < KS; ++mt)
                    o[mt][nt][0] = o[mt][nt][1] = o[mt][nt][2] = o[mt][nt][3] = 0.f;
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
                        // ---- S^T = K Q^T over the codes
                        float st[kTiles][NT][4];
#pragma unroll
                        for (int mt = 0; mt < kTiles; ++mt) {
#pragma unroll
                            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                                for (int e = 0; e < 4; ++e) st[mt][nt][e] = kInt8 ? qoff[nt][e & 1] : 0.f;
                            uint32_t w[2][D / 16];
#pragma unroll
                            for (int r = 0; r < 2; ++r)
#pragma unroll
                                for (int x = 0; x < D / 64; ++x) {
                                    const uint4 y = pa::lds128(stage + koff[x] + (16 * mt + 8 * r) * D);
                                    w[r][4 * x] = y.x, w[r][4 * x + 1] = y.y;
                                    w[r][4 * x + 2] = y.z, w[r][4 * x + 3] = y.w;
                                }
#pragma unroll
                            for (int ks = 0; ks < KS; ++ks) {
                                uint32_t a[4];
                                k_pairs<kInt8>(w[0][ks], a[0], a[2]);
                                k_pairs<kInt8>(w[1][ks], a[1], a[3]);
#pragma unroll
                                for (int nt = 0; nt < NT; ++nt)
                                    pa::mma_16816<false>(st[mt][nt], a, qb[nt][ks][0], qb[nt][ks][1]);
                            }
                        }
                        // ---- the blocks' scales: the score's factor, V's under its power of two
                        float ks_[bpc], vs_[bpc], top_v = 0.f;
#pragma unroll
                        for (int b = 0; b < bpc; ++b) {
                            ks_[b] = pa::lds_f32(stage + 2 * kCodes + 4 * b) * qsc;
                            vs_[b] = pa::lds_f32(stage + 2 * kCodes + 16 + 4 * b);
                            top_v = fmaxf(top_v, vs_[b]);
                        }
                        if (vref == 0.f ? top_v > 0.f : top_v * vref > kTooHigh) {   // the same in all lanes
                            const float now = pa::exp2_int(min(127, kUp + 127 - pa::biased_exponent(top_v)));
                            const float f = vref == 0.f ? 0.f : now / vref;
#pragma unroll
                            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                                for (int e = 0; e < 4; ++e) {
                                    mid[nt][e] *= f;
#pragma unroll
                                    for (int mt = 0; mt < KS; ++mt) o[mt][nt][e] *= f;
                                }
                            vref = now;
                        }
#pragma unroll
                        for (int b = 0; b < bpc; ++b) vs_[b] *= vref;
                        constexpr int kBlockShift = bs_shift - 3;   // groups of 8 keys per block
                        // ---- base-2 logits, relative to the running maxima
                        float x[kTiles][NT][2][NJ];   // [key half][head]
#pragma unroll
                        for (int mt = 0; mt < kTiles; ++mt)
#pragma unroll
                            for (int r = 0; r < 2; ++r)
#pragma unroll
                                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                                    for (int j = 0; j < NJ; ++j)
                                        x[mt][nt][r][j] = fmaf(ks_[(2 * mt + r) >> kBlockShift],
                                                               st[mt][nt][2 * r + j], bias[nt][j]);
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
                                    for (int e = j; e < 4; e += kOne ? 1 : 2) {
                                        mid[nt][e] *= a;
#pragma unroll
                                        for (int mt = 0; mt < KS; ++mt) o[mt][nt][e] *= a;
                                    }
                                }
                        }
                        fresh = false;
                        // ---- P, and O^T += V^T P^T
#pragma unroll
                        for (int mt = 0; mt < kTiles; ++mt) {
                            uint32_t pb[NT][2], pl[NT][2];   // the two parts of P times V's scale
#pragma unroll
                            for (int r = 0; r < 2; ++r) {
                                const float f = vs_[(2 * mt + r) >> kBlockShift];
#pragma unroll
                                for (int nt = 0; nt < NT; ++nt) {
                                    float e[2] = {0.f, 0.f};
#pragma unroll
                                    for (int j = 0; j < NJ; ++j) {
                                        e[j] = pa::fast_exp2(x[mt][nt][r][j]);
                                        l_run[nt][j] += e[j];
                                    }
                                    const float y0 = e[0] * f, y1 = e[1] * f;
                                    const float h0 = upper_half(y0), h1 = upper_half(y1);
                                    if constexpr (kOne) {
                                        pb[nt][r] = pa::movmatrix_trans(pa::pack2<true>(h0, y0 - h0));
                                    } else if constexpr (kDup) {
                                        pb[nt][r] = pa::movmatrix_trans(
                                            pa::pack2<true>(fmaf(dup, y0, -h0), fmaf(dup, y1, -h1)));
                                    } else {
                                        pb[nt][r] = pa::movmatrix_trans(__byte_perm(
                                            __float_as_uint(y0), __float_as_uint(y1), 0x7632));
                                        pl[nt][r] = pa::movmatrix_trans(pa::pack2<true>(y0 - h0, y1 - h1));
                                    }
                                }
                            }
                            // This lane's channels of the keys 16 mt + 8 r + 2 c4 + {0, 1}, the two
                            // keys' words in turn: z[r][w][y] has bytes 2 y, 2 y + 1 of the first
                            // key's word w in its lower half, the second key's in its upper one.
                            uint32_t z[2][NW][2];
#pragma unroll
                            for (int r = 0; r < 2; ++r) {
                                uint32_t w[2][NW];
#pragma unroll
                                for (int i = 0; i < 2; ++i) {
                                    const uint32_t at = stage + voff[i] + (16 * mt + 8 * r) * D;
                                    if constexpr (D == 128) {
                                        const uint4 y = pa::lds128(at);
                                        w[i][0] = y.x, w[i][1] = y.y, w[i][NW - 2] = y.z, w[i][NW - 1] = y.w;
                                    } else {
                                        const uint2 y = pa::lds64(at);
                                        w[i][0] = y.x, w[i][1] = y.y;
                                    }
                                }
#pragma unroll
                                for (int x2 = 0; x2 < NW; ++x2) {
                                    z[r][x2][0] = __byte_perm(w[0][x2], w[1][x2], 0x5410);
                                    z[r][x2][1] = __byte_perm(w[0][x2], w[1][x2], 0x7632);
                                }
                            }
                            // One product behind, the second parts: no two in a row into one
                            // accumulator.
                            constexpr bool kTwo = !kOne && !kDup;
                            uint32_t a[4] = {}, was[4];
#pragma unroll
                            for (int y = 0; y < KS; ++y) {
                                const int w = y >> 2, u = y & 3;
#pragma unroll
                                for (int i = 0; i < 4; ++i) {
                                    was[i] = a[i];
                                    // rows cr, cr + 8 (words w, w + NW / 2) of keys r = 0, then of r = 1
                                    a[i] = v_pair<kInt8>(z[i >> 1][w + (i & 1) * (NW / 2)][u >> 1], u & 1);
                                }
#pragma unroll
                                for (int nt = 0; nt < NT; ++nt) {
                                    pa::mma_16816<true>(o[y][nt], a, pb[nt][0], pb[nt][1]);
                                    if (kInt8 && y == 0) pa::mma_16816<true>(mid[nt], all128, pb[nt][0], pb[nt][1]);
                                }
                                if constexpr (kTwo)
#pragma unroll
                                    for (int nt = 0; nt < NT; ++nt) {
                                        if (y > 0) pa::mma_16816<true>(o[y - 1][nt], was, pl[nt][0], pl[nt][1]);
                                        if (kInt8 && y == KS - 1)
                                            pa::mma_16816<true>(mid[nt], all128, pl[nt][0], pl[nt][1]);
                                        if (y == KS - 1) pa::mma_16816<true>(o[y][nt], a, pl[nt][0], pl[nt][1]);
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
                if constexpr (kInt8)
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
#pragma unroll
                            for (int mt = 0; mt < KS; ++mt) o[mt][nt][e] -= mid[nt][e];
                            mid[nt][e] = 0.f;
                        }
            }
            pos += c_end - c0 + (c_end == s.nc ? kPairCost : 0);

            // ---- the pair's chunks of this warp are done
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int j = 0; j < NJ; ++j)
#pragma unroll
                    for (int off = 4; off < 32; off <<= 1)
                        l_run[nt][j] += __shfl_xor_sync(0xffffffffu, l_run[nt][j], off);
            const bool whole = c0 == 0 && c_end == s.nc;
            // The warp's first run may end while its ring is in use: a slot of its own.
            // A later unfinished run is its last: the ring is free.
            const uint32_t at = segn == 0 ? L.slots + (uint32_t)warp * slot_floats(G, D) * 4
                                          : (uint32_t)warp * S * kStage;
            float* slot = reinterpret_cast<float*>(smem + at);
            // The sums' unit: codes 2^-133 or 2^-120 times theirs, V scales vref times theirs.
            const float unit = vref > 0.f ? kVUnit<kInt8> / vref : 0.f;
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
                    float v[D / 8];
#pragma unroll
                    for (int u = 0; u < D / 8; ++u) {
                        const int e = u < KS ? j : 2 + j;
                        // both parts of P
                        float sum = kOne ? o[u % KS][nt][e] + o[u % KS][nt][e + 1] : o[u % KS][nt][e];
                        sum *= 1.2676506002282294e30f;   // 2^100
                        if constexpr (kDup) {
                            const float part = c4 < 2 ? -sum : sum;
                            sum = part + __shfl_xor_sync(0xffffffffu, part, 2);
                        }
                        v[u] = sum * unit * inv;
                    }
                    if (kDup && (h >= G || c4 >= 2)) continue;
                    if (whole) {
                        uint4* to = reinterpret_cast<uint4*>(
                            p.out.out + ((int64_t)s.i * p.out.H + s.g * G + h) * D + D / 8 * cr);
#pragma unroll
                        for (int u = 0; u < D / 8; u += 8)
                            to[u / 8] = make_uint4(pa::pack2<kBF16>(v[u], v[u + 1]), pa::pack2<kBF16>(v[u + 2], v[u + 3]),
                                                   pa::pack2<kBF16>(v[u + 4], v[u + 5]), pa::pack2<kBF16>(v[u + 6], v[u + 7]));
                    } else {
                        float4* to = reinterpret_cast<float4*>(slot + slot_head(G) + h * D + D / 8 * cr);
#pragma unroll
                        for (int u = 0; u < D / 8; u += 4) to[u / 4] = make_float4(v[u], v[u + 1], v[u + 2], v[u + 3]);
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
    __syncthreads();
    join_runs<D, kBF16>(p.out, cut, cta_lo, nw, smem, S * kStage, L.slots, runs, is_last, scan);
}

// ---- host side -----------------------------------------------------------------

// As many warps as shared memory holds rings and slots for; 0: not even four.
int choose_warps(int D, int G, int B) {
    for (int w = max_warps(D, form_of(G)); w >= 4; --w)
        if (make_layout(w * ring_stages(D) * stage_bytes(D), D, G, B, w).total <= kSmemBudget) return w;
    return 0;
}

template <int D, bool kBF16, bool kInt8, int kForm, int kShift>
pa_status launch(const Block8Params& p, cudaStream_t stream) {
    auto kern = decode_block8_kernel<D, kBF16, kInt8, kForm, kShift>;
    static pa::DeviceOnce once;
    if (!pa::allow_smem(once, kern, kSmemBudget)) return PA_ERR_CUDA;
    int ctas = pa::device_sm_count();
    if (ctas <= 0) return PA_ERR_CUDA;
    if (ctas > kMaxCtas) ctas = kMaxCtas;
    // Started early, so that its launch hides behind the append's or another call's end.
    cudaLaunchAttribute attr{};
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)ctas);
    cfg.blockDim = dim3((unsigned)p.warps * 32);
    cfg.dynamicSmemBytes = make_layout(p.warps * ring_stages(D) * stage_bytes(D), D, p.out.G, p.B, p.warps).total;
    cfg.stream = stream;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    return pa::cuda_status(cudaLaunchKernelEx(&cfg, kern, p));
}

template <int D, bool kBF16, bool kInt8, int kForm>
pa_status launch_b(const Block8Params& p, int32_t block_size, cudaStream_t stream) {
    if (block_size == 8) return launch<D, kBF16, kInt8, kForm, 3>(p, stream);
    if (block_size == 16) return launch<D, kBF16, kInt8, kForm, 4>(p, stream);
    return launch<D, kBF16, kInt8, kForm, 5>(p, stream);
}

template <int D, bool kBF16, bool kInt8>
pa_status launch_g(const Block8Params& p, int32_t block_size, cudaStream_t stream) {
    switch (form_of(p.out.G)) {
        case kG1: return launch_b<D, kBF16, kInt8, kG1>(p, block_size, stream);
        case kG4: return launch_b<D, kBF16, kInt8, kG4>(p, block_size, stream);
        case kG8: return launch_b<D, kBF16, kInt8, kG8>(p, block_size, stream);
        default: return launch_b<D, kBF16, kInt8, kG16>(p, block_size, stream);
    }
}

template <bool kInt8>
pa_status decode(const void* q, const void* k_cache, const void* v_cache, const float* k_scale,
                 const float* v_scale, const int32_t* block_tables, int32_t max_blocks,
                 const int32_t* context_lens, int32_t max_context_len, int32_t B, int32_t H,
                 int32_t Hkv, int32_t d, int32_t block_size, int32_t num_blocks, float scale,
                 pa_dtype dtype, void* out, void* workspace, size_t ws_bytes, void* stream) {
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
    if ((int64_t)num_blocks * Hkv > INT32_MAX || B > kMaxBatch ||
        (int64_t)num_blocks * block_size > INT32_MAX || (int64_t)max_blocks * block_size > INT32_MAX)
        return PA_ERR_UNSUPPORTED;
    // A block's codes over all KV heads are counted in 32 bits.
    if ((int64_t)Hkv * d * block_size > UINT32_MAX) return PA_ERR_UNSUPPORTED;
    // Positions in the list are int32.
    const int64_t max_chunks = ((int64_t)max_blocks * block_size + kChunk - 1) / kChunk;
    if ((int64_t)B * Hkv * subs * (max_chunks + kPairCost) >= ((int64_t)1 << 30)) return PA_ERR_UNSUPPORTED;
    if (B > 0 && ws_bytes < pa_decode_workspace_size(B, H, d)) return PA_ERR_INVALID;
    if (B == 0) return PA_OK;
    if (!q || !k_cache || !v_cache || !k_scale || !v_scale || !block_tables || !context_lens ||
        !out || !workspace)
        return PA_ERR_INVALID;
    if ((reinterpret_cast<uintptr_t>(k_cache) | reinterpret_cast<uintptr_t>(v_cache) |
         reinterpret_cast<uintptr_t>(q) | reinterpret_cast<uintptr_t>(out) |
         reinterpret_cast<uintptr_t>(workspace)) & 15u)
        return PA_ERR_INVALID;
    if ((reinterpret_cast<uintptr_t>(k_scale) | reinterpret_cast<uintptr_t>(v_scale)) & 3u)
        return PA_ERR_INVALID;
    Block8Params p;
    p.warps = choose_warps(d, G, B);
    if (!p.warps) return PA_ERR_UNSUPPORTED;
    p.err = pa::device_error_word();
    if (!p.err) return PA_ERR_CUDA;
    p.q = static_cast<const uint16_t*>(q);
    p.k_cache = static_cast<const uint8_t*>(k_cache);
    p.v_cache = static_cast<const uint8_t*>(v_cache);
    p.k_scale = k_scale;
    p.v_scale = v_scale;
    p.block_tables = block_tables;
    p.context_lens = context_lens;
    p.out.out = static_cast<uint16_t*>(out);
    p.out.counters = static_cast<int32_t*>(workspace);
    p.out.partials = reinterpret_cast<float*>(static_cast<unsigned char*>(workspace) + ticket_bytes(B, H));
    p.out.H = H;
    p.out.Hkv = Hkv * subs;
    p.out.G = G;
    p.max_blocks = max_blocks;
    p.B = B;
    p.num_blocks = num_blocks;
    p.subs = subs;
    p.scale_log2 = scale * kLog2e;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (d == 128)
        return dtype == PA_BF16 ? launch_g<128, true, kInt8>(p, block_size, st)
                                : launch_g<128, false, kInt8>(p, block_size, st);
    return dtype == PA_BF16 ? launch_g<64, true, kInt8>(p, block_size, st)
                            : launch_g<64, false, kInt8>(p, block_size, st);
}

}  // namespace
