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

namespace {

constexpr int kChunk = 32;              // tokens per stage
constexpr int kTiles = kChunk / 16;     // 16-key MMA tiles per chunk
constexpr int kMaxG = 16;
constexpr int kMaxBatch = 4096;
constexpr int kMaxCtas = 512;
// Stages of a warp's ring: it computes on one while the others fill.
__host__ __device__ constexpr int ring_stages(int D) { return D == 128 ? 2 : 4; }
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

// One partial result in shared memory: row maxima [G], row sums [G], padding to 16 bytes,
// outputs [G][D]; in the workspace: maxima and sums [kMaxG] each.
__host__ __device__ constexpr int slot_head(int G) { return (2 * G + 3) & ~3; }
__host__ __device__ constexpr int slot_floats(int G, int D) { return slot_head(G) + G * D; }
__host__ __device__ constexpr int partial_floats(int D) { return 2 * kMaxG + kMaxG * D; }

// A run of chunks [c0, end) of one pair that a warp left in shared memory.
struct Run {
    int32_t a;    // position of the pair in the list; -1: none
    int32_t i, g, c0, end, nc;
    uint32_t at;  // at the end, entry x: the set of runs of the CTA's x-th pair,
    int32_t pad;  // and the first of them (+ 256: other CTAs hold more)
};

struct Layout {
    uint32_t stage, rows, slots, runs, last, scan, prefix, total;
};

__host__ __device__ inline Layout make_layout(int D, int G, int B, int warps) {
    const int stages = ring_stages(D);
    Layout L;
    L.stage = 2u * kChunk * (D / 2 + D / 64 * 4);            // K, V codes, K, V scales
    L.rows = warps * stages * L.stage;                      // per warp: K and V of 32 rows
    L.slots = L.rows + warps * 2 * kChunk * (D / 64) * 8;   // a slot per warp
    L.runs = L.slots + warps * slot_floats(G, D) * 4;       // [2 * warps]
    L.last = L.runs + 2 * warps * (uint32_t)sizeof(Run);     // "the last CTA of the pair"
    L.scan = L.last + 8;
    L.prefix = L.scan + warps * 8;                          // [B + 1]
    L.total = L.prefix + (uint32_t)(B + 1) * 4;
    return L;
}

__device__ __forceinline__ int32_t clamp_len(int32_t n, int32_t cap) {
    return n < 0 ? 0 : (n > cap ? cap : n);
}

// W units cut into n parts, the first W % n of them one unit longer.
struct Cut {
    int32_t q, r;
    __device__ Cut(int32_t W, int32_t n) : q(W / n), r(W - W / n * n) {}
    __device__ int32_t begin(int32_t x) const { return x * q + min(x, r); }
    // the part that holds position c
    __device__ int32_t part(int32_t c) const {
        const int32_t big = r * (q + 1);
        return c < big ? c / (q + 1) : r + (c - big) / q;
    }
};

// The list of pairs is cut by cost, in units of a chunk: kPairCost of them for the pair itself
// (its q, its table's first entries, its end), then its nc chunks, from position a on.  Cut
// by chunks alone, CTAs with many short pairs ended 10 us after those with few: 64 sequences
// of 128 .. 2048 tokens, 40 heads, took 75.5 us against 72.3 with 2 (71.5 with 1, 73.9 with
// 3), 32 long-tailed contexts 26.5 us against 24.6 (25.4, 24.4).
constexpr int kPairCost = 2;

// A position in the list: chunk c of pair (i, g).
struct Cursor {
    int32_t i, g, c, nc, a;
};

__device__ __forceinline__ Cursor find(const int32_t* prefix, int32_t B, int32_t Hkv, int32_t pos) {
    int32_t lo = 0, hi = B;   // largest i with prefix[i] <= pos
#pragma unroll 1
    while (hi - lo > 1) {
        const int32_t mid = (lo + hi) >> 1;
        if (prefix[mid] <= pos) lo = mid; else hi = mid;
    }
    Cursor s;
    s.i = lo;
    const int32_t cost = (prefix[lo + 1] - prefix[lo]) / Hkv, local = pos - prefix[lo];
    s.nc = cost - kPairCost;
    s.g = local / cost;
    s.a = prefix[lo] + s.g * cost;
    s.c = max(0, pos - s.a - kPairCost);
    return s;
}

// The pair after s (there is one).
__device__ __forceinline__ Cursor next_pair(const int32_t* prefix, int32_t Hkv, Cursor s) {
    s.a += kPairCost + s.nc;
    s.c = 0;
    if (++s.g == Hkv) {
        s.g = 0;
        do ++s.i; while (prefix[s.i + 1] == prefix[s.i]);
        s.nc = (prefix[s.i + 1] - prefix[s.i]) / Hkv - kPairCost;
    }
    return s;
}

// 16 bytes global -> shared, asynchronously; zeros and no read unless ok.
__device__ __forceinline__ void copy16(uint32_t to, const void* from, bool ok, uint64_t policy) {
    asm volatile("cp.async.cg.shared.global.L2::cache_hint [%0], [%1], 16, %2, %3;" ::"r"(to), "l"(from),
                 "r"(ok ? 16 : 0), "l"(policy) : "memory");
}
__device__ __forceinline__ void commit_group() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void wait_group() {   // until at most N of this thread's groups are in flight
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

__device__ __forceinline__ void prefetch_l2(const void* p) {
    asm volatile("prefetch.global.L2 [%0];" ::"l"(p));
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
    const Layout L = make_layout(D, G, B, nw);
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

    // ---- prefix[i] = Hkv * (chunks and kPairCost) of the sequences before i that hold any
    {
        const int per = (B + threads - 1) / threads;
        const int beg = min(tid * per, B), end = min(beg + per, B);
        int32_t local = 0, held = 0;   // cost; sequences that are not empty
#pragma unroll 1
        for (int i = beg; i < end; ++i) {
            const int32_t raw = pa::ld_behind_wait(p.context_lens + i);
            if (blockIdx.x == 0) {
                if (raw < 0) pa::raise_error(p.err, PA_DEVERR_CONTEXT);
                if (raw > max_len) pa::raise_error(p.err, PA_DEVERR_TABLE_WIDTH);
            }
            const int32_t chunks = (clamp_len(raw, max_len) + kChunk - 1) / kChunk;
            local += chunks ? chunks + kPairCost : 0;
            held += chunks > 0;
        }
        held = __reduce_add_sync(0xffffffffu, held);
        int32_t x = local;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int32_t y = __shfl_up_sync(0xffffffffu, x, o);
            if (lane >= o) x += y;
        }
        if (lane == 31) {
            scan[warp] = x;
            scan[nw + warp] = held;
        }
        if (tid < 2 * nw) runs[tid].a = -1;
        __syncthreads();
        int32_t run = x - local;
#pragma unroll 1
        for (int w = 0; w < warp; ++w) run += scan[w];
#pragma unroll 1
        for (int i = beg; i < end; ++i) {
            prefix[i] = run * Hkv;
            const int32_t chunks = (clamp_len(pa::ld_behind_wait(p.context_lens + i), max_len) + kChunk - 1) / kChunk;
            run += chunks ? chunks + kPairCost : 0;
        }
        if (tid == 0) {
            int32_t total = 0, all = 0;
#pragma unroll 1
            for (int w = 0; w < nw; ++w) {
                total += scan[w];
                all += scan[nw + w];
            }
            prefix[B] = total * Hkv;
            is_last[0] = (total - kPairCost * all) * Hkv;   // chunks
        }
        __syncthreads();
    }

    // ---- zero rows of empty contexts
#pragma unroll 1
    for (int32_t i = blockIdx.x; i < B; i += gridDim.x) {
        if (prefix[i + 1] != prefix[i]) continue;
        uint4* row = reinterpret_cast<uint4*>(p.out + (int64_t)i * p.H * D);
#pragma unroll 1
        for (int v = tid; v < p.H * D / 8; v += threads) row[v] = make_uint4(0, 0, 0, 0);
    }

    const int32_t W = is_last[0];
    // CTAs in use have a chunk per warp at least: smaller batches take fewer CTAs
    // rather than more partial results.
    const int32_t C = min((W + nw - 1) / nw, (int32_t)gridDim.x);
    if ((int32_t)blockIdx.x >= C) return;
    const Cut cut(prefix[B], C);
    const int32_t cta_lo = cut.begin(blockIdx.x), cta_hi = cut.begin(blockIdx.x + 1);
    const Cut mine(cta_hi - cta_lo, nw);
    const int32_t lo = cta_lo + mine.begin(warp), hi = cta_lo + mine.begin(warp + 1);

    const uint32_t ring = sbase + (uint32_t)warp * S * kStage;
    const uint32_t krows = sbase + L.rows + (uint32_t)warp * (2 * kChunk * NG * 8);
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

    // ====================== runs of one pair in several warps ======================
    // Runs lie in list order: a pair's runs are neighbours, warps without a second run
    // between them.  Lane k of every warp looks at run k (such gaps go with the pair
    // before them): whether it leads its pair, and whether the pair is whole or other CTAs
    // hold some of it (true of at most the CTA's first and last pair).
    const Run my = runs[lane < 2 * nw ? lane : 0];
    const bool valid_run = lane < 2 * nw && my.a >= 0;
    const uint32_t upto = 0xffffffffu >> (31 - lane);
    const uint32_t before = __ballot_sync(0xffffffffu, valid_run) & upto;
    const int32_t pair_of = __shfl_sync(0xffffffffu, my.a, before ? 31 - __clz(before) : 0);
    const int32_t seg = before ? pair_of : -1;
    const uint32_t same = __match_any_sync(0xffffffffu, seg);      // a contiguous set
    const int seg_last = 31 - __clz(same);
    const bool leads = valid_run && (same & upto) == (1u << lane);
    const uint32_t in_pair = same & __ballot_sync(0xffffffffu, valid_run);
    const int32_t pair_end = __shfl_sync(0xffffffffu, my.end, in_pair ? 31 - __clz(in_pair) : 0);
    const bool shared = my.c0 != 0 || pair_end != my.nc;
    const uint32_t lead = __ballot_sync(0xffffffffu, leads);
    const uint32_t open = __ballot_sync(0xffffffffu, leads && shared);
    // A warp's first run has its slot, a later one its ring.
    auto slot_at = [&](int k) {
        return reinterpret_cast<float*>(smem + (k & 1 ? (uint32_t)(k >> 1) * S * kStage
                                                      : L.slots + (uint32_t)(k >> 1) * slot_floats(G, D) * 4));
    };
    // A CTA's first partial holds the pair that its share begins in or with, its second
    // the one that begins later.
    auto partial_at = [&](int32_t a) {
        return p.partials + (2 * (int64_t)blockIdx.x + (cta_lo >= a ? 0 : 1)) * partial_floats(D);
    };
    // Head by head: maximum and sum over each pair's runs (a segmented scan over the
    // lanes), each run's factor 2^(m_k - M) in place of its maximum.
#pragma unroll 1
    for (int h = warp; h < G; h += nw) {
        float* slot = slot_at(lane < 2 * nw ? lane : 0);
        const float m = valid_run ? slot[h] : -INFINITY;
        float M = m;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const float y = __shfl_up_sync(0xffffffffu, M, o);
            if (lane >= o && (same >> (lane - o) & 1)) M = fmaxf(M, y);
        }
        M = __shfl_sync(0xffffffffu, M, seg_last);
        const float f = valid_run ? pa::fast_exp2(m - M) : 0.f;
        float l = valid_run ? f * slot[G + h] : 0.f;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const float y = __shfl_up_sync(0xffffffffu, l, o);
            if (lane >= o && (same >> (lane - o) & 1)) l += y;
        }
        l = __shfl_sync(0xffffffffu, l, seg_last);
        if (valid_run) slot[h] = f;
        if (leads && !shared) slot[G + h] = 1.f / l;
        if (leads && shared) {
            partial_at(my.a)[h] = M;
            partial_at(my.a)[kMaxG + h] = l;
        }
    }
    if (warp == 0 && leads) {   // the pairs in order, for the loop below
        const int at = __popc(lead & (upto >> 1));
        runs[at].pad = lane | (shared ? 256 : 0);
        runs[at].at = in_pair;
    }
    __syncthreads();
    auto store4 = [&](int32_t i, int32_t h, int d4, float4 v, float inv) {
        *reinterpret_cast<uint2*>(p.out + ((int64_t)i * p.H + h) * D + d4) =
            make_uint2(pa::pack2<kBF16>(v.x * inv, v.y * inv), pa::pack2<kBF16>(v.z * inv, v.w * inv));
    };
    const int outs = G * D / 4;     // four outputs each
#pragma unroll 1
    for (int x = tid; x < __popc(lead) * outs; x += threads) {
        const int at = x / outs, e = x - at * outs;
        const int k = runs[at].pad & 255;
        const int h = e / (D / 4), d4 = e % (D / 4) * 4;
        float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
        for (uint32_t set = runs[at].at; set; set &= set - 1) {
            const float* slot = slot_at(__ffs(set) - 1);
            const float f = slot[h];
            const float4 y = *reinterpret_cast<const float4*>(slot + slot_head(G) + h * D + d4);
            v.x += f * y.x;
            v.y += f * y.y;
            v.z += f * y.z;
            v.w += f * y.w;
        }
        if (runs[at].pad & 256)
            *reinterpret_cast<float4*>(partial_at(runs[k].a) + 2 * kMaxG + e * 4) = v;
        else
            store4(runs[k].i, runs[k].g * G + h, d4, v, slot_at(k)[G + h]);
    }
    if (!open) return;

    // ================= pairs shared with other CTAs, by the whole CTA =================
    // Publish: the barrier orders every thread's stores before the ticket's release; the
    // ticket names the pair's last CTA and, for it, acquires the other CTAs' partials.
    constexpr int kPartial = partial_floats(D);
    const int n_open = __popc(open);   // one or two
    auto open_lead = [&](int w) { return w ? 31 - __clz(open) : __ffs(open) - 1; };
    __syncthreads();
    if (warp < n_open && lane == 0) {
        const Run& r = runs[open_lead(warp)];
        int32_t* ticket = p.counters + (int64_t)r.i * Hkv + r.g;
        const int32_t before_me = pa::atomic_add_acq_rel_gpu(ticket, 1);
        const int32_t first = cut.part(r.a + kPairCost);
        const int32_t n = cut.part(r.a + kPairCost + r.nc - 1) - first + 1;
        const bool last = before_me == n - 1;
        if (last) atomicExch(ticket, 0);   // ready for the next launch
        is_last[warp] = last ? n : 0;      // the pair's CTAs
        scan[warp] = first;
    }
    __syncthreads();
    // Two pairs to join: half the threads each, so that their loads are under way together.
    const bool both = n_open == 2 && is_last[0] && is_last[1];
    const int team = both ? threads / 2 : threads, my_w = both && tid >= team ? 1 : 0;
    const int ltid = tid - my_w * team;
#pragma unroll 1
    for (int w0 = 0; w0 < (both ? 1 : n_open); ++w0) {
        const int w = both ? my_w : w0;
        if (!is_last[w]) continue;
        const Run r = runs[open_lead(w)];
        const int c_first = scan[w], n = is_last[w], most = both ? max(is_last[0], is_last[1]) : n;
        const float* first = p.partials + (2 * (int64_t)c_first + (cut.begin(c_first) >= r.a ? 0 : 1)) * kPartial;
        const float* rest = p.partials + 2 * (int64_t)c_first * kPartial;
        // A group of threads has the outputs, four each, and eight partials' loads in flight;
        // of more than eight the groups take turns, and join in shared memory.
        const int wide = min(outs, team), groups = most > 8 ? team / wide : 1;
        const int grp = ltid / wide;
        float4* acc_at = reinterpret_cast<float4*>(smem) + my_w * team;   // [groups][outs]
        float2* ml_at = reinterpret_cast<float2*>(reinterpret_cast<float4*>(smem) + threads) + my_w * team;
#pragma unroll 1
        for (int e = ltid - grp * wide; e < outs && grp < groups; e += wide) {
            const int h = e / (D / 4);
            float M = -INFINITY, l = 0.f;
            float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 1
            for (int c0 = grp; c0 < n; c0 += 8 * groups) {
                float pm[8], pl[8];
                float4 po[8];
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const int c = c0 + j * groups;
                    if (c < n) {
                        const float* q = c ? rest + 2 * (int64_t)c * kPartial : first;
                        pm[j] = __ldcg(q + h);
                        pl[j] = __ldcg(q + kMaxG + h);
                        po[j] = __ldcg(reinterpret_cast<const float4*>(q + 2 * kMaxG) + e);
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
            if (groups == 1) {
                store4(r.i, r.g * G + h, e % (D / 4) * 4, acc, 1.f / l);
            } else {
                acc_at[grp * outs + e] = acc;
                ml_at[grp * outs + e] = make_float2(M, l);
            }
        }
        if (groups > 1) {
            __syncthreads();
#pragma unroll 1
            for (int e = ltid; e < outs; e += team) {
                const int use = min(groups, n);
                float M = -INFINITY, l = 0.f;
                float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 1
                for (int q = 0; q < use; ++q) M = fmaxf(M, ml_at[q * outs + e].x);
#pragma unroll 1
                for (int q = 0; q < use; ++q) {
                    const float2 ml = ml_at[q * outs + e];
                    const float4 y = acc_at[q * outs + e];
                    const float f = pa::fast_exp2(ml.x - M);
                    l += f * ml.y;
                    acc.x += f * y.x;
                    acc.y += f * y.y;
                    acc.z += f * y.z;
                    acc.w += f * y.w;
                }
                store4(r.i, r.g * G + e / (D / 4), e % (D / 4) * 4, acc, 1.f / l);
            }
            __syncthreads();
        }
    }
}

// ---- host side -----------------------------------------------------------------

// As many warps as shared memory holds rings and slots for; 0: not even four.
int choose_warps(int D, int G, int B) {
    for (int w = max_warps(D, form_of(G)); w >= 4; --w)
        if (make_layout(D, G, B, w).total <= kSmemBudget) return w;
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
    const Layout L = make_layout(D, p.G, p.B, p.warps);
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
    if (d == 128)
        return dtype == PA_BF16 ? launch_g<128, true>(p, st) : launch_g<128, false>(p, st);
    return dtype == PA_BF16 ? launch_g<64, true>(p, st) : launch_g<64, false>(p, st);
}

}  // extern "C"
