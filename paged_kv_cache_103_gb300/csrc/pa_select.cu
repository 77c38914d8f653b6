// Block summaries (pa_summarize_blocks) and the selection of the blocks that a
// decode step attends over (pa_select_blocks); pa_decode_selected then reads
// only those.
//
// A context's keys are summarised per (block, KV head) by the smallest and the
// largest key value of each head-dim channel, lo_c and hi_c, as INT8 codes with
// one fp32 scale.  For a query q the block's largest possible score is at most
//     sum_c max(q_c lo_c, q_c hi_c) = sum_c q_c (q_c > 0 ? hi_c : lo_c),
// so a block where that is low holds no key that matters.  The query is coded
// in INT8 too, which makes the sum an integer: the score, and with it the
// selection, does not depend on the order of summation.  Codes are the nearest, so
// what is ranked is the bound to within half a step of both codes and not the
// bound itself: a key's score may pass it by
//     sum_c ((|q_c| S + max(|lo_c|, |hi_c|) sq) / 2 + sq S / 4).
//     sq = max |q_c| / 127,  c_c = rint(q_c / sq),  dot = sum_c c_c (..) ,
//     score = max over the group's query heads of (dot sq) S
// with every operation rounded to fp32 once.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cstring>

#include "pa.h"
#include "pa_common.cuh"

namespace {

constexpr int kThreads = 256;

template <bool kBF16>
__device__ __forceinline__ float2 widen2(uint32_t v) {
    if constexpr (kBF16) {
        return make_float2(__uint_as_float(v << 16), __uint_as_float(v & 0xFFFF0000u));
    } else {
        __half2 h;
        memcpy(&h, &v, 4);
        return __half22float2(h);
    }
}

__device__ __forceinline__ uint32_t code8(float x, float s) {
    return (uint32_t)max(-127, min(127, __float2int_rn(__fdiv_rn(x, s)))) & 0xFFu;
}

// One warp per (listed block, KV head): lane l owns channels 8 (l % (D / 8)) .. + 7 of every
// (32 / (D / 8))-th row, so a block's rows are in flight at once.  Bound by HBM: 2048
// blocks of 16 x 8 x 128 values (71.4 MB) take 15.0 us, 4.8 TB/s (16.0 us before a lane
// had four rows in flight).  Afterwards the first half of the warp has the smallest values
// to code, the second the largest.
template <bool kBF16, int D>
__global__ void __launch_bounds__(kThreads)
summarize_kernel(const uint4* __restrict__ k_cache, const int32_t* __restrict__ block_ids,
                 const int32_t* __restrict__ fills, uint32_t pairs, uint32_t Hkv, int32_t bs,
                 int32_t num_blocks, uint2* __restrict__ boxes, float* __restrict__ box_scale,
                 unsigned int* __restrict__ err) {
    constexpr uint32_t kRow = D / 8, kSets = 32 / kRow, kFlight = 4;
    const uint32_t pair = (blockIdx.x * kThreads + threadIdx.x) >> 5, lane = threadIdx.x & 31;
    if (pair >= pairs) return;
    const uint32_t e = pair / Hkv, h = pair - e * Hkv, l = lane % kRow, set = lane / kRow;
    const int32_t id = __ldg(block_ids + e);
    const bool ok = (uint32_t)id < (uint32_t)num_blocks;
    int32_t fill = fills ? __ldg(fills + e) : bs;
    if (lane == 0 && h == 0) {
        if (!ok) pa::raise_error(err, PA_DEVERR_BLOCK_ID);
        if (fill < 0 || fill > bs) pa::raise_error(err, PA_DEVERR_CONTEXT);
    }
    if (!ok) return;
    fill = max(0, min(bs, fill));
    uint32_t lo[4] = {0, 0, 0, 0}, hi[4] = {0, 0, 0, 0};
    if (fill > 0) {
        const int64_t stride = (int64_t)Hkv * kRow;   // between token rows
        const uint4* src = k_cache + (int64_t)id * bs * stride + h * kRow + l;
        for (int32_t r0 = 0; r0 < fill; r0 += kFlight * kSets) {
            uint4 x[kFlight];
#pragma unroll
            for (int r = 0; r < (int)kFlight; ++r)   // the last row again past the fill
                x[r] = __ldg(src + min(r0 + r * (int)kSets + (int)set, fill - 1) * stride);
#pragma unroll
            for (int r = 0; r < (int)kFlight; ++r) {
                const uint32_t w[4] = {x[r].x, x[r].y, x[r].z, x[r].w};
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const bool start = r0 == 0 && r == 0;
                    lo[j] = start ? w[j] : pa::min_x2<kBF16>(lo[j], w[j]);
                    hi[j] = start ? w[j] : pa::max_x2<kBF16>(hi[j], w[j]);
                }
            }
        }
    }
#pragma unroll
    for (uint32_t o = kRow; o < 32; o <<= 1)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            lo[j] = pa::min_x2<kBF16>(lo[j], __shfl_xor_sync(0xffffffffu, lo[j], o));
            hi[j] = pa::max_x2<kBF16>(hi[j], __shfl_xor_sync(0xffffffffu, hi[j], o));
        }
    const bool upper = lane >= 16;       // codes the largest
    float x[8], a = 0.f;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const float2 f = widen2<kBF16>(upper ? hi[j] : lo[j]);
        x[2 * j] = f.x;
        x[2 * j + 1] = f.y;
        a = fmaxf(a, fmaxf(fabsf(f.x), fabsf(f.y)));
    }
    // the bit patterns of non-negative floats order like the values
    a = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(a)));
    const float s = __fdiv_rn(a, 127.f);
    uint32_t c[2] = {0, 0};
    if (s > 0.f)
#pragma unroll
        for (int j = 0; j < 8; ++j) c[j >> 2] |= code8(x[j], s) << (8 * (j & 3));
    const int64_t row = (int64_t)id * Hkv + h;
    if (lane % 16 < kRow) boxes[(row * 2 + (upper ? 1 : 0)) * kRow + l] = make_uint2(c[0], c[1]);
    if (lane == 0) box_scale[row] = s;
}

struct SelectParams {
    const uint16_t* q;
    const uint4* boxes;
    const float* box_scale;
    const int32_t* block_tables;
    const int32_t* context_lens;
    int32_t* sel_blocks;
    int32_t* sel_lens;
    uint32_t* keys;      // [B * Hkv][max_blocks]: the scores, as ordered numbers
    unsigned int* err;
    int32_t max_blocks, H, Hkv, G, bs, num_blocks, keep, first, last;
    int32_t tile, heads;   // of a scoring CTA: blocks and KV heads, at most
    int32_t unit;          // blocks of a scoring CTA's whole step
};

// A float as an unsigned number of the same order (-0 as +0).
__device__ __forceinline__ uint32_t ordered(float x) {
    const uint32_t u = __float_as_uint(x + 0.f);
    return (u >> 31) ? ~u : (u | 0x80000000u);
}

__device__ __forceinline__ int32_t context_of(const SelectParams& p, int32_t i) {
    const int32_t n = __ldg(p.context_lens + i);
    return max(0, min(n, p.max_blocks * p.bs));
}

// 0xFF in the bytes that are negative.
__device__ __forceinline__ uint32_t sign_bytes(uint32_t x) {
    uint32_t r;
    asm("prmt.b32 %0, %1, 0, 0xBA98;" : "=r"(r) : "r"(x));
    return r;
}

// Scores of a share of one sequence's blocks under up to `heads` KV heads: blockIdx = (share,
// sequence, group of KV heads).  The shares are cut from the table, whose width the host
// knows, for a context that has a quarter of it or more (its ids are read before its length is
// known: 21.1 us instead of 21.5 for the step of 8 ragged contexts), and else from the context:
// 8 contexts of 512 blocks in tables of 8192 take 12.6 us, where shares of the table, most of
// them empty, took 31.4 (tables of 512: 7.4).  What bounds it is HBM: the boxes, 260 bytes a (block,
// KV head) at d = 128.  A box belongs to D / 16 lanes, 16 channels of lo and of hi each,
// and neighbouring lane groups take neighbouring KV heads, whose boxes are contiguous; a
// group works on four boxes at once while the next ones arrive in shared memory, each lane's
// bytes by its own asynchronous copies and for its own reading, so nothing is waited for but
// the lane's own copies.  A group keeps its KV head, so a query head's codes are read from
// shared memory once for the four.  16 contexts of 2048 blocks, 8 KV heads, G = 4 (68 MB)
// take some 14 us, 4.9 TB/s, and the selection behind them 6: 20.1 us together, 26.6
// while the boxes were loaded straight into registers.
constexpr int kMaxTile = 2048;
constexpr int kItems = 4, kRing = 3;                       // boxes per step; steps in the ring
constexpr uint32_t kStepBytes = kThreads * (kItems * 32 + 4);   // lo and hi; one scale a lane
constexpr int kCodeBytes = 32 * 1024;                      // of query codes and steps, at most
constexpr int kScoreSmem = kRing * kStepBytes + kCodeBytes + kMaxTile * 4;

__device__ __forceinline__ void copy16(uint32_t to, const void* from) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to), "l"(from) : "memory");
}
__device__ __forceinline__ void copy4(uint32_t to, const void* from) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(to), "l"(from) : "memory");
}

template <bool kBF16, int D>
__global__ void __launch_bounds__(kThreads, 2) score_kernel(const SelectParams p) {
    constexpr int kLanes = D / 16, kUnits = kThreads / kLanes;
    extern __shared__ __align__(16) uint32_t smem[];
    asm volatile("griddepcontrol.launch_dependents;");   // the selection may be launched: it waits
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int32_t i = blockIdx.y, g0 = blockIdx.z * p.heads, heads = min(p.heads, p.Hkv - g0);
    // Shared memory: the ring, the query codes [heads * G][D / 4] and their steps, the share's
    // block ids (-1: not the pool's).  Before the context's length is known, query heads are
    // read up to one a warp and ids as though the context filled its table: three reads under
    // way at once.
    const int nq = heads * p.G;
    uint32_t* codes = smem + kRing * kStepBytes / 4;
    float* sq = reinterpret_cast<float*>(codes + nq * (D / 4));
    int32_t* ids = reinterpret_cast<int32_t*>(sq + nq);
    const int32_t* table = p.block_tables + (int64_t)i * p.max_blocks;
    const int32_t guess = p.first + blockIdx.x * p.tile, room = p.max_blocks - p.last - guess;
    const int32_t id0 = tid < min(p.tile, room) ? __ldg(table + guess + tid) : 0;
    uint32_t qw[D / 64];
    auto load_q = [&](int h) {
#pragma unroll
        for (int j = 0; j < D / 64; ++j)
            qw[j] = __ldg(reinterpret_cast<const uint32_t*>(
                p.q + ((int64_t)i * p.H + g0 * p.G + h) * D + j * 64 + lane * 2));
    };
    load_q(min(warp, nq - 1));
    const int32_t nb = (context_of(p, i) + p.bs - 1) / p.bs;
    const int32_t m = nb - p.first - p.last, parts = gridDim.x;
    const int32_t share = m >= (p.max_blocks - p.first - p.last) / 4
                              ? p.tile : ((m + parts - 1) / parts + p.unit - 1) / p.unit * p.unit;   // <= tile
    const int32_t j0 = p.first + blockIdx.x * share, j1 = min(nb - p.last, j0 + share);
    if (nb <= p.keep || j0 >= j1) return;
    table += j0;
    for (int32_t t = tid; t < j1 - j0; t += kThreads) {
        int32_t id = t == tid && j0 == guess ? id0 : __ldg(table + t);
        if ((uint32_t)id >= (uint32_t)p.num_blocks) {
            if (g0 == 0) pa::raise_error(p.err, PA_DEVERR_BLOCK_ID);
            id = -1;
        }
        ids[t] = id;
    }
    __syncthreads();
    const int unit = tid / kLanes, l = tid % kLanes, rows = kUnits / heads;
    // KV head, and which of the blocks in flight (none for the lane groups left over, which
    // go along for the shuffles' sake)
    const int g = unit % heads, r = unit / heads < rows ? unit / heads : 1 << 28;
    const uint4* qc = reinterpret_cast<const uint4*>(codes) + g * p.G * kLanes + l;
    uint32_t* keys = p.keys + ((int64_t)i * p.Hkv + g0 + g) * p.max_blocks + j0;
    const int32_t count = j1 - j0, stride = kItems * rows, steps = (count + stride - 1) / stride;
    // the box of four that this lane finishes, after the sums below
    const int mine = kLanes == 8 ? (l >> 1) & 3 : l & 3;
    const uint32_t ring = pa::smem_addr(smem);
    auto load = [&](int32_t step) {   // a group per step, empty or not
        if (step < steps) {
            const uint32_t to = ring + step % kRing * kStepBytes + tid * 16;
#pragma unroll
            for (int q = 0; q < kItems; ++q) {
                const int32_t t = r + step * stride + q * rows, id = t < count ? max(ids[t], 0) : 0;
                const int64_t row = (int64_t)id * p.Hkv + g0 + g;
                copy16(to + (2 * q) * kThreads * 16, p.boxes + row * 2 * kLanes + l);
                copy16(to + (2 * q + 1) * kThreads * 16, p.boxes + row * 2 * kLanes + kLanes + l);
                if (q == mine) copy4(to - tid * 12 + kItems * 32 * kThreads, p.box_scale + row);
            }
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
    for (int step = 0; step < kRing - 1; ++step) load(step);
    // ---- the query's codes, while the first boxes are under way
    for (int h = warp; h < nq; h += kThreads / 32) {
        if (h != warp) load_q(h);
        float2 x[D / 64];
        float a = 0.f;
#pragma unroll
        for (int j = 0; j < D / 64; ++j) {
            x[j] = widen2<kBF16>(qw[j]);
            a = fmaxf(a, fmaxf(fabsf(x[j].x), fabsf(x[j].y)));
        }
        // the bit patterns of non-negative floats order like the values
        a = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(a)));
        const float s = __fdiv_rn(a, 127.f);
#pragma unroll
        for (int j = 0; j < D / 64; ++j)
            reinterpret_cast<uint16_t*>(codes)[h * (D / 2) + j * 32 + lane] =
                s > 0.f ? (uint16_t)(code8(x[j].x, s) | code8(x[j].y, s) << 8) : 0;
        if (lane == 0) sq[h] = s;
    }
    __syncthreads();
    for (int32_t step = 0; step < steps; ++step) {
        load(step + kRing - 1);
        asm volatile("cp.async.wait_group %0;" ::"n"(kRing - 1) : "memory");
        const int32_t t = r + step * stride;
        const unsigned char* at = reinterpret_cast<const unsigned char*>(smem) + step % kRing * kStepBytes;
        uint32_t lw[kItems][4], hw[kItems][4];
#pragma unroll
        for (int q = 0; q < kItems; ++q) {
            const uint4 lo = reinterpret_cast<const uint4*>(at)[(2 * q) * kThreads + tid];
            const uint4 hi = reinterpret_cast<const uint4*>(at)[(2 * q + 1) * kThreads + tid];
            lw[q][0] = lo.x, lw[q][1] = lo.y, lw[q][2] = lo.z, lw[q][3] = lo.w;
            hw[q][0] = hi.x, hw[q][1] = hi.y, hw[q][2] = hi.z, hw[q][3] = hi.w;
        }
        const float S = reinterpret_cast<const float*>(at + kItems * 32 * kThreads)[tid];
        float best = 0.f;
#pragma unroll 4
        for (int h = 0; h < p.G; ++h) {
            const uint4 cv = qc[h * kLanes];
            const uint32_t c[4] = {cv.x, cv.y, cv.z, cv.w};
            uint32_t neg[4];
#pragma unroll
            for (int w = 0; w < 4; ++w) neg[w] = sign_bytes(c[w]);
            int dot[kItems] = {};
#pragma unroll
            for (int q = 0; q < kItems; ++q)
#pragma unroll
                for (int w = 0; w < 4; ++w)
                    dot[q] = __dp4a((int)((lw[q][w] & neg[w]) | (hw[q][w] & ~neg[w])), (int)c[w], dot[q]);
            // Sums over the lanes, halving the boxes of each lane on the way.
            constexpr int kTop = kLanes / 2;
            const bool up = l & kTop, up2 = l & (kTop / 2);
            const int d0 = (up ? dot[2] : dot[0]) + __shfl_xor_sync(0xffffffffu, up ? dot[0] : dot[2], kTop);
            const int d1 = (up ? dot[3] : dot[1]) + __shfl_xor_sync(0xffffffffu, up ? dot[1] : dot[3], kTop);
            int sum = (up2 ? d1 : d0) + __shfl_xor_sync(0xffffffffu, up2 ? d0 : d1, kTop / 2);
            if constexpr (kLanes == 8) sum += __shfl_xor_sync(0xffffffffu, sum, 1);
            // S >= 0 and rounding is monotonic: the largest (dot sq) S is the largest dot sq's
            const float x = __fmul_rn((float)sum, sq[g * p.G + h]);
            best = h ? fmaxf(best, x) : x;
        }
        const int32_t tm = t + mine * rows;
        if (tm < count && (kLanes == 4 || !(l & 1)))
            keys[tm] = ids[tm] >= 0 ? ordered(__fmul_rn(best, S)) : 0u;
    }
}

constexpr int kSelThreads = 256;
constexpr int kSelWarps = kSelThreads / 32;
constexpr int kBinBits = 10, kBins = 1 << kBinBits;   // four bins a thread

// One CTA per (sequence, KV head): the k-th largest score, then the chosen ids in context
// order.  Bound by latency (a handful of barriers): some 6 us for 2048 blocks.  The keys'
// range is cut into 1024 bins, whose counts from the top name the bin of the k-th largest;
// that bin is cut again until it is one key wide or wanted whole (four passes at most, one
// or two in practice).  Each thread owns a contiguous stretch of the context's keys: up to kPer
// of them in registers, or (0) any number, read again from L2 by each pass.
template <int kPer>
__global__ void __launch_bounds__(kSelThreads) select_kernel(const SelectParams p) {
    __shared__ __align__(16) uint32_t hist[kBins];
    __shared__ uint32_t s_top[kSelWarps], s_low[kSelWarps], wsum[kSelWarps], wsum2[kSelWarps];
    __shared__ uint32_t s_bin, s_rank, s_count;
    // What reads the lists may be launched: it waits for this grid's end.
    asm volatile("griddepcontrol.launch_dependents;");
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int32_t g = blockIdx.x, i = blockIdx.y;
    const int64_t pair = (int64_t)i * p.Hkv + g;
    if (tid == 0 && g == 0) {
        const int32_t raw = __ldg(p.context_lens + i);
        if (raw < 0) pa::raise_error(p.err, PA_DEVERR_CONTEXT);
        if (raw > p.max_blocks * p.bs) pa::raise_error(p.err, PA_DEVERR_TABLE_WIDTH);
    }
    const int32_t n = context_of(p, i), nb = (n + p.bs - 1) / p.bs;
    const int32_t* table = p.block_tables + (int64_t)i * p.max_blocks;
    int32_t* sel = p.sel_blocks + pair * p.keep;
    const int32_t count = min(nb, p.keep);
    if (tid == 0) p.sel_lens[pair] = nb ? (count - 1) * p.bs + n - (nb - 1) * p.bs : 0;
    for (int32_t j = count + tid; j < p.keep; j += kSelThreads) sel[j] = -1;
    const int32_t k = p.keep - p.first - p.last, m = nb - p.first - p.last;   // k < m below
    const int32_t head = nb <= p.keep ? nb : p.first;
    auto keep_always = [&](int32_t to, int32_t from) {   // no score looks at these ids
        const int32_t id = __ldg(table + from);
        if (g == 0 && (uint32_t)id >= (uint32_t)p.num_blocks) pa::raise_error(p.err, PA_DEVERR_BLOCK_ID);
        sel[to] = id;
    };
    for (int32_t j = tid; j < head; j += kSelThreads) keep_always(j, j);
    if (nb > p.keep)
        for (int32_t j = tid; j < p.last; j += kSelThreads) keep_always(p.keep - p.last + j, nb - p.last + j);
    for (int b = tid; b < kBins; b += kSelThreads) hist[b] = 0;
    const int32_t per = (m + kSelThreads - 1) / kSelThreads;   // kPer at most, if not 0
    const int32_t beg = min(max(m, 0), tid * per), end = min(max(m, 0), beg + per);
    int32_t id[kPer ? kPer : 1] = {};
    if constexpr (kPer > 0)
#pragma unroll
        for (int q = 0; q < kPer; ++q)
            id[q] = beg + q < end && nb > p.keep ? __ldg(table + p.first + beg + q) : 0;
    // The scores; CTAs that need none wait too, so that this grid ends after theirs.
    asm volatile("griddepcontrol.wait;" ::: "memory");
    if (nb <= p.keep || k == 0) return;
    const uint32_t* keys = p.keys + pair * p.max_blocks + p.first;
    uint32_t own[kPer ? kPer : 1];
    uint32_t top = 0, low = 0;    // the largest key, and the smallest's complement
    // f(key, place in the stretch) for each key of this thread
    auto each = [&](auto f) {
        if constexpr (kPer > 0) {
#pragma unroll
            for (int q = 0; q < kPer; ++q)
                if (beg + q < end) f(own[q], q);
        } else {
            for (int32_t j = beg; j < end; ++j) f(__ldcg(keys + j), j - beg);
        }
    };
    if constexpr (kPer > 0)
#pragma unroll
        for (int q = 0; q < kPer; ++q) own[q] = beg + q < end ? __ldcg(keys + beg + q) : 0;
    each([&](uint32_t x, int) {
        top = max(top, x);
        low = max(low, ~x);
    });
    top = __reduce_max_sync(0xffffffffu, top);
    low = __reduce_max_sync(0xffffffffu, low);
    if (lane == 0) {
        s_top[warp] = top;
        s_low[warp] = low;
    }
    __syncthreads();
    top = __reduce_max_sync(0xffffffffu, s_top[lane % kSelWarps]);
    uint32_t base = ~__reduce_max_sync(0xffffffffu, s_low[lane % kSelWarps]);
    int width = 32 - __clz(top - base);            // bits of the range; 0: all keys are equal
    int shift = max(0, width - kBinBits);
    uint32_t rank = (uint32_t)k, limit, ties;      // chosen: keys above limit, and `ties` equal ones
    for (;;) {
        each([&](uint32_t x, int) {
            x -= base;                             // keys below base wrap to large numbers
            if (width == 32 || (x >> width) == 0) atomicAdd(&hist[x >> shift], 1u);
        });
        __syncthreads();
        // Counts from the top: thread t owns bins 4 t' .. 4 t' + 3 with t' = kSelThreads - 1 - t.
        const int b0 = (kSelThreads - 1 - tid) * (kBins / kSelThreads);
        const uint4 c4 = *reinterpret_cast<const uint4*>(hist + b0);
        *reinterpret_cast<uint4*>(hist + b0) = make_uint4(0, 0, 0, 0);
        const uint32_t mine = c4.x + c4.y + c4.z + c4.w;
        uint32_t upto = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const uint32_t y = __shfl_up_sync(0xffffffffu, upto, o);
            if (lane >= o) upto += y;
        }
        if (lane == 31) wsum[warp] = upto;
        __syncthreads();
        upto += __reduce_add_sync(0xffffffffu, lane < warp ? wsum[lane % kSelWarps] : 0u);
        if (upto >= rank && upto - mine < rank) {   // one thread
            uint32_t want = rank - (upto - mine), c = c4.w;
            int q = 3;
            if (c < want) want -= c, c = c4.z, q = 2;
            if (q == 2 && c < want) want -= c, c = c4.y, q = 1;
            if (q == 1 && c < want) want -= c, c = c4.x, q = 0;
            s_bin = b0 + q;
            s_rank = want;
            s_count = c;
        }
        __syncthreads();
        base += s_bin << shift;
        rank = s_rank;
        if (shift == 0) {
            limit = base;
            ties = rank;
            break;
        }
        if (rank == s_count) {      // the whole bin is wanted; base > 0, for k < m
            limit = base - 1;
            ties = 0;
            break;
        }
        width = shift;
        shift = max(0, shift - kBinBits);
    }
    // ---- ids in context order
    uint32_t above = 0, equal = 0;
    each([&](uint32_t x, int) {
        above += x > limit;
        equal += x == limit;
    });
    uint32_t a = above, e = equal;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const uint32_t ya = __shfl_up_sync(0xffffffffu, a, o), ye = __shfl_up_sync(0xffffffffu, e, o);
        if (lane >= o) {
            a += ya;
            e += ye;
        }
    }
    if (lane == 31) {
        wsum[warp] = a;
        wsum2[warp] = e;
    }
    __syncthreads();
    a += __reduce_add_sync(0xffffffffu, lane < warp ? wsum[lane % kSelWarps] : 0u) - above;
    e += __reduce_add_sync(0xffffffffu, lane < warp ? wsum2[lane % kSelWarps] : 0u) - equal;
    uint32_t at = a + min(e, ties);
    each([&](uint32_t x, int q) {
        const bool take = x > limit || (x == limit && e < ties);
        e += x == limit;
        if (take) sel[p.first + at++] = kPer ? id[kPer ? q : 0] : __ldg(table + p.first + beg + q);
    });
}

template <bool kBF16, int D>
pa_status launch_score(const SelectParams& p, dim3 grid, size_t smem, cudaStream_t stream) {
    auto kern = score_kernel<kBF16, D>;
    static pa::DeviceOnce once;
    if (!pa::allow_smem(once, kern, kScoreSmem)) return PA_ERR_CUDA;
    kern<<<grid, kThreads, smem, stream>>>(p);
    return pa::cuda_status(cudaGetLastError());
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

}  // namespace

extern "C" {

PA_API pa_status pa_summarize_blocks(const void* k_cache, const int32_t* block_ids,
                                     const int32_t* fills, int32_t n, void* boxes,
                                     float* box_scale, int32_t num_blocks, int32_t block_size,
                                     int32_t Hkv, int32_t d, pa_dtype dtype, void* stream) {
    if (n < 0 || num_blocks < 0 || Hkv <= 0) return PA_ERR_INVALID;
    if (dtype != PA_F16 && dtype != PA_BF16) return PA_ERR_UNSUPPORTED;
    if (d != 64 && d != 128) return PA_ERR_UNSUPPORTED;
    if (block_size != 8 && block_size != 16 && block_size != 32) return PA_ERR_UNSUPPORTED;
    if ((int64_t)n * Hkv > ((int64_t)1 << 27)) return PA_ERR_UNSUPPORTED;   // a warp each
    if (n == 0) return PA_OK;
    if (!k_cache || !block_ids || !boxes || !box_scale) return PA_ERR_INVALID;
    if (!aligned16(k_cache) || !aligned16(boxes)) return PA_ERR_INVALID;
    unsigned int* err = pa::device_error_word();
    if (!err) return PA_ERR_CUDA;
    const uint32_t pairs = (uint32_t)((int64_t)n * Hkv);
    auto kern = d == 128 ? (dtype == PA_BF16 ? summarize_kernel<true, 128> : summarize_kernel<false, 128>)
                         : (dtype == PA_BF16 ? summarize_kernel<true, 64> : summarize_kernel<false, 64>);
    kern<<<(pairs + kThreads / 32 - 1) / (kThreads / 32), kThreads, 0, static_cast<cudaStream_t>(stream)>>>(
        static_cast<const uint4*>(k_cache), block_ids, fills, pairs, (uint32_t)Hkv, block_size,
        num_blocks, static_cast<uint2*>(boxes), box_scale, err);
    return pa::cuda_status(cudaGetLastError());
}

PA_API size_t pa_select_blocks_workspace_size(int32_t B, int32_t Hkv, int32_t max_blocks) {
    if (B < 0 || Hkv <= 0 || max_blocks <= 0) return 0;
    return (size_t)B * Hkv * (size_t)max_blocks * sizeof(uint32_t);
}

PA_API pa_status pa_select_blocks(const void* q, const void* boxes, const float* box_scale,
                                  const int32_t* block_tables, int32_t max_blocks,
                                  const int32_t* context_lens, int32_t B, int32_t H, int32_t Hkv,
                                  int32_t d, int32_t block_size, int32_t num_blocks, int32_t keep,
                                  int32_t first, int32_t last, pa_dtype dtype,
                                  int32_t* sel_blocks, int32_t* sel_lens, void* workspace,
                                  size_t ws_bytes, void* stream) {
    if (B < 0 || H <= 0 || Hkv <= 0 || max_blocks <= 0 || num_blocks <= 0 || first < 0 || last < 1 ||
        keep < 1 || (int64_t)first + last > keep)
        return PA_ERR_INVALID;
    if (dtype != PA_F16 && dtype != PA_BF16) return PA_ERR_UNSUPPORTED;
    if (H % Hkv != 0 || H / Hkv > 128 || Hkv > 65535) return PA_ERR_UNSUPPORTED;
    if (d != 64 && d != 128) return PA_ERR_UNSUPPORTED;
    if (block_size != 8 && block_size != 16 && block_size != 32) return PA_ERR_UNSUPPORTED;
    if (B > 4096 || (int64_t)max_blocks * block_size > INT32_MAX) return PA_ERR_UNSUPPORTED;
    if (B == 0) return PA_OK;
    if (ws_bytes < pa_select_blocks_workspace_size(B, Hkv, max_blocks)) return PA_ERR_INVALID;
    if (!q || !boxes || !box_scale || !block_tables || !context_lens || !sel_blocks || !sel_lens ||
        !workspace)
        return PA_ERR_INVALID;
    if (!aligned16(q) || !aligned16(boxes) || (reinterpret_cast<uintptr_t>(workspace) & 3u))
        return PA_ERR_INVALID;
    SelectParams p;
    p.q = static_cast<const uint16_t*>(q);
    p.boxes = static_cast<const uint4*>(boxes);
    p.box_scale = box_scale;
    p.block_tables = block_tables;
    p.context_lens = context_lens;
    p.sel_blocks = sel_blocks;
    p.sel_lens = sel_lens;
    p.keys = static_cast<uint32_t*>(workspace);
    p.err = pa::device_error_word();
    if (!p.err) return PA_ERR_CUDA;
    p.max_blocks = max_blocks;
    p.H = H;
    p.Hkv = Hkv;
    p.G = H / Hkv;
    p.bs = block_size;
    p.num_blocks = num_blocks;
    p.keep = keep;
    p.first = first;
    p.last = last;
    const int sms = pa::device_sm_count();
    if (!sms) return PA_ERR_CUDA;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    const int32_t most = max_blocks - first - last;   // blocks to score, at most
    if (max_blocks > keep && keep > first + last) {
        // KV heads of a CTA: as many as it has lane groups for and query codes fit.
        const int units = kThreads / (d / 16);
        const int fit = kCodeBytes / (p.G * (d + 4));
        p.heads = Hkv < units ? Hkv : units;
        if (p.heads > fit) p.heads = fit;
        const int groups = (Hkv + p.heads - 1) / p.heads;
        // Blocks of a CTA at most: two CTAs per SM share all there may be, in whole steps.
        const int64_t all = (int64_t)B * groups * most;
        int64_t tile = (all + 2ll * sms - 1) / (2ll * sms);
        const int least = 4 * (units / p.heads);      // one step of every lane group
        tile = (tile + least - 1) / least * least;
        if (tile > kMaxTile) tile = kMaxTile / least * least;
        p.unit = least;
        p.tile = (int32_t)(tile < most ? tile : most);
        const dim3 grid((unsigned)((most + p.tile - 1) / p.tile), (unsigned)B, (unsigned)groups);
        const size_t smem = kRing * kStepBytes + (size_t)p.heads * p.G * (d + 4) + (size_t)p.tile * 4;
        const pa_status done =
            d == 128 ? (dtype == PA_BF16 ? launch_score<true, 128>(p, grid, smem, st)
                                         : launch_score<false, 128>(p, grid, smem, st))
                     : (dtype == PA_BF16 ? launch_score<true, 64>(p, grid, smem, st)
                                         : launch_score<false, 64>(p, grid, smem, st));
        if (done != PA_OK) return done;
    }
    // The selection starts while the scores are computed and waits for them.
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)Hkv, (unsigned)B);
    cfg.blockDim = dim3(kSelThreads);
    cfg.stream = st;
    cudaLaunchAttribute attr{};
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = max_blocks > keep && keep > first + last ? 1 : 0;
    auto select = most <= 2 * kSelThreads ? select_kernel<2>
                  : most <= 8 * kSelThreads ? select_kernel<8>
                  : most <= 32 * kSelThreads ? select_kernel<32> : select_kernel<0>;
    return pa::cuda_status(cudaLaunchKernelEx(&cfg, select, p));
}

}  // extern "C"
