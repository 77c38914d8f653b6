// Block summaries (pa_summarize_blocks) and the selection of the blocks that a
// decode step attends over (pa_select_blocks); pa_decode_selected then reads
// only those.
//
// A context's keys are summarised per (block, KV head) by the smallest and the
// largest key value of each head-dim channel, lo_c and hi_c, as INT8 codes with
// one fp32 scale.  For a query q the block's largest possible score is at most
//     sum_c max(q_c lo_c, q_c hi_c) = sum_c q_c (q_c > 0 ? hi_c : lo_c),
// so a block whose bound is low holds no key that matters.  The query is coded
// in INT8 too, which makes the sum an integer: the score, and with it the
// selection, does not depend on the order of summation.
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

template <bool kBF16>
__device__ __forceinline__ uint32_t min2(uint32_t a, uint32_t b) {
    uint32_t r;
    if constexpr (kBF16)
        asm("min.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    else
        asm("min.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}

template <bool kBF16>
__device__ __forceinline__ uint32_t max2(uint32_t a, uint32_t b) {
    uint32_t r;
    if constexpr (kBF16)
        asm("max.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    else
        asm("max.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}

__device__ __forceinline__ uint32_t code8(float x, float s) {
    return (uint32_t)max(-127, min(127, __float2int_rn(__fdiv_rn(x, s)))) & 0xFFu;
}

// Thread v: channels 8 (v % (D / 8)) .. + 7 of one (listed block, KV head).
template <bool kBF16, int D>
__global__ void __launch_bounds__(kThreads)
summarize_kernel(const uint4* __restrict__ k_cache, const int32_t* __restrict__ block_ids,
                 const int32_t* __restrict__ fills, uint32_t vecs, uint32_t Hkv, int32_t bs,
                 int32_t num_blocks, uint2* __restrict__ boxes, float* __restrict__ box_scale,
                 unsigned int* __restrict__ err) {
    constexpr uint32_t kRow = D / 8;
    const uint32_t v = blockIdx.x * kThreads + threadIdx.x;
    const bool live = v < vecs;   // vecs is a multiple of kRow
    const uint32_t pair = (live ? v : 0) / kRow, l = v % kRow;
    const uint32_t e = pair / Hkv, h = pair - e * Hkv;
    const int32_t id = live ? __ldg(block_ids + e) : -1;
    const bool ok = id >= 0 && id < num_blocks;
    int32_t fill = live && fills ? __ldg(fills + e) : bs;
    if (live && l == 0 && h == 0) {
        if (!ok) pa::raise_error(err, PA_DEVERR_BLOCK_ID);
        if (fill < 0 || fill > bs) pa::raise_error(err, PA_DEVERR_CONTEXT);
    }
    fill = max(0, min(bs, fill));
    uint32_t lo[4] = {0, 0, 0, 0}, hi[4] = {0, 0, 0, 0};
    if (ok && fill > 0) {
        const int64_t stride = (int64_t)Hkv * kRow;   // between token rows
        const uint4* src = k_cache + (int64_t)id * bs * stride + h * kRow + l;
        for (int32_t r0 = 0; r0 < fill; r0 += 8) {
            uint4 x[8];
#pragma unroll
            for (int r = 0; r < 8; ++r)   // the last row again past the fill: min and max keep
                x[r] = __ldg(src + min(r0 + r, fill - 1) * stride);
#pragma unroll
            for (int r = 0; r < 8; ++r) {
                const uint32_t w[4] = {x[r].x, x[r].y, x[r].z, x[r].w};
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const bool start = r0 == 0 && r == 0;
                    lo[j] = start ? w[j] : min2<kBF16>(lo[j], w[j]);
                    hi[j] = start ? w[j] : max2<kBF16>(hi[j], w[j]);
                }
            }
        }
    }
    float a = 0.f;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const float2 x = widen2<kBF16>(lo[j]), y = widen2<kBF16>(hi[j]);
        a = fmaxf(a, fmaxf(fmaxf(fabsf(x.x), fabsf(x.y)), fmaxf(fabsf(y.x), fabsf(y.y))));
    }
#pragma unroll
    for (uint32_t o = 1; o < kRow; o <<= 1) a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, o));
    if (!ok) return;
    const float s = __fdiv_rn(a, 127.f);
    uint32_t c[4] = {0, 0, 0, 0};   // lo codes, hi codes
    if (s > 0.f) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const float2 x = widen2<kBF16>(lo[j]), y = widen2<kBF16>(hi[j]);
            c[j >> 1] |= (code8(x.x, s) | code8(x.y, s) << 8) << (16 * (j & 1));
            c[2 + (j >> 1)] |= (code8(y.x, s) | code8(y.y, s) << 8) << (16 * (j & 1));
        }
    }
    const int64_t row = (int64_t)id * Hkv + h;
    boxes[row * 2 * kRow + l] = make_uint2(c[0], c[1]);
    boxes[row * 2 * kRow + kRow + l] = make_uint2(c[2], c[3]);
    if (l == 0) box_scale[row] = s;
}

struct SelectParams {
    const uint16_t* q;
    const uint4* boxes;
    const float* box_scale;
    const int32_t* block_tables;
    const int32_t* context_lens;
    int32_t* sel_blocks;
    int32_t* sel_lens;
    uint32_t* keys;      // [B * Hkv][max_blocks]
    unsigned int* err;
    int32_t max_blocks, H, Hkv, G, bs, num_blocks, keep, first, last;
};

// A float as an unsigned number of the same order (-0 as +0).
__device__ __forceinline__ uint32_t ordered(float x) {
    const uint32_t u = __float_as_uint(x + 0.f);
    return (u >> 31) ? ~u : (u | 0x80000000u);
}

// One CTA per (sequence, KV head): scores, the k-th largest by radix, and the
// chosen ids in context order.
template <bool kBF16, int D>
__global__ void __launch_bounds__(kThreads) select_kernel(const SelectParams p) {
    constexpr int kLanes = D / 16;           // lanes per block: 16 channels each
    constexpr int kPerWarp = 32 / kLanes;    // blocks per warp and step
    constexpr int kWarps = kThreads / 32;
    extern __shared__ uint32_t smem[];
    uint32_t* qc = smem;                                       // [G][D / 4] query codes
    float* sq = reinterpret_cast<float*>(smem + p.G * (D / 4));  // [G]
    __shared__ uint32_t hist[256];
    __shared__ uint32_t wsum[2][kWarps], s_prefix, s_rank;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int32_t g = blockIdx.x, i = blockIdx.y;
    const int64_t pair = (int64_t)i * p.Hkv + g;
    int32_t n = __ldg(p.context_lens + i);
    if (tid == 0 && g == 0) {
        if (n < 0) pa::raise_error(p.err, PA_DEVERR_CONTEXT);
        if (n > (int64_t)p.max_blocks * p.bs) pa::raise_error(p.err, PA_DEVERR_TABLE_WIDTH);
    }
    n = (int32_t)max((int64_t)0, min((int64_t)n, (int64_t)p.max_blocks * p.bs));
    const int32_t nb = (n + p.bs - 1) / p.bs;
    const int32_t* table = p.block_tables + (int64_t)i * p.max_blocks;
    int32_t* sel = p.sel_blocks + pair * p.keep;
    const int32_t count = min(nb, p.keep);
    if (tid == 0) p.sel_lens[pair] = nb ? (count - 1) * p.bs + n - (nb - 1) * p.bs : 0;
    for (int32_t j = count + tid; j < p.keep; j += kThreads) sel[j] = -1;
    if (nb <= p.keep) {
        for (int32_t j = tid; j < nb; j += kThreads) sel[j] = __ldg(table + j);
        return;
    }
    // ---- query codes
    for (int h = warp; h < p.G; h += kWarps) {
        const uint16_t* q = p.q + ((int64_t)i * p.H + g * p.G + h) * D;
        float2 x[D / 64];
        float a = 0.f;
#pragma unroll
        for (int j = 0; j < D / 64; ++j) {
            x[j] = widen2<kBF16>(*reinterpret_cast<const uint32_t*>(q + j * 64 + lane * 2));
            a = fmaxf(a, fmaxf(fabsf(x[j].x), fabsf(x[j].y)));
        }
        for (int o = 16; o > 0; o >>= 1) a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, o));
        const float s = __fdiv_rn(a, 127.f);
#pragma unroll
        for (int j = 0; j < D / 64; ++j)
            reinterpret_cast<uint16_t*>(qc)[h * (D / 2) + j * 32 + lane] =
                s > 0.f ? (uint16_t)(code8(x[j].x, s) | code8(x[j].y, s) << 8) : 0;
        if (lane == 0) sq[h] = s;
    }
    __syncthreads();
    // ---- scores of the blocks that are not kept anyway
    const int32_t lo = p.first, hi = nb - p.last;
    uint32_t* keys = p.keys + pair * p.max_blocks;
    const int sub = lane / kLanes, l = lane % kLanes;
    for (int32_t j0 = lo + warp * kPerWarp; j0 < hi; j0 += kWarps * kPerWarp) {
        const int32_t j = j0 + sub;
        const int32_t id = j < hi ? __ldg(table + j) : -1;
        const bool ok = id >= 0 && id < p.num_blocks;
        if (j < hi && !ok && l == 0) pa::raise_error(p.err, PA_DEVERR_BLOCK_ID);
        const int64_t row = (int64_t)(ok ? id : 0) * p.Hkv + g;
        const uint4 a = __ldg(p.boxes + row * 2 * kLanes + l);
        const uint4 b = __ldg(p.boxes + row * 2 * kLanes + kLanes + l);
        const float S = __ldg(p.box_scale + row);
        const uint32_t lw[4] = {a.x, a.y, a.z, a.w}, hw[4] = {b.x, b.y, b.z, b.w};
        float best = 0.f;
        for (int h = 0; h < p.G; ++h) {
            int dot = 0;
#pragma unroll
            for (int w = 0; w < 4; ++w) {
                const uint32_t c = qc[h * (D / 4) + l * 4 + w];
                const uint32_t neg = __vcmpgts4(0u, c);
                dot = __dp4a((int)((lw[w] & neg) | (hw[w] & ~neg)), (int)c, dot);
            }
#pragma unroll
            for (int o = 1; o < kLanes; o <<= 1) dot += __shfl_xor_sync(0xffffffffu, dot, o);
            const float x = __fmul_rn(__fmul_rn((float)dot, sq[h]), S);
            best = h ? fmaxf(best, x) : x;
        }
        if (l == 0 && j < hi) keys[j] = ok ? ordered(best) : 0u;
    }
    __syncthreads();
    // ---- the k-th largest key, eight bits at a time
    const int32_t k = p.keep - p.first - p.last;
    if (tid == 0) {
        s_prefix = 0;
        s_rank = (uint32_t)k;
    }
    for (int pass = 3; pass >= 0; --pass) {
        hist[tid] = 0;
        __syncthreads();
        const uint32_t want = s_prefix;
        for (int32_t j = lo + tid; j < hi; j += kThreads) {
            const uint32_t x = keys[j];
            if (pass == 3 || (x >> (8 * pass + 8)) == want) atomicAdd(&hist[(x >> (8 * pass)) & 255], 1u);
        }
        __syncthreads();
        if (tid == 0 && k > 0) {
            uint32_t rank = s_rank;
            int b = 255;
            while (b > 0 && hist[b] < rank) rank -= hist[b--];
            s_prefix = want << 8 | (uint32_t)b;
            s_rank = rank;   // how many of this digit's keys are still wanted
        }
        __syncthreads();
    }
    const uint32_t limit = k > 0 ? s_prefix : 0xffffffffu;
    const uint32_t ties = k > 0 ? s_rank : 0u;   // keys equal to the limit, lowest index first
    // ---- ids in context order
    for (int32_t j = tid; j < p.first; j += kThreads) sel[j] = __ldg(table + j);
    for (int32_t j = tid; j < p.last; j += kThreads)
        sel[p.keep - p.last + j] = __ldg(table + nb - p.last + j);
    uint32_t taken = 0, tied = 0;   // over the tiles before this one
    for (int32_t j0 = lo; j0 < hi; j0 += kThreads) {
        const int32_t j = j0 + tid;
        const uint32_t x = j < hi ? keys[j] : 0u;
        const bool eq = j < hi && x == limit;
        const uint32_t meq = __ballot_sync(0xffffffffu, eq);
        const uint32_t below = (1u << lane) - 1u;
        if (lane == 0) wsum[0][warp] = __popc(meq);
        __syncthreads();
        uint32_t before = tied, all = 0;
        for (int w = 0; w < kWarps; ++w) {
            if (w < warp) before += wsum[0][w];
            all += wsum[0][w];
        }
        const bool take = k > 0 && j < hi && (x > limit || (eq && before + __popc(meq & below) < ties));
        const uint32_t mt = __ballot_sync(0xffffffffu, take);
        if (lane == 0) wsum[1][warp] = __popc(mt);
        __syncthreads();
        uint32_t at = taken, sum = 0;
        for (int w = 0; w < kWarps; ++w) {
            if (w < warp) at += wsum[1][w];
            sum += wsum[1][w];
        }
        if (take) sel[p.first + at + __popc(mt & below)] = __ldg(table + j);
        taken += sum;
        tied += all;
    }
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
    if ((int64_t)n * Hkv * (d / 8) > ((int64_t)1 << 31)) return PA_ERR_UNSUPPORTED;
    if (n == 0) return PA_OK;
    if (!k_cache || !block_ids || !boxes || !box_scale) return PA_ERR_INVALID;
    if (!aligned16(k_cache) || !aligned16(boxes)) return PA_ERR_INVALID;
    unsigned int* err = pa::device_error_word();
    if (!err) return PA_ERR_CUDA;
    const uint32_t vecs = (uint32_t)((int64_t)n * Hkv * (d / 8));
    auto kern = d == 128 ? (dtype == PA_BF16 ? summarize_kernel<true, 128> : summarize_kernel<false, 128>)
                         : (dtype == PA_BF16 ? summarize_kernel<true, 64> : summarize_kernel<false, 64>);
    kern<<<(vecs + kThreads - 1) / kThreads, kThreads, 0, static_cast<cudaStream_t>(stream)>>>(
        static_cast<const uint4*>(k_cache), block_ids, fills, vecs, (uint32_t)Hkv, block_size,
        num_blocks, static_cast<uint2*>(boxes), box_scale, err);
    return pa::cuda_status(cudaGetLastError());
}

PA_API size_t pa_select_blocks_workspace_size(int32_t B, int32_t Hkv, int32_t max_blocks) {
    if (B < 0 || Hkv <= 0 || max_blocks <= 0) return 0;
    return (size_t)B * Hkv * ((size_t)max_blocks + 1) * sizeof(uint32_t);
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
    if (H % Hkv != 0 || H / Hkv > 128) return PA_ERR_UNSUPPORTED;
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
    p.keys = static_cast<uint32_t*>(workspace) + (size_t)B * Hkv;
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
    const size_t smem = (size_t)p.G * (d + 4);
    auto kern = d == 128 ? (dtype == PA_BF16 ? select_kernel<true, 128> : select_kernel<false, 128>)
                         : (dtype == PA_BF16 ? select_kernel<true, 64> : select_kernel<false, 64>);
    kern<<<dim3((unsigned)Hkv, (unsigned)B), kThreads, smem, static_cast<cudaStream_t>(stream)>>>(p);
    return pa::cuda_status(cudaGetLastError());
}

}  // extern "C"
