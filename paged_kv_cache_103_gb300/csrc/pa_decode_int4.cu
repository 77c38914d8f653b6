// Paged decode attention over the 4-bit cache (pa_decode_int4): what pa_decode
// computes, with K and V the rows that the codes of pa_reshape_and_cache_int4
// stand for (format: pa_cache_int4.cu).
//
// One CTA per (sequence, query head): its four warps take the tokens in turn,
// each with its own running maximum m, sum l and output o, merged at the end:
//     out = sum_w 2^(m_w - M) o_w / sum_w 2^(m_w - M) l_w,  M = max_w m_w.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cmath>

#include "pa.h"
#include "pa_common.cuh"

namespace {

constexpr int kWarps = 4;
constexpr float kLog2e = 1.4426950408889634f;

struct Int4Params {
    const uint16_t* q;
    uint16_t* out;
    const uint8_t *k_cache, *v_cache;
    const __half2 *k_scale, *v_scale;   // (s, m) per group of 64
    const int32_t* block_tables;
    const int32_t* context_lens;
    unsigned int* err;
    int32_t max_blocks, B, H, Hkv, G, bs, num_blocks;
    float scale_log2;
};

template <int D, bool kBF16>
__global__ void __launch_bounds__(kWarps * 32) decode_int4_kernel(const Int4Params p) {
    constexpr int kPer = D / 32;   // values per lane
    const int h = blockIdx.x, i = blockIdx.y, g = h / p.G;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    __shared__ float so[kWarps][D], sm[kWarps], sl[kWarps];
    int32_t n = p.context_lens[i];
    if (n < 0) {
        if (threadIdx.x == 0) pa::raise_error(p.err, PA_DEVERR_CONTEXT);
        n = 0;
    }
    if (n > (int64_t)p.max_blocks * p.bs) {
        if (threadIdx.x == 0) pa::raise_error(p.err, PA_DEVERR_TABLE_WIDTH);
        n = p.max_blocks * p.bs;
    }
    float q[kPer], o[kPer] = {};
    const int64_t qrow = ((int64_t)i * p.H + h) * D + lane * kPer;
    for (int e = 0; e < kPer; ++e) {
        const uint16_t u = p.q[qrow + e];
        q[e] = kBF16 ? __uint_as_float((uint32_t)u << 16) : __half2float(__ushort_as_half(u));
    }
    float m = -INFINITY, l = 0.f;
    for (int32_t t = warp; t < n; t += kWarps) {
        const int32_t blk = p.block_tables[(int64_t)i * p.max_blocks + t / p.bs];
        const bool ok = blk >= 0 && blk < p.num_blocks;
        if (!ok && lane == 0) pa::raise_error(p.err, PA_DEVERR_BLOCK_ID);
        const int64_t row = ((int64_t)(ok ? blk : 0) * p.Hkv + g) * p.bs + t % p.bs;
        const int grp = lane * kPer / 64;
        const float2 ks = __half22float2(p.k_scale[row * (D / 64) + grp]);
        const float2 vs = __half22float2(p.v_scale[row * (D / 64) + grp]);
        float dot = 0.f, v[kPer];
        for (int e = 0; e < kPer; ++e) {
            const int64_t at = row * (D / 2) + (lane * kPer + e) / 2;
            const int sh = 4 * (e & 1);
            dot += q[e] * fmaf(ks.x, (float)((p.k_cache[at] >> sh) & 15), ks.y);
            v[e] = fmaf(vs.x, (float)((p.v_cache[at] >> sh) & 15), vs.y);
        }
        for (int x = 16; x > 0; x >>= 1) dot += __shfl_xor_sync(0xffffffffu, dot, x);
        if (!ok) dot = 0.f;   // a block outside the pool reads as zeros
        const float s = dot * p.scale_log2, mn = fmaxf(m, s);
        const float a = exp2f(m - mn), w = exp2f(s - mn);
        l = l * a + w;
        for (int e = 0; e < kPer; ++e) o[e] = o[e] * a + (ok ? w * v[e] : 0.f);
        m = mn;
    }
    for (int e = 0; e < kPer; ++e) so[warp][lane * kPer + e] = o[e];
    if (lane == 0) {
        sm[warp] = m;
        sl[warp] = l;
    }
    __syncthreads();
    float M = -INFINITY, L = 0.f;
    for (int w = 0; w < kWarps; ++w) M = fmaxf(M, sm[w]);
    for (int w = 0; w < kWarps; ++w) L += n ? exp2f(sm[w] - M) * sl[w] : 0.f;
    for (int e = threadIdx.x; e < D; e += kWarps * 32) {
        float x = 0.f;
        for (int w = 0; w < kWarps; ++w) x += n ? exp2f(sm[w] - M) * so[w][e] : 0.f;
        const uint32_t r = pa::pack2<kBF16>(n ? x / L : 0.f, 0.f);
        p.out[((int64_t)i * p.H + h) * D + e] = (uint16_t)r;
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
    if (H % Hkv != 0 || (H / Hkv > 16 && H / Hkv % 16 != 0)) return PA_ERR_UNSUPPORTED;
    if (d != 64 && d != 128) return PA_ERR_UNSUPPORTED;
    if (block_size != 8 && block_size != 16 && block_size != 32) return PA_ERR_UNSUPPORTED;
    if (B > 4096 || (int64_t)max_blocks * block_size > INT32_MAX ||
        (int64_t)num_blocks * block_size > INT32_MAX)
        return PA_ERR_UNSUPPORTED;
    if (B > 0 && ws_bytes < pa_decode_workspace_size(B, H, d)) return PA_ERR_INVALID;
    if (B == 0) return PA_OK;
    if (!q || !k_cache || !v_cache || !k_scale || !v_scale || !block_tables || !context_lens ||
        !out || !workspace)
        return PA_ERR_INVALID;
    if ((reinterpret_cast<uintptr_t>(k_cache) | reinterpret_cast<uintptr_t>(v_cache) |
         reinterpret_cast<uintptr_t>(k_scale) | reinterpret_cast<uintptr_t>(v_scale)) & 15u)
        return PA_ERR_INVALID;
    if ((reinterpret_cast<uintptr_t>(q) | reinterpret_cast<uintptr_t>(out)) & 15u)
        return PA_ERR_INVALID;
    unsigned int* err = pa::device_error_word();
    if (!err) return PA_ERR_CUDA;
    Int4Params p;
    p.q = static_cast<const uint16_t*>(q);
    p.out = static_cast<uint16_t*>(out);
    p.k_cache = static_cast<const uint8_t*>(k_cache);
    p.v_cache = static_cast<const uint8_t*>(v_cache);
    p.k_scale = static_cast<const __half2*>(k_scale);
    p.v_scale = static_cast<const __half2*>(v_scale);
    p.block_tables = block_tables;
    p.context_lens = context_lens;
    p.err = err;
    p.max_blocks = max_blocks;
    p.B = B;
    p.H = H;
    p.Hkv = Hkv;
    p.G = H / Hkv;
    p.bs = block_size;
    p.num_blocks = num_blocks;
    p.scale_log2 = scale * kLog2e;
    const dim3 grid((unsigned)H, (unsigned)B);
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (d == 128 && dtype == PA_BF16) decode_int4_kernel<128, true><<<grid, kWarps * 32, 0, st>>>(p);
    if (d == 128 && dtype == PA_F16) decode_int4_kernel<128, false><<<grid, kWarps * 32, 0, st>>>(p);
    if (d == 64 && dtype == PA_BF16) decode_int4_kernel<64, true><<<grid, kWarps * 32, 0, st>>>(p);
    if (d == 64 && dtype == PA_F16) decode_int4_kernel<64, false><<<grid, kWarps * 32, 0, st>>>(p);
    return pa::cuda_status(cudaGetLastError());
}

}  // extern "C"
