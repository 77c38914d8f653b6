// Paged decode attention over the block-scaled 8-bit cache (pa_decode_int8_block /
// pa_decode_fp8_block): what pa_decode computes, with K and V the rows that the codes of
// pa_reshape_and_cache_int8_block / _fp8_block stand for (format: pa_cache_block8.cu).
//
// With x = s c for the codes c of a (block, KV head), the scale leaves both sums over codes:
//     q . K_j = s_b (q . c_j),   sum_j p_j V_j = sum_j (p_j s_b) c_j.
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cmath>
#include <cstring>

#include "pa.h"
#include "pa_common.cuh"

namespace {

constexpr int kMaxG = 16;
constexpr int kMaxBatch = 4096;
constexpr float kLog2e = 1.4426950408889634f;

struct Block8Params {
    const uint16_t* q;
    uint16_t* out;
    const uint8_t *k_cache, *v_cache;
    const float *k_scale, *v_scale;
    const int32_t* block_tables;
    const int32_t* context_lens;
    unsigned int* err;
    int32_t max_blocks, B, H, Hkv, bs_shift, num_blocks;
    float scale_log2;
};

template <bool kBF16>
__device__ __forceinline__ float widen(uint16_t v) {
    if constexpr (kBF16) return __uint_as_float((uint32_t)v << 16);
    __half h;
    memcpy(&h, &v, 2);
    return __half2float(h);
}

template <bool kInt8>
__device__ __forceinline__ float number(uint8_t code) {
    if constexpr (kInt8) return (float)(int8_t)code;
    uint32_t lo, hi;
    pa::e4m3x4_to_f16(code, lo, hi);
    return widen<false>((uint16_t)lo);
}

// A warp per (sequence, query head), one key after the other.
template <int D, bool kBF16, bool kInt8>
__global__ void __launch_bounds__(128) decode_kernel(const Block8Params p) {
    constexpr int N = D / 32;
    const int lane = threadIdx.x & 31;
    const int64_t w = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 5);
    const int32_t i = (int32_t)(w / p.H), h = (int32_t)(w % p.H);
    if (i >= p.B) return;
    const int32_t g = h / (p.H / p.Hkv);
    const int32_t raw = p.context_lens[i];
    const int64_t cap = (int64_t)p.max_blocks << p.bs_shift;
    if (h == 0 && lane == 0) {
        if (raw < 0) pa::raise_error(p.err, PA_DEVERR_CONTEXT);
        if (raw > cap) pa::raise_error(p.err, PA_DEVERR_TABLE_WIDTH);
    }
    const int32_t n = raw < 0 ? 0 : (int32_t)(raw > cap ? cap : raw);
    float q[N], o[N], m = -INFINITY, l = 0.f;
    for (int k = 0; k < N; ++k) {
        q[k] = widen<kBF16>(p.q[w * D + k * 32 + lane]) * p.scale_log2;
        o[k] = 0.f;
    }
    for (int32_t j = 0; j < n; ++j) {
        const int32_t b = p.block_tables[(int64_t)i * p.max_blocks + (j >> p.bs_shift)];
        const bool ok = (uint32_t)b < (uint32_t)p.num_blocks;
        if (!ok && lane == 0) pa::raise_error(p.err, PA_DEVERR_BLOCK_ID);
        const int64_t tile = (int64_t)b * p.Hkv + g;
        const int64_t row = ((tile << p.bs_shift) + (j & ((1 << p.bs_shift) - 1))) * D;
        float dot = 0.f;
        if (ok)
            for (int k = 0; k < N; ++k) dot += q[k] * number<kInt8>(p.k_cache[row + k * 32 + lane]);
        for (int off = 16; off; off >>= 1) dot += __shfl_xor_sync(0xffffffffu, dot, off);
        const float x = ok ? dot * p.k_scale[tile] : 0.f;
        const float top = fmaxf(m, x), old = pa::fast_exp2(m - top), e = pa::fast_exp2(x - top);
        m = top;
        l = l * old + e;
        const float f = ok ? e * p.v_scale[tile] : 0.f;
        for (int k = 0; k < N; ++k)
            o[k] = o[k] * old + (ok ? f * number<kInt8>(p.v_cache[row + k * 32 + lane]) : 0.f);
    }
    const float inv = n ? 1.f / l : 0.f;
    for (int k = 0; k < N; ++k)
        p.out[w * D + k * 32 + lane] = (uint16_t)pa::pack2<kBF16>(o[k] * inv, 0.f);
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
    const int G = H / Hkv;
    if (G > kMaxG && G % kMaxG != 0) return PA_ERR_UNSUPPORTED;
    if (d != 64 && d != 128) return PA_ERR_UNSUPPORTED;
    if (block_size != 8 && block_size != 16 && block_size != 32) return PA_ERR_UNSUPPORTED;
    if ((int64_t)num_blocks * Hkv > INT32_MAX || B > kMaxBatch ||
        (int64_t)num_blocks * block_size > INT32_MAX || (int64_t)max_blocks * block_size > INT32_MAX)
        return PA_ERR_UNSUPPORTED;
    const int64_t max_chunks = ((int64_t)max_blocks * block_size + 31) / 32;
    const int64_t subs = G > kMaxG ? G / kMaxG : 1;
    if ((int64_t)B * Hkv * subs * (max_chunks + 2) >= ((int64_t)1 << 30)) return PA_ERR_UNSUPPORTED;
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
    p.err = pa::device_error_word();
    if (!p.err) return PA_ERR_CUDA;
    p.q = static_cast<const uint16_t*>(q);
    p.out = static_cast<uint16_t*>(out);
    p.k_cache = static_cast<const uint8_t*>(k_cache);
    p.v_cache = static_cast<const uint8_t*>(v_cache);
    p.k_scale = k_scale;
    p.v_scale = v_scale;
    p.block_tables = block_tables;
    p.context_lens = context_lens;
    p.max_blocks = max_blocks;
    p.B = B;
    p.H = H;
    p.Hkv = Hkv;
    p.bs_shift = block_size == 8 ? 3 : block_size == 16 ? 4 : 5;
    p.num_blocks = num_blocks;
    p.scale_log2 = scale * kLog2e;
    const bool bf16 = dtype == PA_BF16;
    auto kern = d == 128 ? (bf16 ? decode_kernel<128, true, kInt8> : decode_kernel<128, false, kInt8>)
                         : (bf16 ? decode_kernel<64, true, kInt8> : decode_kernel<64, false, kInt8>);
    kern<<<(unsigned)(((int64_t)B * H + 3) / 4), 128, 0, static_cast<cudaStream_t>(stream)>>>(p);
    return pa::cuda_status(cudaGetLastError());
}

}  // namespace

extern "C" {

PA_API pa_status pa_decode_int8_block(const void* q, const void* k_cache, const void* v_cache,
                                      const float* k_scale, const float* v_scale,
                                      const int32_t* block_tables, int32_t max_blocks,
                                      const int32_t* context_lens, int32_t max_context_len,
                                      int32_t B, int32_t H, int32_t Hkv, int32_t d,
                                      int32_t block_size, int32_t num_blocks, float scale,
                                      pa_dtype dtype, void* out, void* workspace,
                                      size_t ws_bytes, void* stream) {
    return decode<true>(q, k_cache, v_cache, k_scale, v_scale, block_tables, max_blocks,
                        context_lens, max_context_len, B, H, Hkv, d, block_size, num_blocks, scale,
                        dtype, out, workspace, ws_bytes, stream);
}

PA_API pa_status pa_decode_fp8_block(const void* q, const void* k_cache, const void* v_cache,
                                     const float* k_scale, const float* v_scale,
                                     const int32_t* block_tables, int32_t max_blocks,
                                     const int32_t* context_lens, int32_t max_context_len,
                                     int32_t B, int32_t H, int32_t Hkv, int32_t d,
                                     int32_t block_size, int32_t num_blocks, float scale,
                                     pa_dtype dtype, void* out, void* workspace,
                                     size_t ws_bytes, void* stream) {
    return decode<false>(q, k_cache, v_cache, k_scale, v_scale, block_tables, max_blocks,
                         context_lens, max_context_len, B, H, Hkv, d, block_size, num_blocks, scale,
                         dtype, out, workspace, ws_bytes, stream);
}

}  // extern "C"
