// The block-scaled 8-bit KV cache's append (pa_reshape_and_cache_int8_block / _fp8_block)
// and its read back (pa_gather_cache_int8_block / _fp8_block).
//
// Format ("LLM推理优化技术地图：从KV Cache到量化与投机解码", section 4.3, KV cache
// quantisation; the page fixes none).  A code is an INT8 integer or an E4M3 number and
// stands for code * scale, with one fp32 scale per (block, KV head).  Codes are
// [num_blocks][Hkv][block_size][d], heads outside rows: a (block, KV head) tile is one
// contiguous run.  Against a scale per token this leaves 4 bytes a block and head instead of 4
// bytes a token and head to read, and the decode one factor a block.
//
// What an append has to do: with R the rows of a block that the call writes and
// a = max |x| over them, base = 0 if row 0 is among them, else the block's scale,
//     s = max(base, a / TOP);   rows in R: code(x / s);
//     other rows, if 0 < base < s: code(c * (base / s)).
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cstring>

#include "pa.h"
#include "pa_common.cuh"

namespace {

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

// Four values -> four codes, the first in the low byte.
template <bool kInt8>
__device__ __forceinline__ uint32_t code4(float a, float b, float c, float d) {
    if constexpr (kInt8) {
        auto one = [](float x) { return (uint32_t)max(-127, min(127, __float2int_rn(x))) & 255u; };
        return one(a) | one(b) << 8 | one(c) << 16 | one(d) << 24;
    } else {
        uint16_t lo, hi;
        asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(lo) : "f"(b), "f"(a));
        asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(hi) : "f"(d), "f"(c));
        return (uint32_t)lo | (uint32_t)hi << 16;
    }
}

// Four codes -> the numbers that they are.
template <bool kInt8>
__device__ __forceinline__ float4 number4(uint32_t codes) {
    uint32_t lo, hi;
    if constexpr (kInt8)
        pa::s8x4_to_f16(codes, lo, hi);
    else
        pa::e4m3x4_to_f16(codes, lo, hi);
    const float2 a = widen2<false>(lo), b = widen2<false>(hi);
    return make_float4(a.x, a.y, b.x, b.y);
}

constexpr int kThreads = 128;
constexpr int kVec = 4;      // values a lane takes at a time

// A warp per (token, KV head, K or V).  The first token of a block in the call has the block's
// work; the other tokens' warps leave it to that one.
template <bool kBF16, bool kInt8, int D>
__global__ void __launch_bounds__(kThreads)
append_kernel(const uint2* __restrict__ k_new, const uint2* __restrict__ v_new,
              const int64_t* __restrict__ slots, int32_t T, int32_t Hkv, int bs_shift,
              uint32_t* k_cache, uint32_t* v_cache, float* k_scale, float* v_scale,
              int64_t num_slots, unsigned int* err) {
    constexpr int kRow = D / kVec;       // lanes' places of a row
    constexpr float kTop = kInt8 ? 127.f : 448.f;
    const int lane = threadIdx.x & 31;
    const int64_t w = (int64_t)blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5);
    const int32_t t = (int32_t)(w / (2 * Hkv)), hv = (int32_t)(w - (int64_t)t * 2 * Hkv);
    if (t >= T) return;
    const int32_t h = hv >> 1;
    const int64_t slot = slots[t];
    if (slot < 0) return;
    if (slot >= num_slots) {
        if (hv == 0 && lane == 0) pa::raise_error(err, PA_DEVERR_SLOT);
        return;
    }
    const int64_t block = slot >> bs_shift;
    // Is there an earlier token of this block?  The nearest one that is written tells.
    for (int32_t j = t - 1 - lane, first = t - 1; first >= 0; first -= 32, j -= 32) {
        const int64_t s = j >= 0 ? slots[j] : -1;
        const uint32_t some = __ballot_sync(0xffffffffu, s >= 0 && s < num_slots);
        if (!some) continue;
        if (__shfl_sync(0xffffffffu, s, __ffs(some) - 1) >> bs_shift == block) return;
        break;
    }
    const uint2* x = hv & 1 ? v_new : k_new;
    uint32_t* cache = (hv & 1 ? v_cache : k_cache) + ((block * Hkv + h) << bs_shift) * kRow;
    float* scale = (hv & 1 ? v_scale : k_scale) + block * Hkv + h;
    // f(row of the block, token) for each token of the block
    auto each = [&](auto f) {
        for (int32_t first = t; first < T; first += 32) {
            const int64_t s = first + lane < T ? slots[first + lane] : -1;
            const uint32_t some = __ballot_sync(0xffffffffu, s >= 0 && s < num_slots);
            const uint32_t same = __ballot_sync(0xffffffffu, s >= 0 && s >> bs_shift == block);
            const uint32_t other = some & ~same;
            const uint32_t mine = other ? same & ((other & -other) - 1) : same;
            for (uint32_t m = mine; m; m &= m - 1) {
                const int l = __ffs(m) - 1;
                f((int32_t)(__shfl_sync(0xffffffffu, s, l) & ((1 << bs_shift) - 1)), first + l);
            }
            if (other) break;
        }
    };
    float a = 0.f;
    uint32_t written = 0;
    each([&](int32_t r, int32_t j) {
        written |= 1u << r;
        for (int l = lane; l < kRow; l += 32) {
            const uint2 y = x[((int64_t)j * Hkv + h) * kRow + l];
            const float2 p = widen2<kBF16>(y.x), q = widen2<kBF16>(y.y);
            a = fmaxf(a, fmaxf(fmaxf(fabsf(p.x), fabsf(p.y)), fmaxf(fabsf(q.x), fabsf(q.y))));
        }
    });
    a = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(a)));
    const float base = written & 1 ? 0.f : *scale;
    const float s = fmaxf(base, __fdiv_rn(a, kTop));
    if (base > 0.f && base < s) {
        const float ratio = __fdiv_rn(base, s);
        for (int r = 0; r < 1 << bs_shift; ++r) {
            if (written >> r & 1) continue;
            for (int l = lane; l < kRow; l += 32) {
                const float4 c = number4<kInt8>(cache[r * kRow + l]);
                cache[r * kRow + l] = code4<kInt8>(__fmul_rn(c.x, ratio), __fmul_rn(c.y, ratio),
                                                   __fmul_rn(c.z, ratio), __fmul_rn(c.w, ratio));
            }
        }
    }
    each([&](int32_t r, int32_t j) {
        for (int l = lane; l < kRow; l += 32) {
            const uint2 y = x[((int64_t)j * Hkv + h) * kRow + l];
            const float2 p = widen2<kBF16>(y.x), q = widen2<kBF16>(y.y);
            cache[r * kRow + l] = s > 0.f ? code4<kInt8>(__fdiv_rn(p.x, s), __fdiv_rn(p.y, s),
                                                         __fdiv_rn(q.x, s), __fdiv_rn(q.y, s))
                                          : 0u;
        }
    });
    __syncwarp();
    if (lane == 0) *scale = s;
}

// A thread per four values of k_out and of v_out.
template <bool kBF16, bool kInt8, int D>
__global__ void __launch_bounds__(kThreads)
gather_kernel(const uint32_t* k_cache, const uint32_t* v_cache, const float* k_scale,
              const float* v_scale, const int64_t* slots, int64_t vecs, int32_t Hkv, int bs_shift,
              int64_t num_slots, uint2* k_out, uint2* v_out, unsigned int* err) {
    constexpr int kRow = D / kVec;
    const int64_t v = (int64_t)blockIdx.x * kThreads + threadIdx.x;
    if (v >= vecs) return;
    const int64_t row = v / kRow, l = v % kRow, t = row / Hkv, h = row - t * Hkv;
    const int64_t slot = slots[t];
    if (slot < 0) return;
    if (slot >= num_slots) {
        if (h == 0 && l == 0) pa::raise_error(err, PA_DEVERR_SLOT);
        return;
    }
    const int64_t tile = (slot >> bs_shift) * Hkv + h;
    const int64_t at = ((tile << bs_shift) + (slot & ((1 << bs_shift) - 1))) * kRow + l;
    auto one = [&](const uint32_t* cache, const float* scale, uint2* out) {
        const float4 c = number4<kInt8>(cache[at]);
        const float s = scale[tile];
        out[v] = make_uint2(pa::pack2<kBF16>(__fmul_rn(c.x, s), __fmul_rn(c.y, s)),
                            pa::pack2<kBF16>(__fmul_rn(c.z, s), __fmul_rn(c.w, s)));
    };
    one(k_cache, k_scale, k_out);
    one(v_cache, v_scale, v_out);
}

bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

int shift_of(int32_t block_size) {
    return block_size == 8 ? 3 : block_size == 16 ? 4 : block_size == 32 ? 5 : -1;
}

// Checks shared by the append and the read back.
pa_status check(const void* k, const void* v, const int64_t* slots, int32_t T, const void* k_cache,
                const void* v_cache, const void* k_scale, const void* v_scale, int32_t num_blocks,
                int32_t block_size, int32_t Hkv, int32_t d, pa_dtype dtype) {
    if (T < 0 || num_blocks < 0 || Hkv <= 0) return PA_ERR_INVALID;
    if (dtype != PA_F16 && dtype != PA_BF16) return PA_ERR_UNSUPPORTED;
    if (d != 64 && d != 128) return PA_ERR_UNSUPPORTED;
    if (shift_of(block_size) < 0) return PA_ERR_UNSUPPORTED;
    if (Hkv > (1 << 20)) return PA_ERR_UNSUPPORTED;
    if (T == 0) return PA_OK;
    if (!k || !v || !slots || !k_cache || !v_cache || !k_scale || !v_scale) return PA_ERR_INVALID;
    if (!aligned(k, 16) || !aligned(v, 16) || !aligned(k_cache, 16) || !aligned(v_cache, 16) ||
        !aligned(k_scale, 4) || !aligned(v_scale, 4) || !aligned(slots, 8))
        return PA_ERR_INVALID;
    return PA_OK;
}

template <bool kInt8>
pa_status append(const void* k_new, const void* v_new, const int64_t* slots, int32_t T,
                 void* k_cache, void* v_cache, float* k_scale, float* v_scale, int32_t num_blocks,
                 int32_t block_size, int32_t Hkv, int32_t d, pa_dtype dtype, void* stream) {
    const pa_status st = check(k_new, v_new, slots, T, k_cache, v_cache, k_scale, v_scale,
                               num_blocks, block_size, Hkv, d, dtype);
    if (st != PA_OK || T == 0) return st;
    unsigned int* err = pa::device_error_word();
    if (!err) return PA_ERR_CUDA;
    const int64_t warps = (int64_t)T * Hkv * 2, ctas = (warps + kThreads / 32 - 1) / (kThreads / 32);
    if (ctas > INT32_MAX) return PA_ERR_UNSUPPORTED;
    const bool bf16 = dtype == PA_BF16;
    auto kern = d == 128 ? (bf16 ? append_kernel<true, kInt8, 128> : append_kernel<false, kInt8, 128>)
                         : (bf16 ? append_kernel<true, kInt8, 64> : append_kernel<false, kInt8, 64>);
    kern<<<(unsigned)ctas, kThreads, 0, static_cast<cudaStream_t>(stream)>>>(
        static_cast<const uint2*>(k_new), static_cast<const uint2*>(v_new), slots, T, Hkv,
        shift_of(block_size), static_cast<uint32_t*>(k_cache), static_cast<uint32_t*>(v_cache),
        k_scale, v_scale, (int64_t)num_blocks * block_size, err);
    return pa::cuda_status(cudaGetLastError());
}

template <bool kInt8>
pa_status gather(const void* k_cache, const void* v_cache, const float* k_scale,
                 const float* v_scale, const int64_t* slots, int32_t T, void* k_out, void* v_out,
                 int32_t num_blocks, int32_t block_size, int32_t Hkv, int32_t d, pa_dtype dtype,
                 void* stream) {
    const pa_status st = check(k_out, v_out, slots, T, k_cache, v_cache, k_scale, v_scale,
                               num_blocks, block_size, Hkv, d, dtype);
    if (st != PA_OK || T == 0) return st;
    unsigned int* err = pa::device_error_word();
    if (!err) return PA_ERR_CUDA;
    const int64_t vecs = (int64_t)T * Hkv * (d / kVec), ctas = (vecs + kThreads - 1) / kThreads;
    if (ctas > INT32_MAX) return PA_ERR_UNSUPPORTED;
    const bool bf16 = dtype == PA_BF16;
    auto kern = d == 128 ? (bf16 ? gather_kernel<true, kInt8, 128> : gather_kernel<false, kInt8, 128>)
                         : (bf16 ? gather_kernel<true, kInt8, 64> : gather_kernel<false, kInt8, 64>);
    kern<<<(unsigned)ctas, kThreads, 0, static_cast<cudaStream_t>(stream)>>>(
        static_cast<const uint32_t*>(k_cache), static_cast<const uint32_t*>(v_cache), k_scale,
        v_scale, slots, vecs, Hkv, shift_of(block_size), (int64_t)num_blocks * block_size,
        static_cast<uint2*>(k_out), static_cast<uint2*>(v_out), err);
    return pa::cuda_status(cudaGetLastError());
}

}  // namespace

extern "C" {

PA_API pa_status pa_reshape_and_cache_int8_block(const void* k_new, const void* v_new,
                                                 const int64_t* slot_mapping, int32_t T,
                                                 void* k_cache, void* v_cache, float* k_scale,
                                                 float* v_scale, int32_t num_blocks,
                                                 int32_t block_size, int32_t Hkv, int32_t d,
                                                 pa_dtype dtype, void* stream) {
    return append<true>(k_new, v_new, slot_mapping, T, k_cache, v_cache, k_scale, v_scale,
                        num_blocks, block_size, Hkv, d, dtype, stream);
}

PA_API pa_status pa_reshape_and_cache_fp8_block(const void* k_new, const void* v_new,
                                                const int64_t* slot_mapping, int32_t T,
                                                void* k_cache, void* v_cache, float* k_scale,
                                                float* v_scale, int32_t num_blocks,
                                                int32_t block_size, int32_t Hkv, int32_t d,
                                                pa_dtype dtype, void* stream) {
    return append<false>(k_new, v_new, slot_mapping, T, k_cache, v_cache, k_scale, v_scale,
                         num_blocks, block_size, Hkv, d, dtype, stream);
}

PA_API pa_status pa_gather_cache_int8_block(const void* k_cache, const void* v_cache,
                                            const float* k_scale, const float* v_scale,
                                            const int64_t* slot_mapping, int32_t T, void* k_out,
                                            void* v_out, int32_t num_blocks, int32_t block_size,
                                            int32_t Hkv, int32_t d, pa_dtype dtype, void* stream) {
    return gather<true>(k_cache, v_cache, k_scale, v_scale, slot_mapping, T, k_out, v_out,
                        num_blocks, block_size, Hkv, d, dtype, stream);
}

PA_API pa_status pa_gather_cache_fp8_block(const void* k_cache, const void* v_cache,
                                           const float* k_scale, const float* v_scale,
                                           const int64_t* slot_mapping, int32_t T, void* k_out,
                                           void* v_out, int32_t num_blocks, int32_t block_size,
                                           int32_t Hkv, int32_t d, pa_dtype dtype, void* stream) {
    return gather<false>(k_cache, v_cache, k_scale, v_scale, slot_mapping, T, k_out, v_out,
                         num_blocks, block_size, Hkv, d, dtype, stream);
}

}  // extern "C"
