// The 4-bit KV cache's append (pa_reshape_and_cache_int4) and the read back of
// the quantised caches (pa_gather_cache_int4 / _int8 / _fp8).
//
// Format ("LLM推理优化技术地图：从KV Cache到量化与投机解码", section 4.3, KV cache
// quantisation; the page fixes none).  A row is the d values of one (token, KV
// head); each group of 64 values keeps its minimum m and step s as an f16 pair
// and every value as a code c in 0 .. 15 that stands for s c + m:
//     m = f16(min x),  s = f16((max x - min x) / 15),  c = rint((x - m) / s).
// The codes are taken against the rounded m and s, so their rounding costs no
// accuracy of its own.  72 bytes a row of 128 values instead of 256.
// Codes are [num_blocks][Hkv][block_size][d / 2], heads outside rows: a (block,
// KV head) tile is one contiguous run of at least 256 bytes, which the decode
// fetches with one bulk copy, where the 16-bit cache's order would leave 64-byte
// pieces half a cache line long.
//
// Both directions are bound by HBM.  A thread owns eight values (16 bytes of
// the 16-bit side, 4 bytes of codes), so both sides are read and written in
// whole sectors, and takes K and V of the same place together: two independent
// chains hide each other's latency.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cstring>
#include <type_traits>

#include "pa.h"
#include "pa_common.cuh"

namespace {

constexpr int kThreads = 256;
constexpr int kVec = 8;             // values per thread
constexpr int kGroupLanes = 8;      // threads per group of 64 values
constexpr float kF16Max = 65504.f;

template <typename T>
__device__ __forceinline__ float2 to_float2(uint32_t v);
template <>
__device__ __forceinline__ float2 to_float2<__half>(uint32_t v) {
    __half2 h;
    memcpy(&h, &v, 4);
    return __half22float2(h);
}
template <>
__device__ __forceinline__ float2 to_float2<__nv_bfloat16>(uint32_t v) {
    return make_float2(__uint_as_float(v << 16), __uint_as_float(v & 0xFFFF0000u));
}

// Eight values of a group of 64 (the other 56 in this lane's 7 neighbours) ->
// eight codes, lowest value in the lowest nibble, and the group's (s, m).
template <typename T>
__device__ __forceinline__ uint32_t quantise8(uint4 raw, uint32_t& sm) {
    const uint32_t w[4] = {raw.x, raw.y, raw.z, raw.w};
    float x[kVec];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 f = to_float2<T>(w[i]);
        x[2 * i] = f.x;
        x[2 * i + 1] = f.y;
    }
    float lo = x[0], hi = x[0];
#pragma unroll
    for (int i = 1; i < kVec; ++i) {
        lo = fminf(lo, x[i]);
        hi = fmaxf(hi, x[i]);
    }
#pragma unroll
    for (int o = 1; o < kGroupLanes; o <<= 1) {
        lo = fminf(lo, __shfl_xor_sync(0xffffffffu, lo, o));
        hi = fmaxf(hi, __shfl_xor_sync(0xffffffffu, hi, o));
    }
    // f16 keeps 11 bits of m and s; values beyond its range saturate.
    const __half m16 = __float2half_rn(fminf(fmaxf(lo, -kF16Max), kF16Max));
    const __half s16 = __float2half_rn(fminf(__fdiv_rn(__fsub_rn(hi, lo), 15.f), kF16Max));
    sm = (uint32_t)__half_as_ushort(s16) | ((uint32_t)__half_as_ushort(m16) << 16);
    const float m = __half2float(m16), s = __half2float(s16);
    uint32_t codes = 0;
    if (s > 0.f) {
#pragma unroll
        for (int i = 0; i < kVec; ++i) {
            const int c = __float2int_rn(__fdiv_rn(__fsub_rn(x[i], m), s));
            codes |= (uint32_t)max(0, min(15, c)) << (4 * i);
        }
    }
    return codes;
}

// Thread v takes values 8 v .. 8 v + 7 of k_new and of v_new.
template <typename T, int D>
__global__ void __launch_bounds__(kThreads)
reshape_and_cache_int4_kernel(const uint4* __restrict__ k_new, const uint4* __restrict__ v_new,
                              const int64_t* __restrict__ slot_mapping, uint32_t vecs,
                              uint32_t Hkv, int bs_shift, uint32_t* __restrict__ k_cache,
                              uint32_t* __restrict__ v_cache, uint32_t* __restrict__ k_scale,
                              uint32_t* __restrict__ v_scale, int64_t num_slots,
                              unsigned int* __restrict__ err) {
    constexpr uint32_t kRow = D / kVec;        // threads per row
    const uint32_t v = blockIdx.x * kThreads + threadIdx.x;
    // vecs is a multiple of 8 (a group's threads), so a group is whole or
    // absent; absent threads still take part in the shuffles.
    const bool live = v < vecs;
    const uint32_t row = (live ? v : 0) / kRow, l = v % kRow;
    const uint32_t t = row / Hkv, h = row - t * Hkv;
    const int64_t slot = live ? __ldg(slot_mapping + t) : -1;
    uint4 k = make_uint4(0, 0, 0, 0), w = k;
    if (live) {
        k = __ldg(k_new + v);
        w = __ldg(v_new + v);
    }
    uint32_t ksm, vsm;
    const uint32_t kc = quantise8<T>(k, ksm), vc = quantise8<T>(w, vsm);
    if (slot < 0) return;
    if (slot >= num_slots) {
        if (l == 0) pa::raise_error(err, PA_DEVERR_SLOT);
        return;
    }
    const int64_t tile = (slot >> bs_shift) * Hkv + h;
    const int64_t at = (tile << bs_shift) + (slot & ((1 << bs_shift) - 1));
    k_cache[at * kRow + l] = kc;
    v_cache[at * kRow + l] = vc;
    if (l % kGroupLanes == 0) {
        k_scale[at * (D / 64) + l / kGroupLanes] = ksm;
        v_scale[at * (D / 64) + l / kGroupLanes] = vsm;
    }
}

enum Format { kInt4, kInt8, kFp8 };

// Eight codes -> the values they stand for, rounded once to T.
template <typename T, Format F>
__device__ __forceinline__ uint4 dequantise8(uint2 codes, uint32_t sm) {
    float x[kVec];
    if constexpr (F == kInt4) {
        const float2 f = to_float2<__half>(sm);
#pragma unroll
        for (int i = 0; i < kVec; ++i)   // s c is exact (15 bits): one rounding
            x[i] = fmaf(f.x, (float)((codes.x >> (4 * i)) & 15u), f.y);
    } else {
        const float s = __uint_as_float(sm);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const uint32_t c = i ? codes.y : codes.x;
            uint32_t lo, hi;
            if constexpr (F == kInt8)
                pa::s8x4_to_f16(c, lo, hi);
            else
                pa::e4m3x4_to_f16(c, lo, hi);
            const float2 a = to_float2<__half>(lo), b = to_float2<__half>(hi);
            x[4 * i] = __fmul_rn(a.x, s);
            x[4 * i + 1] = __fmul_rn(a.y, s);
            x[4 * i + 2] = __fmul_rn(b.x, s);
            x[4 * i + 3] = __fmul_rn(b.y, s);
        }
    }
    constexpr bool kB = sizeof(T) == 2 && !std::is_same<T, __half>::value;
    return make_uint4(pa::pack2<kB>(x[0], x[1]), pa::pack2<kB>(x[2], x[3]),
                      pa::pack2<kB>(x[4], x[5]), pa::pack2<kB>(x[6], x[7]));
}

// Thread v writes values 8 v .. 8 v + 7 of k_out and of v_out.
template <typename T, Format F, int D>
__global__ void __launch_bounds__(kThreads)
gather_cache_kernel(const void* __restrict__ k_cache, const void* __restrict__ v_cache,
                    const uint32_t* __restrict__ k_scale, const uint32_t* __restrict__ v_scale,
                    const int64_t* __restrict__ slot_mapping, uint32_t vecs, uint32_t Hkv,
                    int bs_shift, int64_t num_slots, uint4* __restrict__ k_out,
                    uint4* __restrict__ v_out, unsigned int* __restrict__ err) {
    constexpr uint32_t kRow = D / kVec;
    const uint32_t v = blockIdx.x * kThreads + threadIdx.x;
    if (v >= vecs) return;
    const uint32_t row = v / kRow, l = v % kRow;
    const uint32_t t = row / Hkv, h = row - t * Hkv;
    const int64_t slot = __ldg(slot_mapping + t);
    if (slot < 0) return;   // padding: the output row is left as it is
    if (slot >= num_slots) {
        if (l == 0) pa::raise_error(err, PA_DEVERR_SLOT);
        return;
    }
    // (block, head, row) of the scales and of the 4-bit codes; the 8-bit codes
    // are in (slot, head) order.
    const int64_t at = ((((slot >> bs_shift) * Hkv) + h) << bs_shift) +
                       (slot & ((1 << bs_shift) - 1));
    uint2 kc, vc;
    uint32_t ks, vs;
    if constexpr (F == kInt4) {
        kc = make_uint2(__ldg(static_cast<const uint32_t*>(k_cache) + at * kRow + l), 0);
        vc = make_uint2(__ldg(static_cast<const uint32_t*>(v_cache) + at * kRow + l), 0);
        ks = __ldg(k_scale + at * (D / 64) + l / kGroupLanes);
        vs = __ldg(v_scale + at * (D / 64) + l / kGroupLanes);
    } else {
        const int64_t c = (slot * Hkv + h) * kRow + l;
        kc = __ldg(static_cast<const uint2*>(k_cache) + c);
        vc = __ldg(static_cast<const uint2*>(v_cache) + c);
        ks = __ldg(k_scale + at);
        vs = __ldg(v_scale + at);
    }
    k_out[v] = dequantise8<T, F>(kc, ks);
    v_out[v] = dequantise8<T, F>(vc, vs);
}

bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

int shift_of(int32_t block_size) {
    return block_size == 8 ? 3 : block_size == 16 ? 4 : block_size == 32 ? 5 : -1;
}

// Checks shared by the append and the read back; *slab receives the tokens of
// one launch (a launch counts its vectors in 32 bits).
pa_status check(const void* k, const void* v, const int64_t* slot_mapping, int32_t T,
                const void* k_cache, const void* v_cache, const void* k_scale, const void* v_scale,
                int32_t num_blocks, int32_t block_size, int32_t Hkv, int32_t d, bool int4,
                pa_dtype dtype, int64_t* slab) {
    if (T < 0 || num_blocks < 0 || Hkv <= 0) return PA_ERR_INVALID;
    if (dtype != PA_F16 && dtype != PA_BF16) return PA_ERR_UNSUPPORTED;
    if (d != 128 && (!int4 || d != 64)) return PA_ERR_UNSUPPORTED;
    if (shift_of(block_size) < 0) return PA_ERR_UNSUPPORTED;
    if (Hkv > (1 << 20)) return PA_ERR_UNSUPPORTED;
    *slab = ((int64_t)1 << 30) / ((int64_t)Hkv * (d / kVec));
    if (T == 0) return PA_OK;
    if (!k || !v || !slot_mapping || !k_cache || !v_cache || !k_scale || !v_scale)
        return PA_ERR_INVALID;
    if (!aligned(k, 16) || !aligned(v, 16) || !aligned(k_cache, 16) || !aligned(v_cache, 16) ||
        !aligned(k_scale, 4) || !aligned(v_scale, 4) || !aligned(slot_mapping, 8))
        return PA_ERR_INVALID;
    return PA_OK;
}

template <typename T, int D>
pa_status append(const void* k_new, const void* v_new, const int64_t* slots, int32_t T_tokens,
                 void* k_cache, void* v_cache, void* k_scale, void* v_scale, int32_t num_blocks,
                 int32_t block_size, int32_t Hkv, int64_t slab, unsigned int* err,
                 cudaStream_t st) {
    const int64_t row = (int64_t)Hkv * (D / kVec);
    for (int64_t t0 = 0; t0 < T_tokens; t0 += slab) {
        const int64_t n = T_tokens - t0 < slab ? T_tokens - t0 : slab;
        const uint32_t vecs = (uint32_t)(n * row);
        reshape_and_cache_int4_kernel<T, D><<<(vecs + kThreads - 1) / kThreads, kThreads, 0, st>>>(
            static_cast<const uint4*>(k_new) + t0 * row, static_cast<const uint4*>(v_new) + t0 * row,
            slots + t0, vecs, (uint32_t)Hkv, shift_of(block_size), static_cast<uint32_t*>(k_cache),
            static_cast<uint32_t*>(v_cache), static_cast<uint32_t*>(k_scale),
            static_cast<uint32_t*>(v_scale), (int64_t)num_blocks * block_size, err);
        if (cudaGetLastError() != cudaSuccess) return PA_ERR_CUDA;
    }
    return PA_OK;
}

template <typename T, Format F, int D>
pa_status gather(const void* k_cache, const void* v_cache, const void* k_scale,
                 const void* v_scale, const int64_t* slots, int32_t T_tokens, void* k_out,
                 void* v_out, int32_t num_blocks, int32_t block_size, int32_t Hkv, int64_t slab,
                 unsigned int* err, cudaStream_t st) {
    const int64_t row = (int64_t)Hkv * (D / kVec);
    for (int64_t t0 = 0; t0 < T_tokens; t0 += slab) {
        const int64_t n = T_tokens - t0 < slab ? T_tokens - t0 : slab;
        const uint32_t vecs = (uint32_t)(n * row);
        gather_cache_kernel<T, F, D><<<(vecs + kThreads - 1) / kThreads, kThreads, 0, st>>>(
            k_cache, v_cache, static_cast<const uint32_t*>(k_scale),
            static_cast<const uint32_t*>(v_scale), slots + t0, vecs, (uint32_t)Hkv,
            shift_of(block_size), (int64_t)num_blocks * block_size,
            static_cast<uint4*>(k_out) + t0 * row, static_cast<uint4*>(v_out) + t0 * row, err);
        if (cudaGetLastError() != cudaSuccess) return PA_ERR_CUDA;
    }
    return PA_OK;
}

template <Format F>
pa_status gather_any(const void* k_cache, const void* v_cache, const void* k_scale,
                     const void* v_scale, const int64_t* slots, int32_t T, void* k_out,
                     void* v_out, int32_t num_blocks, int32_t block_size, int32_t Hkv, int32_t d,
                     pa_dtype dtype, void* stream) {
    int64_t slab = 0;
    const pa_status st = check(k_out, v_out, slots, T, k_cache, v_cache, k_scale, v_scale,
                               num_blocks, block_size, Hkv, d, F == kInt4, dtype, &slab);
    if (st != PA_OK || T == 0) return st;
    unsigned int* err = pa::device_error_word();
    if (!err) return PA_ERR_CUDA;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if constexpr (F == kInt4)
        if (d == 64)
            return dtype == PA_BF16
                       ? gather<__nv_bfloat16, F, 64>(k_cache, v_cache, k_scale, v_scale, slots, T,
                                                      k_out, v_out, num_blocks, block_size, Hkv,
                                                      slab, err, s)
                       : gather<__half, F, 64>(k_cache, v_cache, k_scale, v_scale, slots, T, k_out,
                                               v_out, num_blocks, block_size, Hkv, slab, err, s);
    return dtype == PA_BF16
               ? gather<__nv_bfloat16, F, 128>(k_cache, v_cache, k_scale, v_scale, slots, T, k_out,
                                               v_out, num_blocks, block_size, Hkv, slab, err, s)
               : gather<__half, F, 128>(k_cache, v_cache, k_scale, v_scale, slots, T, k_out, v_out,
                                        num_blocks, block_size, Hkv, slab, err, s);
}

}  // namespace

extern "C" {

PA_API pa_status pa_reshape_and_cache_int4(const void* k_new, const void* v_new,
                                           const int64_t* slot_mapping, int32_t T, void* k_cache,
                                           void* v_cache, void* k_scale, void* v_scale,
                                           int32_t num_blocks, int32_t block_size, int32_t Hkv,
                                           int32_t d, pa_dtype dtype, void* stream) {
    int64_t slab = 0;
    const pa_status st = check(k_new, v_new, slot_mapping, T, k_cache, v_cache, k_scale, v_scale,
                               num_blocks, block_size, Hkv, d, true, dtype, &slab);
    if (st != PA_OK || T == 0) return st;
    unsigned int* err = pa::device_error_word();
    if (!err) return PA_ERR_CUDA;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (d == 64)
        return dtype == PA_BF16
                   ? append<__nv_bfloat16, 64>(k_new, v_new, slot_mapping, T, k_cache, v_cache,
                                               k_scale, v_scale, num_blocks, block_size, Hkv, slab,
                                               err, s)
                   : append<__half, 64>(k_new, v_new, slot_mapping, T, k_cache, v_cache, k_scale,
                                        v_scale, num_blocks, block_size, Hkv, slab, err, s);
    return dtype == PA_BF16
               ? append<__nv_bfloat16, 128>(k_new, v_new, slot_mapping, T, k_cache, v_cache,
                                            k_scale, v_scale, num_blocks, block_size, Hkv, slab,
                                            err, s)
               : append<__half, 128>(k_new, v_new, slot_mapping, T, k_cache, v_cache, k_scale,
                                     v_scale, num_blocks, block_size, Hkv, slab, err, s);
}

PA_API pa_status pa_gather_cache_int4(const void* k_cache, const void* v_cache,
                                      const void* k_scale, const void* v_scale,
                                      const int64_t* slot_mapping, int32_t T, void* k_out,
                                      void* v_out, int32_t num_blocks, int32_t block_size,
                                      int32_t Hkv, int32_t d, pa_dtype dtype, void* stream) {
    return gather_any<kInt4>(k_cache, v_cache, k_scale, v_scale, slot_mapping, T, k_out, v_out,
                             num_blocks, block_size, Hkv, d, dtype, stream);
}

PA_API pa_status pa_gather_cache_int8(const void* k_cache, const void* v_cache,
                                      const float* k_scale, const float* v_scale,
                                      const int64_t* slot_mapping, int32_t T, void* k_out,
                                      void* v_out, int32_t num_blocks, int32_t block_size,
                                      int32_t Hkv, int32_t d, pa_dtype dtype, void* stream) {
    return gather_any<kInt8>(k_cache, v_cache, k_scale, v_scale, slot_mapping, T, k_out, v_out,
                             num_blocks, block_size, Hkv, d, dtype, stream);
}

PA_API pa_status pa_gather_cache_fp8(const void* k_cache, const void* v_cache,
                                     const float* k_scale, const float* v_scale,
                                     const int64_t* slot_mapping, int32_t T, void* k_out,
                                     void* v_out, int32_t num_blocks, int32_t block_size,
                                     int32_t Hkv, int32_t d, pa_dtype dtype, void* stream) {
    return gather_any<kFp8>(k_cache, v_cache, k_scale, v_scale, slot_mapping, T, k_out, v_out,
                            num_blocks, block_size, Hkv, d, dtype, stream);
}

}  // extern "C"
