// The 4-bit KV cache's append (pa_reshape_and_cache_int4) and the read back of
// the quantised caches (pa_gather_cache_int4 / _int8 / _fp8 / _int8_block / _fp8_block).
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
// fetches in whole cache lines, where the 16-bit cache's order would leave 64-byte
// pieces half a line long.
//
// Both directions are bound by HBM, the append with little to spare: a value costs it
// some ten instructions.  A thread takes K and V of the same place together, and the read
// back four such places where there are enough, as independent chains of dependent loads
// (slot, then codes) that hide each other's latency.
// Measured at d = 128: append of 8192 x 8 rows 12.3 us (33.6 MB in, 9.4 out: 3.5 TB/s;
// issue and its short grid), read back of 32768 x 8 rows 28.9 us (172 MB: 5.9 TB/s),
// append and read back of 64 x 40 rows 4.5 us, all of it latency.
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cstring>

#include "pa.h"
#include "pa_common.cuh"

namespace {

constexpr int kThreads = 128;
constexpr float kF16Max = 65504.f;

// n / d for n < 2^31 by a multiplication (d is the launch's; Granlund and Montgomery's
// round-up method).
struct FastDiv {
    uint32_t mul, shift;
    explicit FastDiv(uint32_t d) {
        shift = 0;
        while ((1ull << shift) < d) ++shift;
        mul = (uint32_t)(((1ull << 32) * ((1ull << shift) - d)) / d + 1);
    }
    __device__ __forceinline__ uint32_t operator()(uint32_t n) const {
        return (__umulhi(n, mul) + n) >> shift;
    }
};

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

constexpr int kAppend = 16;         // values per thread of the append
constexpr int kAppendGroup = 4;     // threads per group of 64 values

// 1 / x, off by at most one unit in the last place.
__device__ __forceinline__ float about_inverse(float x) {
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// Sixteen values of a group of 64 (the other 48 in this lane's three neighbours) ->
// sixteen codes, lowest value in the lowest nibble, and the group's (s, m).
template <bool kBF16>
__device__ __forceinline__ uint2 quantise16(const uint4 (&raw)[2], uint32_t& sm) {
    const uint32_t w[8] = {raw[0].x, raw[0].y, raw[0].z, raw[0].w,
                           raw[1].x, raw[1].y, raw[1].z, raw[1].w};
    uint32_t lo2 = w[0], hi2 = w[0];
#pragma unroll
    for (int i = 1; i < 8; ++i) {
        lo2 = pa::min_x2<kBF16>(lo2, w[i]);
        hi2 = pa::max_x2<kBF16>(hi2, w[i]);
    }
#pragma unroll
    for (int o = 1; o < kAppendGroup; o <<= 1) {
        lo2 = pa::min_x2<kBF16>(lo2, __shfl_xor_sync(0xffffffffu, lo2, o));
        hi2 = pa::max_x2<kBF16>(hi2, __shfl_xor_sync(0xffffffffu, hi2, o));
    }
    const float2 lo = widen2<kBF16>(lo2), hi = widen2<kBF16>(hi2);
    const float least = fminf(lo.x, lo.y), most = fmaxf(hi.x, hi.y);
    // f16 keeps 11 bits of m and s; values beyond its range saturate.
    const __half m16 = __float2half_rn(fminf(fmaxf(least, -kF16Max), kF16Max));
    const __half s16 = __float2half_rn(fminf(__fdiv_rn(__fsub_rn(most, least), 15.f), kF16Max));
    sm = (uint32_t)__half_as_ushort(s16) | ((uint32_t)__half_as_ushort(m16) << 16);
    const float m = __half2float(m16), s = __half2float(s16);
    if (!(s > 0.f)) return make_uint2(0, 0);
    // c = rint((x - m) / s), clamped: (x - m) / (15 s) saturates to [0, 1] at no cost, and
    // 15 times it is rounded by adding 1.5 2^23 (nearest integer, ties to even).  It is
    // within 15 (2^-23 + 3 2^-24) of the quotient (the reciprocal's error and three
    // roundings) and the quotient's own rounding is at most 15 2^-24: together below 6e-6.
    // The few threads with a value within 1e-5 of a tie divide.
    constexpr float kRound = 12582912.f;
    const float inv15 = about_inverse(s) * (1.f / 15.f);
    float off = 0.f;      // largest distance from an integer
    uint32_t c[4];        // four codes each, packed as a sum below 2^16
#pragma unroll
    for (int g = 0; g < 4; ++g) {
        float sum = 0.f;
#pragma unroll
        for (int j = 3; j >= 0; --j) {
            const int i = 4 * g + j;
            const float2 f = widen2<kBF16>(w[i >> 1]);
            const float y = __saturatef(__fmul_rn(__fsub_rn(i & 1 ? f.y : f.x, m), inv15));
            const float z = __fsub_rn(__fmaf_rn(y, 15.f, kRound), kRound);
            off = fmaxf(off, fabsf(__fmaf_rn(y, 15.f, -z)));
            sum = __fmaf_rn(sum, 16.f, z);
        }
        c[g] = __float_as_uint(__fadd_rn(sum, 8388608.f));   // 2^23: the sum in the low bits
    }
    if (off <= 0.49999f)
        return make_uint2(__byte_perm(c[0], c[1], 0x5410), __byte_perm(c[2], c[3], 0x5410));
    uint32_t d[2] = {0, 0};
#pragma unroll
    for (int i = 0; i < kAppend; ++i) {
        const float2 f = widen2<kBF16>(w[i >> 1]);
        const int q = __float2int_rn(__fdiv_rn(__fsub_rn(i & 1 ? f.y : f.x, m), s));
        d[i >> 3] |= (uint32_t)max(0, min(15, q)) << (4 * (i & 7));
    }
    return make_uint2(d[0], d[1]);
}

// Thread v takes values 16 v .. 16 v + 15 of k_new and of v_new.
template <bool kBF16, int D>
__global__ void __launch_bounds__(kThreads)
reshape_and_cache_int4_kernel(const uint4* __restrict__ k_new, const uint4* __restrict__ v_new,
                              const int64_t* __restrict__ slot_mapping, uint32_t vecs,
                              FastDiv by_heads, uint32_t Hkv, int bs_shift,
                              uint2* __restrict__ k_cache, uint2* __restrict__ v_cache,
                              uint32_t* __restrict__ k_scale, uint32_t* __restrict__ v_scale,
                              int64_t num_slots, unsigned int* __restrict__ err) {
    constexpr uint32_t kRow = D / kAppend;     // threads per row
    asm volatile("griddepcontrol.launch_dependents;");   // the decode may be launched: it waits
    const uint32_t v = blockIdx.x * kThreads + threadIdx.x;
    // vecs is a multiple of 4 (a group's threads), so a group is whole or absent; absent
    // threads still take part in the shuffles.
    const bool live = v < vecs;
    const uint32_t row = (live ? v : 0) / kRow, l = v % kRow;
    const uint32_t t = by_heads(row), h = row - t * Hkv;
    const int64_t slot = live ? __ldg(slot_mapping + t) : -1;
    uint4 k[2] = {}, w[2] = {};
    if (live) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            k[i] = __ldg(k_new + 2 * (size_t)v + i);
            w[i] = __ldg(v_new + 2 * (size_t)v + i);
        }
    }
    uint32_t ksm, vsm;
    const uint2 kc = quantise16<kBF16>(k, ksm), vc = quantise16<kBF16>(w, vsm);
    if (slot < 0) return;
    if (slot >= num_slots) {
        if (l == 0) pa::raise_error(err, PA_DEVERR_SLOT);
        return;
    }
    const int64_t tile = (slot >> bs_shift) * Hkv + h;
    const int64_t at = (tile << bs_shift) + (slot & ((1 << bs_shift) - 1));
    k_cache[at * kRow + l] = kc;
    v_cache[at * kRow + l] = vc;
    if (l % kAppendGroup == 0) {
        k_scale[at * (D / 64) + l / kAppendGroup] = ksm;
        v_scale[at * (D / 64) + l / kAppendGroup] = vsm;
    }
}

constexpr int kVec = 8;             // values per piece of the read back: 16 bytes out
constexpr int kGroupLanes = 8;      // pieces per group of 64 values

// Piece u of this thread, of kUnroll: a warp's width apart, so that each instruction of the
// warp moves one contiguous run.
template <int kUnroll>
__device__ __forceinline__ uint32_t piece(int u) {
    return (blockIdx.x * kUnroll * kThreads + (threadIdx.x & ~31u) * kUnroll) + 32 * u + (threadIdx.x & 31);
}

enum Format { kInt4, kInt8, kFp8, kInt8Block, kFp8Block };
template <Format F>
constexpr bool kBlockScaled = F == kInt8Block || F == kFp8Block;

// Eight codes -> the values they stand for, rounded once to 16 bits.
template <bool kBF16, Format F>
__device__ __forceinline__ uint4 dequantise8(uint2 codes, uint32_t sm) {
    float x[8];
    if constexpr (F == kInt4) {
        const float2 f = widen2<false>(sm);
#pragma unroll
        for (int i = 0; i < 8; ++i)   // s c is exact (15 bits): one rounding
            x[i] = fmaf(f.x, (float)((codes.x >> (4 * i)) & 15u), f.y);
    } else {
        const float s = __uint_as_float(sm);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const uint32_t c = i ? codes.y : codes.x;
            uint32_t lo, hi;
            if constexpr (F == kInt8 || F == kInt8Block)
                pa::s8x4_to_f16(c, lo, hi);
            else
                pa::e4m3x4_to_f16(c, lo, hi);
            const float2 a = widen2<false>(lo), b = widen2<false>(hi);
            x[4 * i] = __fmul_rn(a.x, s);
            x[4 * i + 1] = __fmul_rn(a.y, s);
            x[4 * i + 2] = __fmul_rn(b.x, s);
            x[4 * i + 3] = __fmul_rn(b.y, s);
        }
    }
    return make_uint4(pa::pack2<kBF16>(x[0], x[1]), pa::pack2<kBF16>(x[2], x[3]),
                      pa::pack2<kBF16>(x[4], x[5]), pa::pack2<kBF16>(x[6], x[7]));
}

// Piece v is values 8 v .. 8 v + 7 of k_out and of v_out.
template <bool kBF16, Format F, int D, int kUnroll>
__global__ void __launch_bounds__(kThreads)
gather_cache_kernel(const void* k_cache, const void* v_cache, const uint32_t* k_scale,
                    const uint32_t* v_scale, const int64_t* slot_mapping, uint32_t vecs, FastDiv by_heads,
                    uint32_t Hkv, int bs_shift, int64_t num_slots, uint4* k_out, uint4* v_out,
                    unsigned int* err) {
    constexpr uint32_t kRow = D / kVec;
    asm volatile("griddepcontrol.wait;" ::: "memory");   // launched while an append may run
    int64_t slot[kUnroll];
    uint32_t h[kUnroll];
    uint2 kc[kUnroll], vc[kUnroll];
    uint32_t ks[kUnroll], vs[kUnroll];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
        const uint32_t v = piece<kUnroll>(u), row = v / kRow, t = by_heads(row);
        h[u] = row - t * Hkv;
        slot[u] = v < vecs ? pa::ld_behind_wait(slot_mapping + t) : -1;
    }
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
        const uint32_t l = piece<kUnroll>(u) % kRow;
        if (slot[u] >= num_slots) {
            if (l == 0) pa::raise_error(err, PA_DEVERR_SLOT);
            slot[u] = -1;
        }
        if (slot[u] < 0) continue;   // padding: the output row is left as it is
        // (block, head, row) of the scales and of the 4-bit codes; the 8-bit codes
        // are in (slot, head) order, those of the block-scaled cache in (block, head, row) order with
        // a scale per (block, head).
        const int64_t tile = ((slot[u] >> bs_shift) * Hkv) + h[u];
        const int64_t at = (tile << bs_shift) + (slot[u] & ((1 << bs_shift) - 1));
        if constexpr (F == kInt4) {
            kc[u] = make_uint2(pa::ld_behind_wait(static_cast<const uint32_t*>(k_cache) + at * kRow + l), 0);
            vc[u] = make_uint2(pa::ld_behind_wait(static_cast<const uint32_t*>(v_cache) + at * kRow + l), 0);
            ks[u] = pa::ld_behind_wait(k_scale + at * (D / 64) + l / kGroupLanes);
            vs[u] = pa::ld_behind_wait(v_scale + at * (D / 64) + l / kGroupLanes);
        } else {
            const int64_t c = (kBlockScaled<F> ? at : slot[u] * Hkv + h[u]) * kRow + l;
            const int64_t sc = kBlockScaled<F> ? tile : at;
            kc[u] = pa::ld_behind_wait(static_cast<const uint2*>(k_cache) + c);
            vc[u] = pa::ld_behind_wait(static_cast<const uint2*>(v_cache) + c);
            ks[u] = pa::ld_behind_wait(k_scale + sc);
            vs[u] = pa::ld_behind_wait(v_scale + sc);
        }
    }
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
        if (slot[u] < 0) continue;
        k_out[piece<kUnroll>(u)] = dequantise8<kBF16, F>(kc[u], ks[u]);
        v_out[piece<kUnroll>(u)] = dequantise8<kBF16, F>(vc[u], vs[u]);
    }
}

bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

int shift_of(int32_t block_size) {
    return block_size == 8 ? 3 : block_size == 16 ? 4 : block_size == 32 ? 5 : -1;
}

// Checks shared by the append and the read back; *slab receives the tokens of
// one launch (a launch counts its vectors in 32 bits).
pa_status check(const void* k, const void* v, const int64_t* slot_mapping, int32_t T,
                const void* k_cache, const void* v_cache, const void* k_scale, const void* v_scale,
                int32_t num_blocks, int32_t block_size, int32_t Hkv, int32_t d, bool d64,
                pa_dtype dtype, int64_t* slab) {
    if (T < 0 || num_blocks < 0 || Hkv <= 0) return PA_ERR_INVALID;
    if (dtype != PA_F16 && dtype != PA_BF16) return PA_ERR_UNSUPPORTED;
    if (d != 128 && (!d64 || d != 64)) return PA_ERR_UNSUPPORTED;
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

template <bool kBF16, int D>
pa_status append(const void* k_new, const void* v_new, const int64_t* slots, int32_t T_tokens,
                 void* k_cache, void* v_cache, void* k_scale, void* v_scale, int32_t num_blocks,
                 int32_t block_size, int32_t Hkv, int64_t slab, unsigned int* err,
                 cudaStream_t st) {
    const int64_t row = (int64_t)Hkv * (D / kAppend);   // threads per token
    const FastDiv by_heads((uint32_t)Hkv);
    for (int64_t t0 = 0; t0 < T_tokens; t0 += slab) {
        const int64_t n = T_tokens - t0 < slab ? T_tokens - t0 : slab;
        const uint32_t vecs = (uint32_t)(n * row);
        reshape_and_cache_int4_kernel<kBF16, D><<<(vecs + kThreads - 1) / kThreads, kThreads, 0, st>>>(
            static_cast<const uint4*>(k_new) + 2 * t0 * row, static_cast<const uint4*>(v_new) + 2 * t0 * row,
            slots + t0, vecs, by_heads, (uint32_t)Hkv, shift_of(block_size),
            static_cast<uint2*>(k_cache), static_cast<uint2*>(v_cache),
            static_cast<uint32_t*>(k_scale), static_cast<uint32_t*>(v_scale),
            (int64_t)num_blocks * block_size, err);
        if (cudaGetLastError() != cudaSuccess) return PA_ERR_CUDA;
    }
    return PA_OK;
}

template <bool kBF16, Format F, int D>
pa_status gather(const void* k_cache, const void* v_cache, const void* k_scale,
                 const void* v_scale, const int64_t* slots, int32_t T_tokens, void* k_out,
                 void* v_out, int32_t num_blocks, int32_t block_size, int32_t Hkv, int64_t slab,
                 unsigned int* err, cudaStream_t st) {
    const int64_t row = (int64_t)Hkv * (D / kVec);      // pieces per token
    const FastDiv by_heads((uint32_t)Hkv);
    // Four pieces a thread once they fill the SMs' threads all the same, else one: the read
    // back of 32768 x 8 rows took 29.6 us with four and 34.1 us with one, that of 1001 x 4
    // rows 2.4 us with four and 1.9 us with one (28.9 and 1.6 with what came after).
    const int64_t fill = 4ll * 2048 * pa::device_sm_count();
    for (int64_t t0 = 0; t0 < T_tokens; t0 += slab) {
        const int64_t n = T_tokens - t0 < slab ? T_tokens - t0 : slab;
        const uint32_t vecs = (uint32_t)(n * row), per = vecs >= fill ? 4 : 1;
        auto kern = per == 4 ? gather_cache_kernel<kBF16, F, D, 4> : gather_cache_kernel<kBF16, F, D, 1>;
        // Started early, so that its launch hides behind an append's end.
        cudaLaunchAttribute attr{};
        attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr.val.programmaticStreamSerializationAllowed = 1;
        cudaLaunchConfig_t cfg{};
        cfg.gridDim = dim3((vecs + per * kThreads - 1) / (per * kThreads));
        cfg.blockDim = dim3(kThreads);
        cfg.stream = st;
        cfg.attrs = &attr;
        cfg.numAttrs = 1;
        if (cudaLaunchKernelEx(&cfg, kern, k_cache, v_cache, static_cast<const uint32_t*>(k_scale),
                               static_cast<const uint32_t*>(v_scale), slots + t0, vecs, by_heads,
                               (uint32_t)Hkv, shift_of(block_size), (int64_t)num_blocks * block_size,
                               static_cast<uint4*>(k_out) + t0 * row,
                               static_cast<uint4*>(v_out) + t0 * row, err) != cudaSuccess)
            return PA_ERR_CUDA;
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
                               num_blocks, block_size, Hkv, d, F == kInt4 || kBlockScaled<F>, dtype,
                               &slab);
    if (st != PA_OK || T == 0) return st;
    unsigned int* err = pa::device_error_word();
    if (!err) return PA_ERR_CUDA;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if constexpr (F == kInt4 || kBlockScaled<F>)
        if (d == 64)
            return dtype == PA_BF16
                       ? gather<true, F, 64>(k_cache, v_cache, k_scale, v_scale, slots, T,
                                                      k_out, v_out, num_blocks, block_size, Hkv,
                                                      slab, err, s)
                       : gather<false, F, 64>(k_cache, v_cache, k_scale, v_scale, slots, T, k_out,
                                               v_out, num_blocks, block_size, Hkv, slab, err, s);
    return dtype == PA_BF16
               ? gather<true, F, 128>(k_cache, v_cache, k_scale, v_scale, slots, T, k_out,
                                               v_out, num_blocks, block_size, Hkv, slab, err, s)
               : gather<false, F, 128>(k_cache, v_cache, k_scale, v_scale, slots, T, k_out, v_out,
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
                   ? append<true, 64>(k_new, v_new, slot_mapping, T, k_cache, v_cache,
                                               k_scale, v_scale, num_blocks, block_size, Hkv, slab,
                                               err, s)
                   : append<false, 64>(k_new, v_new, slot_mapping, T, k_cache, v_cache, k_scale,
                                        v_scale, num_blocks, block_size, Hkv, slab, err, s);
    return dtype == PA_BF16
               ? append<true, 128>(k_new, v_new, slot_mapping, T, k_cache, v_cache,
                                            k_scale, v_scale, num_blocks, block_size, Hkv, slab,
                                            err, s)
               : append<false, 128>(k_new, v_new, slot_mapping, T, k_cache, v_cache, k_scale,
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

PA_API pa_status pa_gather_cache_int8_block(const void* k_cache, const void* v_cache,
                                            const float* k_scale, const float* v_scale,
                                            const int64_t* slot_mapping, int32_t T, void* k_out,
                                            void* v_out, int32_t num_blocks, int32_t block_size,
                                            int32_t Hkv, int32_t d, pa_dtype dtype, void* stream) {
    return gather_any<kInt8Block>(k_cache, v_cache, k_scale, v_scale, slot_mapping, T, k_out, v_out,
                              num_blocks, block_size, Hkv, d, dtype, stream);
}

PA_API pa_status pa_gather_cache_fp8_block(const void* k_cache, const void* v_cache,
                                           const float* k_scale, const float* v_scale,
                                           const int64_t* slot_mapping, int32_t T, void* k_out,
                                           void* v_out, int32_t num_blocks, int32_t block_size,
                                           int32_t Hkv, int32_t d, pa_dtype dtype, void* stream) {
    return gather_any<kFp8Block>(k_cache, v_cache, k_scale, v_scale, slot_mapping, T, k_out, v_out,
                              num_blocks, block_size, Hkv, d, dtype, stream);
}

}  // extern "C"
