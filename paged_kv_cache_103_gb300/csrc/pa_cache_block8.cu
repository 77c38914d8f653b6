// The block-scaled 8-bit KV cache's append (pa_reshape_and_cache_int8_block / _fp8_block).
// Its read back is with those of the other quantised caches (pa_cache_int4.cu).
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
// The maximum is over the block's tokens in the call, so the tile is the unit of work: the
// first token of a block leads it, its warp finds the others, reads their rows once into
// registers, and writes the block's codes and scale.  Nothing is left for another launch, and
// no two warps meet.
//
// What bounds it: in a prompt HBM (3 bytes a value) and issue slots (some seven instructions
// a value, 68 % of them taken) in a launch that is over before either is full; in a decode step
// a chain of dependent loads (slots, rows and scale, earlier codes where the scale grows).
// Measured at d = 128 (device time): 8192 x 8 rows, bf16, E4M3 15.1 us (50 MB: 3.3 TB/s), 32768 x 8
// rows INT8 44.5 (201 MB: 4.5 TB/s), 64 x 40 rows of as many blocks, f16, INT8 5.3 (15.3 where every scale
// grows and the blocks' other 15 rows are coded again), one token 2.6.
// Rows that are neighbours in the call and in the block, as they nearly always are, have places
// by addition, and the divisions that an odd scale needs are out of the way of the others: with each
// row's place from its bit and both ways to a code in every step it was 16.2, 53.0, 6.5 and 3.1.
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

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kVec = 4;      // values of a lane
constexpr int kWindow = 8;   // tokens of a CTA

// x / s for one s, correctly rounded without a division each: with y = 1 / s correctly rounded and q
// = x y, q + (x - q s) y rounds to the quotient (Markstein, IBM J. Res. Dev. 34, 1990), unless
// s's fraction is all ones or x - q s loses bits below the smallest float, which a quotient
// of 2^-11 or more (smaller ones are codes of 0 either way) does not for s >= 2^-90.
struct Divider {
    float s, y;
    bool fast;
    __device__ explicit Divider(float s_) : s(s_), y(0.f), fast(false) {
        if (s > 0.f) {
            fast = s >= 8.0779356694631609e-28f && (__float_as_uint(s) & 0x7FFFFFu) != 0x7FFFFFu;   // 2^-90
            if (fast) y = __frcp_rn(s);
        }
    }
    __device__ __forceinline__ float operator()(float x) const {
        const float q = __fmul_rn(x, y);
        return __fmaf_rn(__fmaf_rn(-q, s, x), y, q);
    }
};

// Four values' codes by a Divider that is fast.  |x| <= TOP s (1 + 2^-24): INT8 codes need no clamp.
template <bool kBF16, bool kInt8>
__device__ __forceinline__ uint32_t codes_fast(uint2 w, const Divider& by) {
    const float2 p = widen2<kBF16>(w.x), q = widen2<kBF16>(w.y);
    if constexpr (kInt8) {
        // 1.5 2^23 more, an fp32 number's low byte is the nearest integer's (ties to even)
        constexpr float kRound = 12582912.f;
        auto one = [&](float x) { return __float_as_uint(__fadd_rn(by(x), kRound)); };
        const uint32_t lo = __byte_perm(one(p.x), one(p.y), 0x0040), hi = __byte_perm(one(q.x), one(q.y), 0x0040);
        return __byte_perm(lo, hi, 0x5410);
    } else {
        return code4<false>(by(p.x), by(p.y), by(q.x), by(q.y));
    }
}

// The same by divisions, for any s >= 0; zeros for 0.
template <bool kBF16, bool kInt8>
__device__ __forceinline__ uint32_t codes_divided(uint2 w, float s) {
    const float2 p = widen2<kBF16>(w.x), q = widen2<kBF16>(w.y);
    if (!(s > 0.f)) return 0u;
    return code4<kInt8>(__fdiv_rn(p.x, s), __fdiv_rn(p.y, s), __fdiv_rn(q.x, s), __fdiv_rn(q.y, s));
}

struct AppendParams {
    const uint2 *k_new, *v_new;
    const int64_t* slots;
    uint32_t *k_cache, *v_cache;
    float *k_scale, *v_scale;
    unsigned int* err;
    int64_t num_slots;
    int32_t T, Hkv, groups, per;   // a CTA takes `per` of the 2 Hkv (KV head, K or V) tiles, one of `groups`
};

// A CTA has kWindow tokens and some (KV head, K or V) pairs.  A token that is the first of its
// block in the call leads the block's tokens, wherever they end; each (leader, pair) is a
// warp's: a tile of at most kRows rows, read once into registers, 8 bytes a lane.
template <bool kBF16, bool kInt8, int D, int kShift>
__global__ void __launch_bounds__(kThreads) append_kernel(const AppendParams p) {
    constexpr int kLanes = D / kVec, kPer = 32 / kLanes;   // lanes of a row, rows of an instruction
    constexpr int kRows = 1 << kShift, kSteps = kRows / kPer;
    constexpr float kTop = kInt8 ? 127.f : 448.f;
    asm volatile("griddepcontrol.launch_dependents;");   // what reads the cache may be launched: it waits
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, l = lane % kLanes, sub = lane / kLanes;
    const int32_t window = blockIdx.x / p.groups, group = blockIdx.x - window * p.groups;
    const int32_t t0 = window * kWindow, T = p.T;
    auto slot_at = [&](int32_t t) {   // -1: padding, or outside the pool
        const int64_t s = t >= 0 && t < T ? __ldg(p.slots + t) : -1;
        return s < p.num_slots ? s : -1;
    };
    // The nearest written token before `t` (step -1: t - 1, t - 2, ..) or from t on (step 1), as a
    // slot; -1: none.  512 entries at a time: a padded batch has thousands between two sequences.
    auto nearest = [&](int32_t t, int step) {
        constexpr int kWide = 16;
        for (int32_t at = step < 0 ? t - 1 - lane : t + lane; step < 0 ? at + lane >= 0 : at - lane < T;
             at += step * 32 * kWide) {
            int64_t s[kWide];
#pragma unroll
            for (int q = 0; q < kWide; ++q) s[q] = slot_at(at + step * 32 * q);
#pragma unroll
            for (int q = 0; q < kWide; ++q) {
                const uint32_t some = __ballot_sync(0xffffffffu, s[q] >= 0);
                if (some) return __shfl_sync(0xffffffffu, s[q], __ffs(some) - 1);
            }
        }
        return (int64_t)-1;
    };
    // ---- leaders: the nearest written token before has another block
    const int64_t mine = lane < kWindow ? slot_at(t0 + lane) : -1;
    const int64_t before = slot_at(t0 - 32 + lane);
    if (group == 0 && warp == 0 && lane < kWindow && t0 + lane < T && __ldg(p.slots + t0 + lane) >= p.num_slots)
        pa::raise_error(p.err, PA_DEVERR_SLOT);
    const uint32_t live = __ballot_sync(0xffffffffu, mine >= 0);
    if (!live) return;
    const uint32_t some = __ballot_sync(0xffffffffu, before >= 0);
    const int64_t last = some ? __shfl_sync(0xffffffffu, before, 31 - __clz(some)) : nearest(t0 - 32, -1);
    const uint32_t lower = live & ((1u << lane) - 1);
    const int64_t prev = __shfl_sync(0xffffffffu, mine, lower ? 31 - __clz(lower) : 0);
    const int64_t prev_block = (lower ? prev : last) >> kShift;   // -1: none
    const uint32_t leaders = __ballot_sync(0xffffffffu, mine >= 0 && prev_block != mine >> kShift);
    const int32_t hv0 = group * p.per, tiles = min(p.per, 2 * p.Hkv - hv0);
    const int items = __popc(leaders) * tiles;
#pragma unroll 1
    for (int it = warp; it < items; it += kWarps) {
        const int lead = it / tiles;
        const int32_t hv = hv0 + it - lead * tiles, h = hv >> 1;
        uint32_t m = leaders;
        for (int x = 0; x < lead; ++x) m &= m - 1;
        const int32_t t = t0 + __ffs(m) - 1;
        const int64_t block = __shfl_sync(0xffffffffu, mine, __ffs(m) - 1) >> kShift;
        const uint2* x = (hv & 1 ? p.v_new : p.k_new) + l;
        uint32_t* cache = (hv & 1 ? p.v_cache : p.k_cache) + ((block * p.Hkv + h) << kShift) * kLanes + l;
        float* scale = (hv & 1 ? p.v_scale : p.k_scale) + block * p.Hkv + h;
        const float was = *scale;
        // ---- the block's tokens among 32 from the leader on
        const int64_t s = slot_at(t + lane);
        const uint32_t any = __ballot_sync(0xffffffffu, s >= 0);
        const uint32_t same = __ballot_sync(0xffffffffu, s >= 0 && s >> kShift == block);
        const uint32_t other = any & ~same;
        uint32_t run = other ? same & ((other & -other) - 1) : same;
        const int32_t r_lane = (int32_t)(s & (kRows - 1));
        if (other || t + 32 >= T || __popc(run) >= kRows || nearest(t + 32, 1) >> kShift != block) {
            // These are all of them.  (A slot named twice would make more: those are left out.)
            const int count = min(__popc(run), kRows), r0 = __shfl_sync(0xffffffffu, r_lane, 0);
            const bool in_run = run >> lane & 1;
            const uint32_t written = __reduce_or_sync(0xffffffffu, in_run ? 1u << r_lane : 0u);
            // As a rule they are neighbours in the call and in the block.
            const bool plain = !(run & (run + 1)) && __all_sync(0xffffffffu, !in_run || r_lane == r0 + lane);
            // f(step, token from t on, row) for this lane's row of each step that has one
            auto rows_of = [&](auto f) {
                if (plain) {
#pragma unroll
                    for (int q = 0; q < kSteps; ++q)
                        if (q * kPer + sub < count) f(q, q * kPer + sub, r0 + q * kPer + sub);
                } else {
                    uint32_t todo = run;
#pragma unroll
                    for (int q = 0; q < kSteps; ++q) {
                        const int a = __ffs(todo) - 1;
                        todo &= todo - 1;
                        int from = a;
                        if constexpr (kPer == 2) {
                            const int b = __ffs(todo) - 1;
                            todo &= todo - 1;
                            from = sub ? b : a;
                        }
                        const int r = __shfl_sync(0xffffffffu, r_lane, from & 31);
                        if (from >= 0) f(q, from, r);
                    }
                }
            };
            const uint2* mine_x = x + ((int64_t)t * p.Hkv + h) * kLanes;
            const int64_t stride = (int64_t)p.Hkv * kLanes;
            uint2 w[kSteps];
#pragma unroll
            for (int q = 0; q < kSteps; ++q) w[q] = make_uint2(0, 0);
            rows_of([&](int q, int from, int) { w[q] = __ldg(mine_x + from * stride); });
            uint32_t top2 = 0;
#pragma unroll
            for (int q = 0; q < kSteps; ++q) {
                top2 = pa::max_x2<kBF16>(top2, w[q].x & 0x7FFF7FFFu);
                top2 = pa::max_x2<kBF16>(top2, w[q].y & 0x7FFF7FFFu);
            }
            const float2 top = widen2<kBF16>(top2);
            const float a = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(fmaxf(top.x, top.y))));
            const float base = written & 1 ? 0.f : was, now = fmaxf(base, __fdiv_rn(a, kTop));
            if (base > 0.f && base < now) {
                const float ratio = __fdiv_rn(base, now);
#pragma unroll 4
                for (int r = sub; r < kRows; r += kPer) {
                    if (written >> r & 1) continue;
                    const float4 c = number4<kInt8>(cache[r * kLanes]);
                    cache[r * kLanes] = code4<kInt8>(__fmul_rn(c.x, ratio), __fmul_rn(c.y, ratio),
                                                     __fmul_rn(c.z, ratio), __fmul_rn(c.w, ratio));
                }
            }
            const Divider by(now);
            if (by.fast) {
                rows_of([&](int q, int, int r) { cache[r * kLanes] = codes_fast<kBF16, kInt8>(w[q], by); });
            } else {
#pragma unroll 1
                for (uint32_t todo = run; todo; todo &= todo - 1) {
                    const int from = __ffs(todo) - 1, r = __shfl_sync(0xffffffffu, r_lane, from);
                    if (sub == 0) cache[r * kLanes] = codes_divided<kBF16, kInt8>(__ldg(mine_x + from * stride), now);
                }
            }
            if (lane == 0) *scale = now;
            continue;
        }
        // ---- padding between them: row by row, twice
        auto each = [&](auto f) {   // f(row of the block, token)
            for (int32_t first = t; first < T; first += 32) {
                const int64_t sl = slot_at(first + lane);
                const uint32_t all = __ballot_sync(0xffffffffu, sl >= 0);
                const uint32_t ours = __ballot_sync(0xffffffffu, sl >= 0 && sl >> kShift == block);
                const uint32_t end = all & ~ours;
                for (uint32_t y = end ? ours & ((end & -end) - 1) : ours; y; y &= y - 1) {
                    const int at = __ffs(y) - 1;
                    f((int32_t)(__shfl_sync(0xffffffffu, sl, at) & (kRows - 1)), first + at);
                }
                if (end) break;
            }
        };
        auto row = [&](int32_t j) {
            return sub == 0 ? __ldg(x + ((int64_t)j * p.Hkv + h) * kLanes) : make_uint2(0, 0);
        };
        uint32_t written = 0, top2 = 0;
        each([&](int32_t r, int32_t j) {
            const uint2 y = row(j);
            written |= 1u << r;
            top2 = pa::max_x2<kBF16>(top2, pa::max_x2<kBF16>(y.x & 0x7FFF7FFFu, y.y & 0x7FFF7FFFu));
        });
        const float2 top = widen2<kBF16>(top2);
        const float a = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(fmaxf(top.x, top.y))));
        const float base = written & 1 ? 0.f : was, now = fmaxf(base, __fdiv_rn(a, kTop));
        if (base > 0.f && base < now) {
            const float ratio = __fdiv_rn(base, now);
            for (int r = sub; r < kRows; r += kPer) {
                if (written >> r & 1) continue;
                const float4 c = number4<kInt8>(cache[r * kLanes]);
                cache[r * kLanes] = code4<kInt8>(__fmul_rn(c.x, ratio), __fmul_rn(c.y, ratio),
                                                 __fmul_rn(c.z, ratio), __fmul_rn(c.w, ratio));
            }
        }
        each([&](int32_t r, int32_t j) {
            if (sub == 0) cache[r * kLanes] = codes_divided<kBF16, kInt8>(row(j), now);
        });
        if (lane == 0) *scale = now;
    }
}

bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

template <bool kInt8, int D, int kShift>
pa_status launch(const AppendParams& p, bool bf16, cudaStream_t stream) {
    auto kern = bf16 ? append_kernel<true, kInt8, D, kShift> : append_kernel<false, kInt8, D, kShift>;
    const int64_t ctas = ((int64_t)p.T + kWindow - 1) / kWindow * p.groups;
    if (ctas > INT32_MAX) return PA_ERR_UNSUPPORTED;
    kern<<<(unsigned)ctas, kThreads, 0, stream>>>(p);
    return pa::cuda_status(cudaGetLastError());
}

template <bool kInt8>
pa_status append(const void* k_new, const void* v_new, const int64_t* slots, int32_t T,
                 void* k_cache, void* v_cache, float* k_scale, float* v_scale, int32_t num_blocks,
                 int32_t block_size, int32_t Hkv, int32_t d, pa_dtype dtype, void* stream) {
    if (T < 0 || num_blocks < 0 || Hkv <= 0) return PA_ERR_INVALID;
    if (dtype != PA_F16 && dtype != PA_BF16) return PA_ERR_UNSUPPORTED;
    if (d != 64 && d != 128) return PA_ERR_UNSUPPORTED;
    if (block_size != 8 && block_size != 16 && block_size != 32) return PA_ERR_UNSUPPORTED;
    if (Hkv > (1 << 20)) return PA_ERR_UNSUPPORTED;
    if (T == 0) return PA_OK;
    if (!k_new || !v_new || !slots || !k_cache || !v_cache || !k_scale || !v_scale) return PA_ERR_INVALID;
    if (!aligned(k_new, 16) || !aligned(v_new, 16) || !aligned(k_cache, 16) || !aligned(v_cache, 16) ||
        !aligned(k_scale, 4) || !aligned(v_scale, 4) || !aligned(slots, 8))
        return PA_ERR_INVALID;
    AppendParams p{static_cast<const uint2*>(k_new), static_cast<const uint2*>(v_new), slots,
                   static_cast<uint32_t*>(k_cache), static_cast<uint32_t*>(v_cache), k_scale, v_scale,
                   pa::device_error_word(), (int64_t)num_blocks * block_size, T, Hkv, 0, 16};
    const int sms = pa::device_sm_count();
    if (!p.err || !sms) return PA_ERR_CUDA;
    // A prompt's window has a leader or none, a decode step's eight: two tiles a warp for the former
    // where that leaves four CTAs an SM (32768 x 8 rows 44.5 us, one tile 51.8), fewer where it does
    // not.
    const int64_t windows = ((int64_t)T + kWindow - 1) / kWindow;
    for (; p.per > 1 && windows * ((2 * Hkv + p.per - 1) / p.per) < 4 * sms; p.per /= 2) {}
    p.groups = (2 * Hkv + p.per - 1) / p.per;
    const bool bf16 = dtype == PA_BF16;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (d == 128)
        return block_size == 8    ? launch<kInt8, 128, 3>(p, bf16, st)
               : block_size == 16 ? launch<kInt8, 128, 4>(p, bf16, st)
                                  : launch<kInt8, 128, 5>(p, bf16, st);
    return block_size == 8    ? launch<kInt8, 64, 3>(p, bf16, st)
           : block_size == 16 ? launch<kInt8, 64, 4>(p, bf16, st)
                              : launch<kInt8, 64, 5>(p, bf16, st);
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

}  // extern "C"
