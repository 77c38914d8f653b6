// Eviction by accumulated attention weight: the choice of the tokens that stay
// (pa_select_tokens) and the move that puts them together (pa_compact_tokens).  The pages
// have no counterpart; what they do with a full pool is swap and preemption ("LLM推理优化：
// vLLM PagedAttention深度解析与工程实践", section 3.2).
#include <cuda_runtime.h>

#include <cmath>

#include "pa.h"
#include "pa_common.cuh"

namespace {

// ---- pa_select_tokens ------------------------------------------------------------
// Of the m = n - first - last tokens between, the k = keep - first - last with the largest
// weights, ties to the lower position.  One CTA per (sequence, KV head): the weights' order
// as unsigned keys, the range of the keys in 1024 bins whose counts from the top name the
// bin of the k-th largest, which is cut again until it is one key wide or wanted whole; then the
// chosen positions in order.
struct ChooseParams {
    const float* weights;
    float* new_weights;
    const int32_t *rows, *context_lens;
    int32_t *kept, *kept_lens;
    unsigned int* err;
    int32_t num_rows, width, Hkv, keep, first, last;
};

// Unsigned numbers that order like the floats; -0 as 0, a NaN below every number.
__device__ __forceinline__ uint32_t ordered(float x) {
    const uint32_t u = __float_as_uint(x + 0.f);
    return isnan(x) ? 0u : u ^ (u >> 31 ? 0xffffffffu : 0x80000000u);
}

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kBinBits = 10, kBins = 1 << kBinBits;   // four bins a thread

__global__ void __launch_bounds__(kThreads) select_tokens_kernel(const ChooseParams p) {
    __shared__ __align__(16) uint32_t hist[kBins];
    __shared__ uint32_t s_top[kWarps], s_low[kWarps], wsum[kWarps], wsum2[kWarps];
    __shared__ uint32_t s_bin, s_rank, s_count;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int32_t g = blockIdx.x, i = blockIdx.y;
    int32_t* kept = p.kept + ((int64_t)i * p.Hkv + g) * p.keep;
    const int32_t row = p.rows[i], raw = p.context_lens[i];
    const bool part = row >= 0 && row < p.num_rows;
    if (tid == 0 && g == 0) {
        if (row >= p.num_rows) pa::raise_error(p.err, PA_DEVERR_SLOT);
        if (raw < 0) pa::raise_error(p.err, PA_DEVERR_CONTEXT);
        if (part && raw > p.width) pa::raise_error(p.err, PA_DEVERR_TABLE_WIDTH);
    }
    const int32_t n = part ? max(0, min(raw, p.width)) : 0, count = min(n, p.keep);
    if (tid == 0 && g == 0) p.kept_lens[i] = count;
    for (int32_t j = count + tid; j < p.keep; j += kThreads) kept[j] = -1;
    if (!part) return;
    const float* w = p.weights + ((int64_t)row * p.Hkv + g) * p.width;
    const int32_t k = p.keep - p.first - p.last, m = n - p.first - p.last;   // k < m where tokens go
    const int32_t head = n <= p.keep ? n : p.first;
    for (int32_t j = tid; j < head; j += kThreads) kept[j] = j;
    if (n > p.keep) {
        for (int32_t j = tid; j < p.last; j += kThreads) kept[p.keep - p.last + j] = n - p.last + j;
        for (int b = tid; b < kBins; b += kThreads) hist[b] = 0;
    }
    if (n > p.keep && k > 0) {
        const int32_t per = (m + kThreads - 1) / kThreads;
        const int32_t beg = min(m, tid * per), end = min(m, beg + per);
        auto each = [&](auto f) {   // f(key, place) for each key of this thread's stretch
            for (int32_t j = beg; j < end; ++j) f(ordered(w[p.first + j]), j);
        };
        uint32_t top = 0, low = 0;    // the largest key, and the smallest's complement
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
        top = __reduce_max_sync(0xffffffffu, s_top[lane % kWarps]);
        uint32_t base = ~__reduce_max_sync(0xffffffffu, s_low[lane % kWarps]);
        int width = 32 - __clz(top - base);            // bits of the range; 0: all keys are equal
        int shift = max(0, width - kBinBits);
        uint32_t rank = (uint32_t)k, limit, ties;      // chosen: keys above limit, and `ties` equal ones
        for (;;) {
            each([&](uint32_t x, int) {
                x -= base;                             // keys below base wrap to large numbers
                if (width == 32 || (x >> width) == 0) atomicAdd(&hist[x >> shift], 1u);
            });
            __syncthreads();
            // Counts from the top: thread t owns bins 4 t' .. 4 t' + 3 with t' = kThreads - 1 - t.
            const int b0 = (kThreads - 1 - tid) * (kBins / kThreads);
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
            upto += __reduce_add_sync(0xffffffffu, lane < warp ? wsum[lane % kWarps] : 0u);
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
            if (rank == s_count && base > 0) {   // the whole bin is wanted
                limit = base - 1;
                ties = 0;
                break;
            }
            width = shift;
            shift = max(0, shift - kBinBits);
        }
        // ---- positions in order
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
        a += __reduce_add_sync(0xffffffffu, lane < warp ? wsum[lane % kWarps] : 0u) - above;
        e += __reduce_add_sync(0xffffffffu, lane < warp ? wsum2[lane % kWarps] : 0u) - equal;
        uint32_t at = a + min(e, ties);
        each([&](uint32_t x, int32_t j) {
            const bool take = x > limit || (x == limit && e < ties);
            e += x == limit;
            if (take) kept[p.first + at++] = p.first + j;
        });
    }
    if (!p.new_weights) return;
    // The kept weights move down, kept[r] >= r: a stretch is read before any of it is written.
    float* to = p.new_weights + ((int64_t)row * p.Hkv + g) * p.width;
    for (int32_t r = tid; r - tid < count; r += kThreads) {
        __syncthreads();
        const float x = r < count ? w[kept[r]] : 0.f;
        __syncthreads();
        if (r < count) to[r] = x;
    }
    __syncthreads();
    for (int32_t r = count + tid; r < p.width; r += kThreads) to[r] = 0.f;
}

// ---- pa_compact_tokens -------------------------------------------------------------
struct CompactParams {
    uint4 *k_cache, *v_cache;
    const int32_t *kept, *kept_lens, *block_tables, *new_tables;
    unsigned int* err;
    int32_t keep, max_blocks, new_max_blocks, Hkv, vecs, bs_shift, num_blocks;   // vecs: 16-byte pieces of a row
};

constexpr int kMove = 4;   // rows of a thread at a time, K and V each

// One CTA per (sequence, KV head).  Row r comes from kept[r] >= r, and both ascend: once a
// stretch of rows has been read, nothing that is still to be read lies in the stretch.
__global__ void __launch_bounds__(kThreads) compact_kernel(const CompactParams p) {
    const int32_t g = blockIdx.x, i = blockIdx.y, mask = (1 << p.bs_shift) - 1;
    const int32_t raw = p.kept_lens[i];
    if (threadIdx.x == 0 && g == 0 && (raw < 0 || raw > p.keep)) pa::raise_error(p.err, PA_DEVERR_CONTEXT);
    const int32_t n = max(0, min(raw, p.keep));
    const int32_t* kept = p.kept + ((int64_t)i * p.Hkv + g) * p.keep;
    const int rows = kThreads / p.vecs, r0 = threadIdx.x / p.vecs, c = threadIdx.x % p.vecs;
    for (int32_t base = 0; base < n; base += rows * kMove) {
        uint4 k[kMove], v[kMove];
        int64_t to[kMove];
#pragma unroll
        for (int u = 0; u < kMove; ++u) {
            const int32_t r = base + u * rows + r0;
            to[u] = -1;
            if (r >= n) continue;
            const int32_t pos = kept[r], sb = pos >> p.bs_shift, db = r >> p.bs_shift;
            if (pos < 0 || sb >= p.max_blocks || db >= p.new_max_blocks) {
                pa::raise_error(p.err, PA_DEVERR_TABLE_WIDTH);
                continue;
            }
            const int32_t src = p.block_tables[(int64_t)i * p.max_blocks + sb];
            const int32_t dst = p.new_tables[(int64_t)i * p.new_max_blocks + db];
            if ((uint32_t)src >= (uint32_t)p.num_blocks || (uint32_t)dst >= (uint32_t)p.num_blocks) {
                pa::raise_error(p.err, PA_DEVERR_BLOCK_ID);
                continue;
            }
            if (src == dst && pos == r) continue;
            const int64_t from = ((((int64_t)src << p.bs_shift) + (pos & mask)) * p.Hkv + g) * p.vecs + c;
            to[u] = ((((int64_t)dst << p.bs_shift) + (r & mask)) * p.Hkv + g) * p.vecs + c;
            k[u] = p.k_cache[from];
            v[u] = p.v_cache[from];
        }
        __syncthreads();
#pragma unroll
        for (int u = 0; u < kMove; ++u) {
            if (to[u] < 0) continue;
            p.k_cache[to[u]] = k[u];
            p.v_cache[to[u]] = v[u];
        }
    }
}

bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

}  // namespace

extern "C" {

PA_API pa_status pa_select_tokens(const float* weights, int32_t num_rows, int32_t width,
                                  const int32_t* rows, const int32_t* context_lens, int32_t B,
                                  int32_t Hkv, int32_t keep, int32_t first, int32_t last,
                                  int32_t* kept, int32_t* kept_lens, float* new_weights,
                                  void* stream) {
    if (B < 0 || Hkv <= 0 || num_rows <= 0 || width <= 0 || keep < 1 || first < 0 || last < 0 ||
        (int64_t)first + last > keep)
        return PA_ERR_INVALID;
    if (B > 4096) return PA_ERR_UNSUPPORTED;
    if (B == 0) return PA_OK;
    if (!weights || !rows || !context_lens || !kept || !kept_lens) return PA_ERR_INVALID;
    if (!aligned(weights, 4) || !aligned(rows, 4) || !aligned(context_lens, 4) || !aligned(kept, 4) ||
        !aligned(kept_lens, 4) || !aligned(new_weights, 4))
        return PA_ERR_INVALID;
    ChooseParams p{weights, new_weights, rows, context_lens, kept, kept_lens,
                   pa::device_error_word(), num_rows, width, Hkv, keep, first, last};
    if (!p.err) return PA_ERR_CUDA;
    select_tokens_kernel<<<dim3((unsigned)Hkv, (unsigned)B), kThreads, 0, static_cast<cudaStream_t>(stream)>>>(p);
    return pa::cuda_status(cudaGetLastError());
}

PA_API pa_status pa_compact_tokens(void* k_cache, void* v_cache, const int32_t* kept,
                                   int32_t keep, const int32_t* kept_lens,
                                   const int32_t* block_tables, int32_t max_blocks,
                                   const int32_t* new_tables, int32_t new_max_blocks, int32_t B,
                                   int32_t Hkv, int32_t d, int32_t block_size,
                                   int32_t num_blocks, pa_dtype dtype, void* stream) {
    if (B < 0 || Hkv <= 0 || keep < 1 || max_blocks <= 0 || new_max_blocks <= 0 || num_blocks <= 0)
        return PA_ERR_INVALID;
    if (dtype != PA_F16 && dtype != PA_BF16) return PA_ERR_UNSUPPORTED;
    if (d != 64 && d != 128) return PA_ERR_UNSUPPORTED;
    if (block_size != 8 && block_size != 16 && block_size != 32) return PA_ERR_UNSUPPORTED;
    if (B > 4096 || (int64_t)num_blocks * block_size > INT32_MAX) return PA_ERR_UNSUPPORTED;
    if (B == 0) return PA_OK;
    if (!k_cache || !v_cache || !kept || !kept_lens || !block_tables || !new_tables)
        return PA_ERR_INVALID;
    if (!aligned(k_cache, 16) || !aligned(v_cache, 16) || !aligned(kept, 4) || !aligned(kept_lens, 4) ||
        !aligned(block_tables, 4) || !aligned(new_tables, 4))
        return PA_ERR_INVALID;
    CompactParams p{static_cast<uint4*>(k_cache), static_cast<uint4*>(v_cache), kept, kept_lens,
                    block_tables, new_tables, pa::device_error_word(), keep, max_blocks,
                    new_max_blocks, Hkv, d / 8, block_size == 8 ? 3 : block_size == 16 ? 4 : 5, num_blocks};
    if (!p.err) return PA_ERR_CUDA;
    compact_kernel<<<dim3((unsigned)Hkv, (unsigned)B), kThreads, 0, static_cast<cudaStream_t>(stream)>>>(p);
    return pa::cuda_status(cudaGetLastError());
}

}  // extern "C"
