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
// And back (0 and NaN as the numbers that ordered() takes them for).
__device__ __forceinline__ float weight_of(uint32_t key) {
    return __uint_as_float(key >> 31 ? key ^ 0x80000000u : ~key);
}

constexpr int kBinBits = 10, kBins = 1 << kBinBits;
constexpr int kMaxKeys = 48 * 1024;   // weights that shared memory holds

// A warp has a contiguous stretch of the weights, 32 neighbours an instruction, so that ranks
// inside it are counts of ballots: up to kPer instructions' in registers, more (an accumulator's width
// says what there may be, its context's length what there is) in shared memory, up to kMaxKeys,
// or read again from L2 by each pass.  Bound by
// latency: the length and row, the weights, two or three passes of three barriers each, two
// scans: 3.5 us for 20 pairs of up to 1000 weights, 12.3 for 256 of 8192, 21 for 32 of 30000.
// (Eight counts a bin, one for every eighth lane, took 20 us for the 256 pairs, 13.4 then: the
// counts' clearing and adding up costs more than lanes that meet in one.)
enum More { kNone, kShared, kAgain };
template <int kThreads, int kPer, More kMore>
__global__ void __launch_bounds__(kThreads) select_tokens_kernel(const ChooseParams p) {
    constexpr int kWarps = kThreads / 32, kOwn = kBins / kThreads;   // bins of a thread
    __shared__ __align__(16) uint32_t hist[kBins];
    extern __shared__ uint32_t held[];   // kShared: the keys between, where registers do not hold them
    __shared__ uint32_t s_top[kWarps], s_low[kWarps], wsum[kWarps], wsum2[kWarps];
    __shared__ uint32_t s_bin, s_rank, s_count;
    // What moves the rows may be launched: it waits for this grid's end.
    asm volatile("griddepcontrol.launch_dependents;");
    asm volatile("griddepcontrol.wait;" ::: "memory");   // launched while the kernel before may run
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const uint32_t below = (1u << lane) - 1;
    const int32_t g = blockIdx.x, i = blockIdx.y;
    int32_t* kept = p.kept + ((int64_t)i * p.Hkv + g) * p.keep;
    const int32_t row = pa::ld_behind_wait(p.rows + i), raw = pa::ld_behind_wait(p.context_lens + i);
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
    float* to = p.new_weights ? p.new_weights + ((int64_t)row * p.Hkv + g) * p.width : nullptr;
    const int32_t k = p.keep - p.first - p.last, m = n - p.first - p.last;   // k < m where tokens go
    const bool choose = n > p.keep && k > 0;
    const bool regs = kMore == kNone || m <= kPer * kThreads;
    const int32_t per = regs ? kPer : (m + kThreads - 1) / kThreads;
    const int32_t beg = warp * per * 32 + lane;
    uint32_t own[kPer];
    auto key_at = [&](int32_t j) { return ordered(pa::ld_behind_wait(w + p.first + j)); };
#pragma unroll
    for (int q = 0; q < kPer; ++q)
        own[q] = choose && regs && beg + q * 32 < m ? key_at(beg + q * 32) : 0u;
    if constexpr (kMore == kShared)
        if (choose && !regs)
#pragma unroll 8
            for (int32_t j = tid; j < m; j += kThreads) held[j] = key_at(j);
    // Of the last ones, a thread's first weight.
    const float tail = to && n > p.keep && tid < p.last ? pa::ld_behind_wait(w + n - p.last + tid) : 0.f;
    const int32_t head = n <= p.keep ? n : p.first;
    for (int32_t j = tid; j < head; j += kThreads) kept[j] = j;
    if (n > p.keep)
        for (int32_t j = tid; j < p.last; j += kThreads) kept[p.keep - p.last + j] = n - p.last + j;
    if (choose) {
        // f(key, place, whether there is one), for whole warps
        auto each = [&](auto f) {
            if (regs) {
#pragma unroll
                for (int q = 0; q < kPer; ++q) f(own[q], beg + q * 32, beg + q * 32 < m);
            } else if constexpr (kMore != kNone) {
#pragma unroll 4
                for (int32_t q = 0; q < per; ++q) {
                    const int32_t j = beg + q * 32;
                    f(j >= m ? 0u : kMore == kShared ? held[j] : key_at(j), j, j < m);
                }
            }
        };
        uint32_t top = 0, low = 0;    // the largest key, and the smallest's complement
        for (int b = tid; b < kBins; b += kThreads) hist[b] = 0;
        if constexpr (kMore == kShared) __syncthreads();
        each([&](uint32_t x, int32_t, bool is) {
            top = max(top, x);        // 0 where there is none
            if (is) low = max(low, ~x);
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
            each([&](uint32_t x, int32_t, bool is) {
                x -= base;                             // keys below base wrap to large numbers
                if (is && (width == 32 || (x >> width) == 0)) atomicAdd(&hist[x >> shift], 1u);
            });
            __syncthreads();
            // Counts from the top: thread t owns kOwn bins, those of thread 0 the highest.
            const int b0 = (kThreads - 1 - tid) * kOwn;
            uint32_t c[kOwn], mine = 0;
#pragma unroll
            for (int q = 0; q < kOwn; ++q) {
                c[q] = hist[b0 + q];
                hist[b0 + q] = 0;
                mine += c[q];
            }
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
                uint32_t want = rank - (upto - mine);
                int q = kOwn - 1;
#pragma unroll
                for (int x = kOwn - 1; x > 0; --x)
                    if (q == x && c[x] < want) want -= c[x], q = x - 1;
                s_bin = b0 + q;
                s_rank = want;
                s_count = c[0];
#pragma unroll
                for (int x = 1; x < kOwn; ++x)
                    if (q == x) s_count = c[x];
            }
            __syncthreads();
            base += s_bin << shift;
            rank = s_rank;
            if (rank == s_count && base > 0) {   // the whole bin is wanted
                limit = base - 1;
                ties = 0;
                break;
            }
            if (shift == 0) {
                limit = base;
                ties = rank;
                break;
            }
            width = shift;
            shift = max(0, shift - kBinBits);
        }
        // ---- positions in order; the weights with them where every weight between has been read
        const bool now = regs || kMore == kShared;
        uint32_t above = 0, equal = 0;
        each([&](uint32_t x, int32_t, bool is) {
            above += is && x > limit;
            if (ties) equal += is && x == limit;
        });
        above = __reduce_add_sync(0xffffffffu, above);
        equal = __reduce_add_sync(0xffffffffu, equal);
        if (lane == 0) {
            wsum[warp] = above;
            wsum2[warp] = equal;
        }
        __syncthreads();
        uint32_t a = p.first + __reduce_add_sync(0xffffffffu, lane < warp ? wsum[lane % kWarps] : 0u);
        if (!ties) {
            each([&](uint32_t x, int32_t j, bool is) {
                const bool take = is && x > limit;
                const uint32_t up = __ballot_sync(0xffffffffu, take);
                if (take) {
                    const uint32_t at = a + __popc(up & below);
                    kept[at] = p.first + j;
                    if (now && to) to[at] = weight_of(x);
                }
                a += __popc(up);
            });
        } else {
            uint32_t e = __reduce_add_sync(0xffffffffu, lane < warp ? wsum2[lane % kWarps] : 0u);
            each([&](uint32_t x, int32_t j, bool is) {
                const uint32_t up = __ballot_sync(0xffffffffu, is && x > limit);
                const uint32_t eq = __ballot_sync(0xffffffffu, is && x == limit);
                const uint32_t my_e = e + __popc(eq & below);
                if (up >> lane & 1 || (eq >> lane & 1 && my_e < ties)) {
                    const uint32_t at = a + __popc(up & below) + min(my_e, ties);
                    kept[at] = p.first + j;
                    if (now && to) to[at] = weight_of(x);
                }
                a += __popc(up);
                e += __popc(eq);
            });
        }
    }
    if (!to) return;
    // The weights move down, to r from kept[r] >= r: what a place held has been read, or is the
    // place's own.
    __syncthreads();
    if (to != w)
        for (int32_t r = tid; r < head; r += kThreads) to[r] = pa::ld_behind_wait(w + r);
    if (n > p.keep) {
        auto move = [&](int32_t r0, int32_t r1, auto from) {   // a stretch is read before any of it is written
            for (int32_t r = r0 + tid; r - tid < r1; r += kThreads) {
                const float x = r < r1 ? pa::ld_behind_wait(w + from(r)) : 0.f;
                __syncthreads();
                if (r < r1) to[r] = x;
                __syncthreads();
            }
        };
        if (kMore == kAgain && choose && !regs) move(p.first, p.keep - p.last, [&](int32_t r) { return kept[r]; });
        if (tid < p.last) to[p.keep - p.last + tid] = tail;
        if (p.last > kThreads) move(p.keep - p.last + kThreads, p.keep, [&](int32_t r) { return n - p.keep + r; });
    }
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

// A cluster of CTAs per (sequence, KV head).  Row r comes from kept[r] >= r, and both ascend:
// once a stretch of rows has been read, nothing that is still to be read lies in the
// stretch.  So the cluster reads a stretch into its registers, meets, writes it, and reads the
// next one, without meeting again.  Bound by HBM: 256 pairs of 4096 rows at d = 128 take 176 us
// (1.07 GB, 6.1 TB/s, 91 % of the measured copy), 2560 of 512 rows 204 (6.6 TB/s); few pairs by
// the latency of a stretch: 8 of 8000 rows 20 us, of which the bytes are 10.
template <int kThreads>
__global__ void __launch_bounds__(kThreads, 1024 / kThreads) compact_kernel(const CompactParams p) {
    asm volatile("griddepcontrol.wait;" ::: "memory");   // launched while the choice may be made
    uint32_t rank, ctas;
    asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(rank));
    asm("mov.u32 %0, %%cluster_nctarank;" : "=r"(ctas));
    const int32_t pair = blockIdx.x / ctas, i = pair / p.Hkv, g = pair - i * p.Hkv, mask = (1 << p.bs_shift) - 1;
    const int32_t raw = pa::ld_behind_wait(p.kept_lens + i);
    if (threadIdx.x == 0 && rank == 0 && g == 0 && (raw < 0 || raw > p.keep))
        pa::raise_error(p.err, PA_DEVERR_CONTEXT);
    const int32_t n = max(0, min(raw, p.keep));
    const int32_t* kept = p.kept + (int64_t)pair * p.keep;
    const int32_t* from_table = p.block_tables + (int64_t)i * p.max_blocks;
    const int32_t* to_table = p.new_tables + (int64_t)i * p.new_max_blocks;
    const int rows = kThreads / p.vecs, r0 = threadIdx.x / p.vecs, c = threadIdx.x % p.vecs;
    const int32_t stretch = rows * kMove * (int32_t)ctas;   // of the cluster
    auto piece = [&](int32_t slot) { return ((int64_t)slot * p.Hkv + g) * p.vecs + c; };
    int32_t from[kMove], to[kMove];   // slots of this thread's rows of a stretch; to -1: not moved
    auto places = [&](int32_t base) {
        const uint32_t at = (uint32_t)base + rank * rows * kMove + r0;   // < 2^31 + 2^14
#pragma unroll
        for (int u = 0; u < kMove; ++u) {
            const uint32_t r = at + u * rows;
            from[u] = r < (uint32_t)n ? pa::ld_behind_wait(kept + r) : -1;
        }
#pragma unroll
        for (int u = 0; u < kMove; ++u) {
            const uint32_t r = at + u * rows;
            to[u] = -1;
            if (r >= (uint32_t)n) continue;
            const int32_t pos = from[u], sb = pos >> p.bs_shift, db = (int32_t)(r >> p.bs_shift);
            if (pos < 0 || sb >= p.max_blocks || db >= p.new_max_blocks) {
                pa::raise_error(p.err, PA_DEVERR_TABLE_WIDTH);
                continue;
            }
            const int32_t src = pa::ld_behind_wait(from_table + sb), dst = pa::ld_behind_wait(to_table + db);
            if ((uint32_t)src >= (uint32_t)p.num_blocks || (uint32_t)dst >= (uint32_t)p.num_blocks) {
                pa::raise_error(p.err, PA_DEVERR_BLOCK_ID);
                continue;
            }
            from[u] = (src << p.bs_shift) + (pos & mask);
            to[u] = (dst << p.bs_shift) + (int32_t)(r & mask);
            if (from[u] == to[u]) to[u] = -1;   // stays
        }
    };
    if (n > 0) places(0);
#pragma unroll 1
    for (int32_t base = 0; base < n;) {
        uint4 k[kMove], v[kMove];
        int32_t now[kMove];
#pragma unroll
        for (int u = 0; u < kMove; ++u)
            if (to[u] >= 0) k[u] = pa::ld_behind_wait(p.k_cache + piece(from[u]));
#pragma unroll
        for (int u = 0; u < kMove; ++u) {
            if (to[u] >= 0) v[u] = pa::ld_behind_wait(p.v_cache + piece(from[u]));
            now[u] = to[u];
        }
        // The next stretch's places, three loads one behind the other, while these rows travel.
        base += min(stretch, n - base);
        if (base < n) places(base);
        // Every row of the stretch has been read before any CTA writes over it: only a release and an
        // acquire say so.  (A relaxed meeting orders nothing, and what the compiler is told about the
        // rows' registers reaches no instruction.)  The release waits for the writes of the stretch
        // before as well.
        if (ctas == 1)
            __syncthreads();
        else
            asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
#pragma unroll
        for (int u = 0; u < kMove; ++u)
            if (now[u] >= 0) {
                p.k_cache[piece(now[u])] = k[u];
                p.v_cache[piece(now[u])] = v[u];
            }
    }
}

template <typename K, typename P>
pa_status launch_early(K kern, dim3 grid, int threads, int cluster, size_t smem, cudaStream_t stream,
                       const P& p) {
    cudaLaunchAttribute attr[2] = {};
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = (unsigned)cluster;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = grid;
    cfg.blockDim = dim3((unsigned)threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = cluster > 0 ? 2 : 1;
    return pa::cuda_status(cudaLaunchKernelEx(&cfg, kern, p));
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
    // The threads walk a row up to 1024 places at a time, in 32 bits.
    if (B > 4096 || width > INT32_MAX - 1024 || keep > INT32_MAX - 1024) return PA_ERR_UNSUPPORTED;
    if (B == 0) return PA_OK;
    if (!weights || !rows || !context_lens || !kept || !kept_lens) return PA_ERR_INVALID;
    if (!aligned(weights, 4) || !aligned(rows, 4) || !aligned(context_lens, 4) || !aligned(kept, 4) ||
        !aligned(kept_lens, 4) || !aligned(new_weights, 4))
        return PA_ERR_INVALID;
    ChooseParams p{weights, new_weights, rows, context_lens, kept, kept_lens,
                   pa::device_error_word(), num_rows, width, Hkv, keep, first, last};
    if (!p.err) return PA_ERR_CUDA;
    const dim3 grid((unsigned)Hkv, (unsigned)B);
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    const int64_t most = (int64_t)width - first - last;   // weights to choose from, at most
    const int sms = pa::device_sm_count();
    if (!sms) return PA_ERR_CUDA;
    if (most <= 4 * 256) return launch_early(select_tokens_kernel<256, 4, kNone>, grid, 256, 0, 0, st, p);
    if (most <= 8 * 256) return launch_early(select_tokens_kernel<256, 8, kNone>, grid, 256, 0, 0, st, p);
    // Many pairs of which few tokens are wanted have contexts to match, whatever the rows' width:
    // small CTAs (2560 pairs, 2048 weights in rows of 4096: 26 us, with 1024 threads each 84; 640 in rows
    // of 40000: 30 and 41; but of 8192 weights 2560 pairs 135 and 108, 640 67 and 28).
    if ((int64_t)B * Hkv > 4 * sms && keep <= 8 * 256)
        return launch_early(select_tokens_kernel<256, 8, kAgain>, grid, 256, 0, 0, st, p);
    if (most <= 8 * 1024) return launch_early(select_tokens_kernel<1024, 8, kNone>, grid, 1024, 0, 0, st, p);
    // Wider rows: shared memory for all of them where each CTA has an SM to itself anyway.
    if (most > kMaxKeys || (int64_t)B * Hkv > sms)
        return launch_early(select_tokens_kernel<1024, 8, kAgain>, grid, 1024, 0, 0, st, p);
    auto kern = select_tokens_kernel<1024, 8, kShared>;
    static pa::DeviceOnce once;
    if (!pa::allow_smem(once, kern, kMaxKeys * 4)) return PA_ERR_CUDA;
    return launch_early(kern, grid, 1024, 0, (size_t)most * 4, st, p);
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
    const int sms = pa::device_sm_count();
    if (!sms) return PA_ERR_CUDA;
    const int64_t pairs = (int64_t)B * Hkv;
    if (pairs > INT32_MAX / 8) return PA_ERR_UNSUPPORTED;
    // CTAs of a pair: one where there are more pairs than SMs (256 pairs of 4096 rows at d = 128: one
    // 176 us, two 186, four 186, eight 188; 160 of 4000: 130, 156, 149, 130; 512 of 1024: 96, 94, 94,
    // 95; 2560 of 512: 204, 214, 217, 232); else as many as its rows fill, until there are four of 256
    // threads for every SM, eight at most (128 pairs of 4000: 102, 96, 95, 96; 32 of 8000: 142, 92, 60,
    // 52); of more threads where there are too few of them to fill the SMs with 1024 each.
    const int small = 256 / p.vecs * kMove;
    int cluster = 1;
    if (pairs <= sms)
        while (cluster < 8 && (int64_t)cluster * small < keep && pairs * cluster < 4 * sms) cluster *= 2;
    const dim3 grid((unsigned)(pairs * cluster));
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (pairs * cluster <= sms) return launch_early(compact_kernel<1024>, grid, 1024, cluster, 0, st, p);
    if (pairs * cluster <= 3 * sms) return launch_early(compact_kernel<512>, grid, 512, cluster, 0, st, p);
    return launch_early(compact_kernel<256>, grid, 256, cluster, 0, st, p);
}

}  // extern "C"
