// The work list of the quantised decodes: (sequence, KV head, 32-token chunk) triples, cut
// into parts of equal cost for the CTAs and, inside each, for its warps, and the joining of
// what warps and CTAs found for the same (sequence, KV head) pair:
//     M = max m_p,  out = sum_p 2^(m_p - M) o_p / sum_p 2^(m_p - M) l_p.
// A warp walks its share run by run (a run: neighbouring chunks of one pair) and meets no
// other before the end.
#pragma once

#include <cuda_runtime.h>

#include "pa.h"
#include "pa_common.cuh"

namespace pa {
namespace runs {

constexpr int kChunk = 32;              // tokens per stage of a warp's ring
constexpr int kMaxG = 16;               // query heads of a pair
constexpr int kMaxBatch = 4096;
constexpr int kMaxCtas = 512;

// One partial result in shared memory: row maxima [G], row sums [G], padding to 16 bytes,
// outputs [G][D]; in the workspace: maxima and sums [kMaxG] each.
__host__ __device__ constexpr int slot_head(int G) { return (2 * G + 3) & ~3; }
__host__ __device__ constexpr int slot_floats(int G, int D) { return slot_head(G) + G * D; }
__host__ __device__ constexpr int partial_floats(int D) { return 2 * kMaxG + kMaxG * D; }

// A run of chunks [c0, end) of one pair that a warp left in shared memory.
struct Run {
    int32_t a;    // position of the pair in the list; -1: none
    int32_t i, g, c0, end, nc;
    uint32_t at;  // at the end, entry x: the set of runs of the CTA's x-th pair,
    int32_t pad;  // and the first of them (+ 256: other CTAs hold more)
};

// Shared memory of a CTA: a ring of stages per warp, a slot per warp for a run that
// ends before the ring is free, and the list.
struct Layout {
    uint32_t slots, runs, last, scan, prefix, total;
};

// rings: bytes of all rings and what the kernel keeps beside them.
__host__ __device__ inline Layout make_layout(uint32_t rings, int D, int G, int B, int warps) {
    Layout L;
    L.slots = rings;
    L.runs = L.slots + warps * slot_floats(G, D) * 4;       // [2 * warps]
    L.last = L.runs + 2 * warps * (uint32_t)sizeof(Run);    // "the last CTA of the pair"
    L.scan = L.last + 8;
    L.prefix = L.scan + warps * 8;                          // [B + 1]
    L.total = L.prefix + (uint32_t)(B + 1) * 4;
    return L;
}

__device__ __forceinline__ int32_t clamp_len(int32_t n, int32_t cap) {
    return n < 0 ? 0 : (n > cap ? cap : n);
}

// W units cut into n parts, the first W % n of them one unit longer.
struct Cut {
    int32_t q, r;
    __device__ Cut(int32_t W, int32_t n) : q(W / n), r(W - W / n * n) {}
    __device__ int32_t begin(int32_t x) const { return x * q + min(x, r); }
    // the part that holds position c
    __device__ int32_t part(int32_t c) const {
        const int32_t big = r * (q + 1);
        return c < big ? c / (q + 1) : r + (c - big) / q;
    }
};

// The list of pairs is cut by cost, in units of a chunk: kPairCost of them for the pair itself
// (its q, its table's first entries, its end), then its nc chunks, from position a on.  Cut
// by chunks alone, CTAs with many short pairs ended 10 us after those with few: the 4-bit
// decode of 64 sequences of 128 .. 2048 tokens, 40 heads, took 75.5 us against 72.3 with 2 (71.5
// with 1, 73.9 with 3), that of 32 long-tailed contexts 26.5 us against 24.6 (25.4, 24.4).
constexpr int kPairCost = 2;

// A position in the list: chunk c of pair (i, g).
struct Cursor {
    int32_t i, g, c, nc, a;
};

__device__ __forceinline__ Cursor find(const int32_t* prefix, int32_t B, int32_t Hkv, int32_t pos) {
    int32_t lo = 0, hi = B;   // largest i with prefix[i] <= pos
#pragma unroll 1
    while (hi - lo > 1) {
        const int32_t mid = (lo + hi) >> 1;
        if (prefix[mid] <= pos) lo = mid; else hi = mid;
    }
    Cursor s;
    s.i = lo;
    const int32_t cost = (prefix[lo + 1] - prefix[lo]) / Hkv, local = pos - prefix[lo];
    s.nc = cost - kPairCost;
    s.g = local / cost;
    s.a = prefix[lo] + s.g * cost;
    s.c = max(0, pos - s.a - kPairCost);
    return s;
}

// The pair after s (there is one).
__device__ __forceinline__ Cursor next_pair(const int32_t* prefix, int32_t Hkv, Cursor s) {
    s.a += kPairCost + s.nc;
    s.c = 0;
    if (++s.g == Hkv) {
        s.g = 0;
        do ++s.i; while (prefix[s.i + 1] == prefix[s.i]);
        s.nc = (prefix[s.i + 1] - prefix[s.i]) / Hkv - kPairCost;
    }
    return s;
}

// 16 bytes global -> shared, asynchronously; zeros and no read unless ok.
__device__ __forceinline__ void copy16(uint32_t to, const void* from, bool ok, uint64_t policy) {
    asm volatile("cp.async.cg.shared.global.L2::cache_hint [%0], [%1], 16, %2, %3;" ::"r"(to), "l"(from),
                 "r"(ok ? 16 : 0), "l"(policy) : "memory");
}
// 4 bytes, likewise.
__device__ __forceinline__ void copy4(uint32_t to, const void* from, bool ok) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(to), "l"(from), "r"(ok ? 4 : 0)
                 : "memory");
}
__device__ __forceinline__ void commit_group() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void wait_group() {   // until at most N of this thread's groups are in flight
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

__device__ __forceinline__ void prefetch_l2(const void* p) {
    asm volatile("prefetch.global.L2 [%0];" ::"l"(p));
}

// prefix[i] = Hkv * (chunks and kPairCost) of the sequences before i that hold any; returns the
// chunks of the whole list.  `Hkv` counts pairs of a sequence.  Raises the lengths' errors.
__device__ __forceinline__ int32_t list_prefix(const int32_t* context_lens, int32_t B, int32_t Hkv,
                                               int32_t max_len, unsigned int* err, int nw,
                                               int32_t* prefix, int32_t* scan, int32_t* total_at,
                                               Run* runs) {
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, threads = nw * 32;
    const int per = (B + threads - 1) / threads;
    const int beg = min(tid * per, B), end = min(beg + per, B);
    int32_t local = 0, held = 0;   // cost; sequences that are not empty
#pragma unroll 1
    for (int i = beg; i < end; ++i) {
        const int32_t raw = pa::ld_behind_wait(context_lens + i);
        if (blockIdx.x == 0) {
            if (raw < 0) pa::raise_error(err, PA_DEVERR_CONTEXT);
            if (raw > max_len) pa::raise_error(err, PA_DEVERR_TABLE_WIDTH);
        }
        const int32_t chunks = (clamp_len(raw, max_len) + kChunk - 1) / kChunk;
        local += chunks ? chunks + kPairCost : 0;
        held += chunks > 0;
    }
    held = __reduce_add_sync(0xffffffffu, held);
    int32_t x = local;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int32_t y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
    }
    if (lane == 31) {
        scan[warp] = x;
        scan[nw + warp] = held;
    }
    if (tid < 2 * nw) runs[tid].a = -1;
    __syncthreads();
    int32_t run = x - local;
#pragma unroll 1
    for (int w = 0; w < warp; ++w) run += scan[w];
#pragma unroll 1
    for (int i = beg; i < end; ++i) {
        prefix[i] = run * Hkv;
        const int32_t chunks = (clamp_len(pa::ld_behind_wait(context_lens + i), max_len) + kChunk - 1) / kChunk;
        run += chunks ? chunks + kPairCost : 0;
    }
    if (tid == 0) {
        int32_t total = 0, all = 0;
#pragma unroll 1
        for (int w = 0; w < nw; ++w) {
            total += scan[w];
            all += scan[nw + w];
        }
        prefix[B] = total * Hkv;
        *total_at = (total - kPairCost * all) * Hkv;   // chunks
    }
    __syncthreads();
    return *total_at;
}

// What the joining needs of a decode's parameters.
struct Out {
    uint16_t* out;
    int32_t* counters;   // [B * Hkv] arrival tickets of pairs split between CTAs
    float* partials;     // [2 * CTAs][partial_floats(D)]
    int32_t H, Hkv, G;   // Hkv: pairs of a sequence
};

// Joins the runs that the warps left (a barrier behind the last of them).  `ring`: bytes
// of a warp's ring, at the start of shared memory; a warp's first run lies in its slot, a later
// one in its ring.
template <int D, bool kBF16>
__device__ __forceinline__ void join_runs(const Out& p, const Cut& cut, int32_t cta_lo, int nw,
                                          unsigned char* smem, uint32_t ring, uint32_t slots,
                                          Run* runs, int32_t* is_last, int32_t* scan) {
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, threads = nw * 32;
    const int32_t Hkv = p.Hkv, G = p.G;
    // ====================== runs of one pair in several warps ======================
    // Runs lie in list order: a pair's runs are neighbours, warps without a second run
    // between them.  Lane k of every warp looks at run k (such gaps go with the pair
    // before them): whether it leads its pair, and whether the pair is whole or other CTAs
    // hold some of it (true of at most the CTA's first and last pair).
    const Run my = runs[lane < 2 * nw ? lane : 0];
    const bool valid_run = lane < 2 * nw && my.a >= 0;
    const uint32_t upto = 0xffffffffu >> (31 - lane);
    const uint32_t before = __ballot_sync(0xffffffffu, valid_run) & upto;
    const int32_t pair_of = __shfl_sync(0xffffffffu, my.a, before ? 31 - __clz(before) : 0);
    const int32_t seg = before ? pair_of : -1;
    const uint32_t same = __match_any_sync(0xffffffffu, seg);      // a contiguous set
    const int seg_last = 31 - __clz(same);
    const bool leads = valid_run && (same & upto) == (1u << lane);
    const uint32_t in_pair = same & __ballot_sync(0xffffffffu, valid_run);
    const int32_t pair_end = __shfl_sync(0xffffffffu, my.end, in_pair ? 31 - __clz(in_pair) : 0);
    const bool shared = my.c0 != 0 || pair_end != my.nc;
    const uint32_t lead = __ballot_sync(0xffffffffu, leads);
    const uint32_t open = __ballot_sync(0xffffffffu, leads && shared);
    // A warp's first run has its slot, a later one its ring.
    auto slot_at = [&](int k) {
        return reinterpret_cast<float*>(smem + (k & 1 ? (uint32_t)(k >> 1) * ring
                                                      : slots + (uint32_t)(k >> 1) * slot_floats(G, D) * 4));
    };
    // A CTA's first partial holds the pair that its share begins in or with, its second
    // the one that begins later.
    auto partial_at = [&](int32_t a) {
        return p.partials + (2 * (int64_t)blockIdx.x + (cta_lo >= a ? 0 : 1)) * partial_floats(D);
    };
    // Head by head: maximum and sum over each pair's runs (a segmented scan over the
    // lanes), each run's factor 2^(m_k - M) in place of its maximum.
#pragma unroll 1
    for (int h = warp; h < G; h += nw) {
        float* slot = slot_at(lane < 2 * nw ? lane : 0);
        const float m = valid_run ? slot[h] : -INFINITY;
        float M = m;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const float y = __shfl_up_sync(0xffffffffu, M, o);
            if (lane >= o && (same >> (lane - o) & 1)) M = fmaxf(M, y);
        }
        M = __shfl_sync(0xffffffffu, M, seg_last);
        const float f = valid_run ? pa::fast_exp2(m - M) : 0.f;
        float l = valid_run ? f * slot[G + h] : 0.f;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const float y = __shfl_up_sync(0xffffffffu, l, o);
            if (lane >= o && (same >> (lane - o) & 1)) l += y;
        }
        l = __shfl_sync(0xffffffffu, l, seg_last);
        if (valid_run) slot[h] = f;
        if (leads && !shared) slot[G + h] = 1.f / l;
        if (leads && shared) {
            partial_at(my.a)[h] = M;
            partial_at(my.a)[kMaxG + h] = l;
        }
    }
    if (warp == 0 && leads) {   // the pairs in order, for the loop below
        const int at = __popc(lead & (upto >> 1));
        runs[at].pad = lane | (shared ? 256 : 0);
        runs[at].at = in_pair;
    }
    __syncthreads();
    auto store4 = [&](int32_t i, int32_t h, int d4, float4 v, float inv) {
        *reinterpret_cast<uint2*>(p.out + ((int64_t)i * p.H + h) * D + d4) =
            make_uint2(pa::pack2<kBF16>(v.x * inv, v.y * inv), pa::pack2<kBF16>(v.z * inv, v.w * inv));
    };
    const int outs = G * D / 4;     // four outputs each
#pragma unroll 1
    for (int x = tid; x < __popc(lead) * outs; x += threads) {
        const int at = x / outs, e = x - at * outs;
        const int k = runs[at].pad & 255;
        const int h = e / (D / 4), d4 = e % (D / 4) * 4;
        float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
        for (uint32_t set = runs[at].at; set; set &= set - 1) {
            const float* slot = slot_at(__ffs(set) - 1);
            const float f = slot[h];
            const float4 y = *reinterpret_cast<const float4*>(slot + slot_head(G) + h * D + d4);
            v.x += f * y.x;
            v.y += f * y.y;
            v.z += f * y.z;
            v.w += f * y.w;
        }
        if (runs[at].pad & 256)
            *reinterpret_cast<float4*>(partial_at(runs[k].a) + 2 * kMaxG + e * 4) = v;
        else
            store4(runs[k].i, runs[k].g * G + h, d4, v, slot_at(k)[G + h]);
    }
    if (!open) return;

    // ================= pairs shared with other CTAs, by the whole CTA =================
    // Publish: the barrier orders every thread's stores before the ticket's release; the
    // ticket names the pair's last CTA and, for it, acquires the other CTAs' partials.
    constexpr int kPartial = partial_floats(D);
    const int n_open = __popc(open);   // one or two
    auto open_lead = [&](int w) { return w ? 31 - __clz(open) : __ffs(open) - 1; };
    __syncthreads();
    if (warp < n_open && lane == 0) {
        const Run& r = runs[open_lead(warp)];
        int32_t* ticket = p.counters + (int64_t)r.i * Hkv + r.g;
        const int32_t before_me = pa::atomic_add_acq_rel_gpu(ticket, 1);
        const int32_t first = cut.part(r.a + kPairCost);
        const int32_t n = cut.part(r.a + kPairCost + r.nc - 1) - first + 1;
        const bool last = before_me == n - 1;
        if (last) atomicExch(ticket, 0);   // ready for the next launch
        is_last[warp] = last ? n : 0;      // the pair's CTAs
        scan[warp] = first;
    }
    __syncthreads();
    // Two pairs to join: half the threads each, so that their loads are under way together.
    const bool both = n_open == 2 && is_last[0] && is_last[1];
    const int team = both ? threads / 2 : threads, my_w = both && tid >= team ? 1 : 0;
    const int ltid = tid - my_w * team;
#pragma unroll 1
    for (int w0 = 0; w0 < (both ? 1 : n_open); ++w0) {
        const int w = both ? my_w : w0;
        if (!is_last[w]) continue;
        const Run r = runs[open_lead(w)];
        const int c_first = scan[w], n = is_last[w], most = both ? max(is_last[0], is_last[1]) : n;
        const float* first = p.partials + (2 * (int64_t)c_first + (cut.begin(c_first) >= r.a ? 0 : 1)) * kPartial;
        const float* rest = p.partials + 2 * (int64_t)c_first * kPartial;
        // A group of threads has the outputs, four each, and eight partials' loads in flight;
        // of more than eight the groups take turns, and join in shared memory.
        const int wide = min(outs, team), groups = most > 8 ? team / wide : 1;
        const int grp = ltid / wide;
        float4* acc_at = reinterpret_cast<float4*>(smem) + my_w * team;   // [groups][outs]
        float2* ml_at = reinterpret_cast<float2*>(reinterpret_cast<float4*>(smem) + threads) + my_w * team;
#pragma unroll 1
        for (int e = ltid - grp * wide; e < outs && grp < groups; e += wide) {
            const int h = e / (D / 4);
            float M = -INFINITY, l = 0.f;
            float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 1
            for (int c0 = grp; c0 < n; c0 += 8 * groups) {
                float pm[8], pl[8];
                float4 po[8];
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const int c = c0 + j * groups;
                    if (c < n) {
                        const float* q = c ? rest + 2 * (int64_t)c * kPartial : first;
                        pm[j] = __ldcg(q + h);
                        pl[j] = __ldcg(q + kMaxG + h);
                        po[j] = __ldcg(reinterpret_cast<const float4*>(q + 2 * kMaxG) + e);
                    } else {
                        pm[j] = -INFINITY;
                        pl[j] = 0.f;
                        po[j] = make_float4(0.f, 0.f, 0.f, 0.f);
                    }
                }
                float Mb = M;
#pragma unroll
                for (int j = 0; j < 8; ++j) Mb = fmaxf(Mb, pm[j]);
                if (Mb == -INFINITY) continue;
                const float f0 = pa::fast_exp2(M - Mb);   // 0 while M = -inf
                l *= f0;
                acc.x *= f0;
                acc.y *= f0;
                acc.z *= f0;
                acc.w *= f0;
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const float f = pa::fast_exp2(pm[j] - Mb);
                    l += f * pl[j];
                    acc.x += f * po[j].x;
                    acc.y += f * po[j].y;
                    acc.z += f * po[j].z;
                    acc.w += f * po[j].w;
                }
                M = Mb;
            }
            if (groups == 1) {
                store4(r.i, r.g * G + h, e % (D / 4) * 4, acc, 1.f / l);
            } else {
                acc_at[grp * outs + e] = acc;
                ml_at[grp * outs + e] = make_float2(M, l);
            }
        }
        if (groups > 1) {
            __syncthreads();
#pragma unroll 1
            for (int e = ltid; e < outs; e += team) {
                const int use = min(groups, n);
                float M = -INFINITY, l = 0.f;
                float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 1
                for (int q = 0; q < use; ++q) M = fmaxf(M, ml_at[q * outs + e].x);
#pragma unroll 1
                for (int q = 0; q < use; ++q) {
                    const float2 ml = ml_at[q * outs + e];
                    const float4 y = acc_at[q * outs + e];
                    const float f = pa::fast_exp2(ml.x - M);
                    l += f * ml.y;
                    acc.x += f * y.x;
                    acc.y += f * y.y;
                    acc.z += f * y.z;
                    acc.w += f * y.w;
                }
                store4(r.i, r.g * G + e / (D / 4), e % (D / 4) * 4, acc, 1.f / l);
            }
            __syncthreads();
        }
    }
}

// Bytes of the arrival tickets at a workspace's start.
inline size_t ticket_bytes(int32_t B, int32_t H) {
    return ((size_t)B * H * sizeof(int32_t) + 255) & ~size_t(255);
}

}  // namespace runs
}  // namespace pa
