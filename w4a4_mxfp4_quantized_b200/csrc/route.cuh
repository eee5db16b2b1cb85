// route.cuh -- the router of a mixture-of-experts layer and the row plan that the grouped calls take.
//
// Router: per token, l_e = fp32(logit_e) with NaN read as -inf (a masked expert) and +inf as the largest
// finite fp32. The topk experts of largest l are chosen, ties to the lowest expert; a choice whose l is -inf is
// dropped (id -1, weight 0). With m = max l and the sum over the chosen experts (renormalize) or, for softmax,
// over all E:
//     softmax:  p_e = exp(l_e - m),                          weight = scale * p_e / sum p
//     sigmoid:  p_e = exp(min(l_e, 0) - c) / (1 + exp(-|l_e|)),  weight = scale * p_e / (sum p or 1)
// where c = min(m, 0) when renormalizing (it cancels in the quotient and keeps far negative scores from
// underflowing together) and 0 otherwise: exp(min(l, 0)) / (1 + exp(-|l|)) is the sigmoid without overflow.
//
// Row plan: a stable counting sort of the R = T * topk choices by group. group_offsets[g] is the first sorted
// row of group g, pos[i] the sorted row of entry i (-1 for an id outside [0, E)), row_index[r] the token
// (entry / topk) of sorted row r; entries of no group follow the last group in their order.
//
// Bound by latency: a prefill's 65,536 entries are 0.8 MB. One CTA sorts up to 1,024 entries, a cluster of eight up to 8,192
// and one of sixteen more (their counts meet in distributed shared memory, so one launch and no workspace do); with up to
// 256 tokens the same launch chooses the experts too, a warp per token.
// Measured on B200 (128 experts, top-8): one token 4.9 us, 64 tokens 6.1, 8192 tokens 15.5 us in two launches (5.5 for the
// choice, 9.6 for the sort); the sort of 64 entries 3.4 us.
#pragma once

#include <stdint.h>

#include "ptx.cuh"

namespace macaq {

constexpr int kRouteMaxExperts = 1024;
constexpr int kRouteMaxTopk = 32;
constexpr int kRouteWarps = 8;          // tokens in flight per CTA of the top-k kernel
constexpr int kGroupThreads = 1024;
constexpr int kGroupWarps = kGroupThreads / 32;
constexpr int kGroupCluster = 8;
// Entries that one CTA sorts, and up to which a cluster has 8 CTAs, not 16. Measured with 1, 8, 16 CTAs in a graph, us: of
// 128 groups 512 entries 4.4, 4.8, 5.1; 1024 5.1, 4.9, 5.1; 2048 6.2, 4.9, 5.1; 4096 8.5, 5.1, 5.3; 8192 13.6, 5.9, 5.7;
// 16,384 23.6, 6.9, 6.2; 65,536 84, 14.5, 9.8. Of 1024 groups 1024 entries 6.7, 7.4, 9.5; 8192 16.9, 8.5, 9.9; 32,768 52.7,
// 12.8, 12.1.
constexpr int kGroupOneCta = 1024;
constexpr int kGroupWide = 8192;
constexpr int kRouteFusedTokens = 256;   // tokens whose experts are chosen in the same launch: one per warp of a cluster

struct RouteArgs {
    const void *logits;     // [T, E] bf16 or fp32, rows `ld` elements apart
    int64_t ld;
    int64_t T;
    int32_t E, topk;
    int32_t f32, sigmoid, renorm;
    float scale;
    float *weights;         // [T, topk]
    int32_t *ids;           // [T, topk]
};

struct GroupArgs {
    const int32_t *ids;     // [R]
    int64_t R;
    int32_t topk, E;
    int32_t *offsets;       // [E + 1]
    int32_t *row_index;     // [R]
    int32_t *pos;           // [R]
};

__device__ __forceinline__ float route_logit(const RouteArgs &a, int64_t t, int e) {
    const float v = a.f32 ? static_cast<const float *>(a.logits)[t * a.ld + e]
                          : __uint_as_float(static_cast<uint32_t>(static_cast<const uint16_t *>(a.logits)[t * a.ld + e]) << 16);
    return v != v ? -INFINITY : fminf(v, 3.402823466e38f);
}

// Order-preserving map of an fp32 value (not NaN) to uint32; 0 is below every value's key.
__device__ __forceinline__ uint32_t order_key(float v) {
    const uint32_t u = __float_as_uint(v + 0.0f);   // -0 becomes +0: the two tie
    return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

__device__ __forceinline__ float key_value(uint32_t k) { return __uint_as_float((k & 0x80000000u) ? (k & 0x7FFFFFFFu) : ~k); }

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) v += __shfl_xor_sync(0xffffffffu, v, d);
    return v;
}

// One warp, one token: lane l holds the experts l, l + 32, ... as keys; each round takes the largest key by
// a warp-wide maximum and then the lowest expert that holds it. kVpl: experts per lane.
template <int kVpl>
__device__ __forceinline__ void route_token(const RouteArgs &a, int64_t t, int lane) {
    uint32_t key[kVpl];
#pragma unroll
    for (int v = 0; v < kVpl; ++v) {
        const int e = v * 32 + lane;
        key[v] = e < a.E ? order_key(route_logit(a, t, e)) : 0u;
    }
    const uint32_t kMasked = order_key(-INFINITY);
    uint32_t best = 0;
#pragma unroll
    for (int v = 0; v < kVpl; ++v) best = max(best, key[v]);
    best = __reduce_max_sync(0xffffffffu, best);
    const float m = best > kMasked ? key_value(best) : 0.0f;
    float total = 0.0f;   // softmax over all experts
    if (!a.sigmoid && !a.renorm) {
#pragma unroll
        for (int v = 0; v < kVpl; ++v)
            if (key[v] > kMasked) total += expf(key_value(key[v]) - m);
        total = warp_sum(total);
    }
    int my_id = -1;
    uint32_t my_key = kMasked;
    for (int j = 0; j < a.topk; ++j) {
        uint32_t k = 0;
#pragma unroll
        for (int v = 0; v < kVpl; ++v) k = max(k, key[v]);
        const uint32_t top = __reduce_max_sync(0xffffffffu, k);
        uint32_t id = 0xffffffffu;
#pragma unroll
        for (int v = kVpl - 1; v >= 0; --v)
            if (key[v] == top) id = static_cast<uint32_t>(v * 32 + lane);
        id = __reduce_min_sync(0xffffffffu, id);
#pragma unroll
        for (int v = 0; v < kVpl; ++v)
            if (id == static_cast<uint32_t>(v * 32 + lane)) key[v] = 0u;   // below -inf: not taken again
        if (lane == j && top > kMasked) {
            my_id = static_cast<int>(id);
            my_key = top;
        }
    }
    float p = 0.0f;
    if (my_id >= 0) {
        const float l = key_value(my_key);
        p = a.sigmoid ? expf(fminf(l, 0.0f) - (a.renorm ? fminf(m, 0.0f) : 0.0f)) / (1.0f + expf(-fabsf(l))) : expf(l - m);
    }
    if (a.renorm) total = warp_sum(p);
    if (lane < a.topk) {
        a.weights[t * a.topk + lane] = my_id < 0 ? 0.0f : a.scale * ((a.renorm || !a.sigmoid) ? p / total : p);
        a.ids[t * a.topk + lane] = my_id;
    }
}

template <int kVpl>
__global__ void __launch_bounds__(kRouteWarps * 32) route_topk_kernel(RouteArgs a) {
    griddep_wait();
    griddep_launch_dependents();
    const int lane = threadIdx.x & 31;
    const int64_t stride = static_cast<int64_t>(gridDim.x) * kRouteWarps;
    for (int64_t t = static_cast<int64_t>(blockIdx.x) * kRouteWarps + (threadIdx.x >> 5); t < a.T; t += stride)
        route_token<kVpl>(a, t, lane);
}

// The lanes of `live` whose bucket equals this lane's, by one vote per bit. For 65,536 entries of 128 groups
// on eight CTAs this took 15.0 us, match.any 18.4.
__device__ __forceinline__ uint32_t group_peers(uint32_t live, int b, int bits) {
    uint32_t peers = live;
    for (int i = 0; i < bits; ++i) {
        const uint32_t set = __ballot_sync(live, (b >> i) & 1);
        peers &= ((b >> i) & 1) ? set : ~set;
    }
    return peers;
}

// The row plan, by one CTA or a cluster (`ctas`): CTA c owns a contiguous piece of the tokens, each of its warps a
// contiguous piece of their entries. A warp walks its piece 32 entries at a time, and the lanes with the same group find
// one another by votes, so ranks follow the entries' order and nothing is atomic; an entry's rank among the
// warp's entries of its group waits in pos. Shared memory: counts [warps][E + 1] (bucket E: no group), the CTA's totals,
// the buckets' first rows and the totals of all CTAs [E + 1]. kVpl > 0: choose the experts first (kVpl per lane).
template <int kVpl>
__global__ void __launch_bounds__(kGroupThreads) row_groups_kernel(RouteArgs t, GroupArgs a, int ctas) {
    extern __shared__ int32_t s_counts[];
    __shared__ int32_t s_warp[kGroupWarps];
    griddep_wait();
    griddep_launch_dependents();
    const int B = a.E + 1;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, cta = blockIdx.x;
    int32_t *mine = s_counts + warp * B, *totals = s_counts + kGroupWarps * B, *first = totals + B, *sums = first + B;
    const int64_t T = a.R / a.topk, t_begin = T * cta / ctas, t_end = T * (cta + 1) / ctas;
    for (int i = threadIdx.x; i < kGroupWarps * B; i += kGroupThreads) s_counts[i] = 0;
    if constexpr (kVpl > 0)
        for (int64_t tok = t_begin + warp; tok < t_end; tok += kGroupWarps) route_token<kVpl>(t, tok, lane);
    __syncthreads();
    const int64_t e_begin = t_begin * a.topk, e_end = t_end * a.topk;
    const int64_t piece = ((e_end - e_begin + kGroupWarps - 1) / kGroupWarps + 31) / 32 * 32;
    const int64_t begin = e_begin + warp * piece, end = min(e_end, begin + piece);
    auto bucket = [&](int32_t id) { return id >= 0 && id < a.E ? id : a.E; };
    const int bits = 32 - __clz(a.E);   // of a bucket number
    constexpr int kAhead = 4;           // ids in flight
    for (int64_t i0 = begin; i0 < end; i0 += 32 * kAhead) {
        int32_t id[kAhead];
#pragma unroll
        for (int k = 0; k < kAhead; ++k) id[k] = i0 + 32 * k + lane < end ? __ldcg(a.ids + i0 + 32 * k + lane) : 0;
#pragma unroll
        for (int k = 0; k < kAhead; ++k) {
            const int64_t i = i0 + 32 * k + lane;
            const bool on = i < end;
            const uint32_t live = __ballot_sync(0xffffffffu, on);
            if (on) {
                const int b = bucket(id[k]);
                const uint32_t peers = group_peers(live, b, bits);
                const int32_t before = mine[b];
                a.pos[i] = before + __popc(peers & ((1u << lane) - 1));
                __syncwarp(live);
                if (lane == __ffs(peers) - 1) mine[b] = before + __popc(peers);
            }
            __syncwarp();
        }
    }
    __syncthreads();
    // per bucket: exclusive prefix over the CTA's warps, and the CTA's total
    for (int b = threadIdx.x; b < B; b += kGroupThreads) {
        int32_t sum = 0;
#pragma unroll 8
        for (int w = 0; w < kGroupWarps; ++w) {
            const int32_t c = s_counts[w * B + b];
            s_counts[w * B + b] = sum;
            sum += c;
        }
        totals[b] = sum;
    }
    if (ctas > 1) cluster_sync();
    else __syncthreads();
    // every bucket's entries in the CTAs before this one (below) and in all of them
    for (int b = threadIdx.x; b < B; b += kGroupThreads) {
        int32_t lower = 0, all = ctas > 1 ? 0 : totals[b];
        for (int c0 = 0; ctas > 1 && c0 < ctas; c0 += 8) {
            int32_t v[8];
#pragma unroll
            for (int c = 0; c < 8; ++c)
                asm volatile("ld.shared::cluster.s32 %0, [%1];" : "=r"(v[c]) : "r"(map_to_rank(smem_u32(totals + b), c0 + c)) : "memory");
#pragma unroll
            for (int c = 0; c < 8; ++c) lower += c0 + c < cta ? v[c] : 0, all += v[c];
        }
        first[b] = lower;
        sums[b] = all;
    }
    if (ctas > 1) cluster_arrive();   // done with the others' totals
    __syncthreads();
    const int b = threadIdx.x;
    const int32_t total = b < a.E ? sums[b] : 0;
    int32_t x = total;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const int32_t y = __shfl_up_sync(0xffffffffu, x, d);
        if (lane >= d) x += y;
    }
    if (lane == 31) s_warp[warp] = x;
    __syncthreads();
    if (warp == 0) {
        int32_t y = s_warp[lane];
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const int32_t z = __shfl_up_sync(0xffffffffu, y, d);
            if (lane >= d) y += z;
        }
        s_warp[lane] = y;
    }
    __syncthreads();
    const int32_t base = x - total + (warp > 0 ? s_warp[warp - 1] : 0), live_rows = s_warp[kGroupWarps - 1];
    if (b < a.E) {
        first[b] += base;
        if (cta == 0) a.offsets[b] = base;
    }
    if (threadIdx.x == 0) {   // entries of no group: after the last group
        first[a.E] += live_rows;
        if (cta == 0) a.offsets[a.E] = live_rows;
    }
    __syncthreads();
    for (int64_t i0 = begin; i0 < end; i0 += 32 * kAhead) {
        int32_t id[kAhead], rank[kAhead];
#pragma unroll
        for (int k = 0; k < kAhead; ++k) {
            const int64_t i = i0 + 32 * k + lane;
            if (i < end) {
                id[k] = __ldcg(a.ids + i);
                rank[k] = a.pos[i];   // this thread's own
            }
        }
#pragma unroll
        for (int k = 0; k < kAhead; ++k) {
            const int64_t i = i0 + 32 * k + lane;
            if (i < end) {
                const int bk = bucket(id[k]);
                const int32_t r = first[bk] + mine[bk] + rank[k];
                a.pos[i] = bk < a.E ? r : -1;
                a.row_index[r] = static_cast<int32_t>(static_cast<uint32_t>(i) / static_cast<uint32_t>(a.topk));
            }
        }
    }
    if (ctas > 1) cluster_wait();   // no CTA leaves while its totals are read
}

}  // namespace macaq
