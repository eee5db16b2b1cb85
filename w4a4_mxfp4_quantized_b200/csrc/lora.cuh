// lora.cuh -- low-rank adapters of many requests beside a shared projection.
//
//   out[m, :] = Y[m, :] + scale[a] * (X[m, :] A[a]^T) B[a]^T     for the rows m of adapter a
//
// Bound by HBM: for a prefill by Y in and out, for a decode batch by the active adapters' A and B; for a few rows by latency.
//
// Few rows (kFused): one launch. A cluster of eight CTAs takes a chunk of up to 16 rows of one adapter (rows of no adapter
// are chunks of their own, copied when out is not Y). Each CTA computes the chunk's V = X A^T over an eighth of K, sums the
// cluster's parts of V through distributed shared memory, and adds V B^T to its slice of the columns. With few chunks
// several clusters share one: each makes V for itself and has a part of the columns. While the first product runs the
// CTA's part of B is already on its way into L2.
// Many rows: two launches (kShrink, kExpand) with chunks of 64 rows, because whole clusters of eight leave SMs idle at the
// end of a long launch. The first still has a cluster per chunk, each CTA with its share of K: tiles of X and A come
// through a ring in shared memory, most of a CTA's part at once (4096 wide: 8 tiles, 6 in flight), so that a
// launch of a few microseconds waits for memory once. It ends with V, in the form the second product takes it, in the
// workspace (loads straight to the MMAs, a step ahead, took 5 us more for the 2048 rows below). The second takes
// (chunk, slice of the columns) per CTA without clusters and has its first loads of Y and B under way while the first drains.
// Many adapters, of which few may have rows: grids for every chunk that there could be would mostly be CTAs that find none. There
// the device counts the chunks and each CTA works out its chunk and slice from that.
//
// The other products are bf16 MMAs (m16n8k16) fed straight from global memory: lane (g, t) takes 16 bytes, 8 neighbouring k of
// row g at 8 t of a 32-wide k step, and the two MMAs of the step take their halves; both operands use the same order, so
// the sum over k is complete. In the second product the 32 columns of a step are dealt to the four n8 tiles so that a lane
// ends up with 8 neighbouring columns of a row: Y moves in 16-byte pieces, through a ring of cp.async stages in which each
// lane reads back what it copied itself (no barrier; the copies of the next steps are in flight while one is added). V is held in
// two or three bf16 parts (16 or 24 bits).
// Measured on B200 (4096 -> 14336, a graph that cycles three batches): one row of rank 16 5.5 us; 64 rows over 32 adapters of
// rank 16 12.3 us (19.7 MB; find 1.0, V 1.9, cluster sum 2.0, columns 5 us); 2048 rows of 4 adapters of rank 64 46.4 us
// (142 MB, 3.1 TB/s: 12 us for V, most of it starts and the cluster's sum, and the rest for the columns, whose warps wait on one
// another's MMAs, twice as many for V's two parts, shared memory and stores rather than on HBM), of rank 128 80 us, in fp32
// 89 us. 2048 rows of 4 active adapters of rank 64 in banks of 4, 64, 256 and 1024: 49.8, 50.9, 53.3 and 58.7 us (two batches).
#pragma once

#include <cuda_bf16.h>

#include "groups.cuh"
#include "moe_w4a16.cuh"
#include "ptx.cuh"
#include "route.cuh"

namespace macaq {

constexpr int kLoraThreads = 256;
constexpr int kLoraWarps = kLoraThreads / 32;
constexpr int kLoraCluster = 8;
constexpr int kLoraMaxRank = 128;
constexpr int kLoraShrinkBytes = 96 * 1024;
enum LoraMode { kFused, kShrink, kExpand };
__host__ __device__ constexpr int lora_tiles(LoraMode mode) { return mode == kFused ? 1 : 4; }   // m16 tiles of a chunk

struct LoraArgs {
    const void *y;            // [M, N], rows ldy apart
    void *out;                // [M, N], rows ldo apart
    const uint16_t *x;        // bf16 [M, K], rows ldx apart
    const uint16_t *A;        // bf16 [L, r, K]
    const uint16_t *B;        // bf16 [L, N, r]
    const float *scale;       // [L] or nullptr
    const int32_t *offsets;   // [L + 1]
    const int32_t *row_index; // [M] or nullptr: rows are sorted already
    int64_t ldy, ldo, ldx, M, N, K;
    int32_t r, L;
    uint16_t *v;              // workspace (two launches): V per chunk, [part][row][stride]
    int32_t slices;           // CTAs per chunk, each with its slice of the columns; 0: by the number of chunks that there are
    int32_t chunks;           // the most that a sound plan has
    int32_t room;             // CTAs of one round
};

// Shared memory for rank r, chunks of 16 mt rows and `parts` bf16 parts of V: the CTA's partial V per k split, its sum, the
// parts of V. The parts' rows have the rank of the kernel that serves r (32 kSteps), zero from r on.
__host__ __device__ constexpr int lora_padded_rank(int r) { return r <= 32 ? 32 : (r <= 64 ? 64 : 128); }
__host__ __device__ constexpr int lora_v_stride(int r) {   // bf16; 64 bytes off a multiple of 128: no bank conflicts
    return lora_padded_rank(r) == 32 ? 32 : lora_padded_rank(r) + 32;
}
// bf16 parts that V is held in: three for fp32 outputs (off by at most 2^-24 of a value), two for bf16 outputs (2^-16), in both
// forms alike, so that a row's result does not go by the rows beside it. What that leaves in an output is 2^-16 of the sum of
// |V_j B_j|, also where Y or the terms cancel; one part would leave 2^-8 of it.
__host__ __device__ constexpr int lora_parts(bool f32) { return f32 ? 3 : 2; }
__host__ __device__ constexpr int lora_v_bytes(int r, int mt, int parts) { return parts * 16 * mt * lora_v_stride(r) * 2; }
// The ring of the second product: 16-byte pieces per lane and stage (Y of all rows; for one m16 tile B too), and stages.
__host__ __device__ constexpr int lora_ring_pieces(int mt, int steps, bool f32) {
    return mt * 2 * (f32 ? 2 : 1) + (mt == 1 ? 4 * steps : 0);
}
__host__ __device__ constexpr int lora_ring_stages(int mt, int steps, bool f32) { return mt == 1 && steps == 1 ? (f32 ? 3 : 4) : 2; }
__host__ __device__ constexpr int lora_ring_bytes(int mt, int steps, bool f32) {
    return kLoraWarps * lora_ring_stages(mt, steps, f32) * lora_ring_pieces(mt, steps, f32) * 512;
}
// kShrink: tiles of 64 k of the chunk's 64 rows of X and of A's rows, two CTAs' stages to an SM.
__host__ __device__ constexpr int lora_shrink_stage(int steps) { return (64 + 32 * steps) * 128; }
__host__ __device__ constexpr int lora_shrink_stages(int steps) { return kLoraShrinkBytes / lora_shrink_stage(steps); }
// Offsets, kFused: [ring, over the partial sums][the CTA's sum][parts of V]; kExpand: [ring][parts of V]; kShrink: [ring, under
// the CTA's sum in the end]
__host__ __device__ constexpr int lora_sum_offset(int r, int steps, bool f32) {
    const int part = kLoraWarps * 16 * r * 4, ring = lora_ring_bytes(1, steps, f32);
    return part > ring ? part : ring;
}
__host__ __device__ constexpr int lora_v_offset(int r, int steps, bool f32, LoraMode mode) {
    return mode == kFused ? lora_sum_offset(r, steps, f32) + 16 * r * 4 : lora_ring_bytes(4, steps, f32);
}
__host__ __device__ constexpr int lora_smem_bytes(int r, int steps, bool f32, LoraMode mode) {
    if (mode == kShrink) return lora_shrink_stages(steps) * lora_shrink_stage(steps);
    return lora_v_offset(r, steps, f32, mode) + lora_v_bytes(r, lora_tiles(mode), lora_parts(f32));
}

__device__ __forceinline__ void lora_copy16(uint32_t dst, const void *src, bool on) {   // off: zeros
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(on ? 16 : 0) : "memory");
}

__device__ __forceinline__ void mma_bf16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint4 lora_ld(const uint16_t *p, bool on) {
    return on ? __ldg(reinterpret_cast<const uint4 *>(p)) : make_uint4(0u, 0u, 0u, 0u);
}

// Chunks of up to `most` rows; rows < 2^31, so nothing is added to them.
__host__ __device__ constexpr int32_t lora_chunk_count(int32_t rows, int32_t most) { return rows / most + (rows % most != 0); }

struct LoraChunk {
    int32_t a, rows;   // adapter (L: rows of no adapter), rows; rows = 0: there is no such chunk
    int64_t row0;
};

// Chunk z of the plan: ceil(rows / most) of them per adapter, the rows of none as one more group at the end. Offsets are
// clamped into [0, M]. Every warp finds the same; s_off holds the offsets.
__device__ __forceinline__ LoraChunk lora_find_chunk(const LoraArgs &p, int z, int most, int32_t *s_off) {
    const int lane = threadIdx.x & 31;
    for (int i = threadIdx.x; i <= p.L; i += kLoraThreads)
        s_off[i] = static_cast<int32_t>(min(max(static_cast<int64_t>(__ldcg(p.offsets + i)), int64_t{0}), p.M));
    if (threadIdx.x == 0) s_off[p.L + 1] = static_cast<int32_t>(p.M);
    __syncthreads();
    LoraChunk ch{0, 0, 0};
    int64_t before = 0;
#pragma unroll 1
    for (int base = 0; base <= p.L; base += 32) {
        const int g = base + lane;
        const int32_t lo = g <= p.L ? s_off[g] : 0, rows = g <= p.L ? max(s_off[g + 1] - lo, 0) : 0;
        const int32_t n = lora_chunk_count(rows, most);
        int32_t x = n;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const int32_t y = __shfl_up_sync(0xffffffffu, x, d);
            if (lane >= d) x += y;
        }
        const int64_t at = before + x - n;
        const uint32_t hit = __ballot_sync(0xffffffffu, z >= at && z < at + n);
        if (hit != 0) {
            const int src = __ffs(hit) - 1;
            const int32_t skip = static_cast<int32_t>(z - __shfl_sync(0xffffffffu, at, src)) * most;
            ch.a = base + src;
            ch.row0 = static_cast<int64_t>(__shfl_sync(0xffffffffu, lo, src)) + skip;
            ch.rows = min(__shfl_sync(0xffffffffu, rows, src) - skip, most);
            break;
        }
        before += __shfl_sync(0xffffffffu, x, 31);
    }
    return ch;
}

// The numbers of all groups' first chunks: first[g], and of all chunks first[L + 1]. Thread i has the groups from i * per on.
// s_sum: one entry per warp.
__device__ __forceinline__ void lora_scan_chunks(const LoraArgs &p, int most, int32_t *first, int64_t *s_sum) {
    constexpr int kPer = (kRouteMaxExperts + 1 + kLoraThreads - 1) / kLoraThreads;
    constexpr int64_t kTop = (int64_t{1} << 31) - 1;   // of a plan that lists rows many times
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, per = (p.L + kLoraThreads) / kLoraThreads, g0 = threadIdx.x * per;
    int32_t off[kPer + 1], n[kPer];
#pragma unroll
    for (int i = 0; i <= kPer; ++i)
        off[i] = g0 + i > p.L ? static_cast<int32_t>(p.M)
                              : static_cast<int32_t>(min(max(static_cast<int64_t>(__ldcg(p.offsets + g0 + i)), int64_t{0}), p.M));
    int64_t sum = 0;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
        n[i] = i < per && g0 + i <= p.L ? lora_chunk_count(max(off[i + 1] - off[i], 0), most) : 0;
        sum += n[i];
    }
    int64_t x = sum;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const int64_t y = __shfl_up_sync(0xffffffffu, x, d);
        if (lane >= d) x += y;
    }
    if (lane == 31) s_sum[warp] = x;
    __syncthreads();
    int64_t at = x - sum;
    for (int w = 0; w < warp; ++w) at += s_sum[w];
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
        if (i >= per || g0 + i > p.L) break;
        first[g0 + i] = static_cast<int32_t>(min(at, kTop));
        at += n[i];
        if (g0 + i == p.L) first[p.L + 1] = static_cast<int32_t>(min(at, kTop));
    }
    __syncthreads();
}

// Chunk z from those numbers.
__device__ __forceinline__ LoraChunk lora_chunk_at(const LoraArgs &p, int z, int most, const int32_t *first) {
    int a = 0;   // the last group whose first chunk is not after z
    for (int end = p.L + 1; end - a > 1;) {
        const int mid = (a + end) / 2;
        if (first[mid] <= z) a = mid;
        else end = mid;
    }
    auto offset = [&](int i) { return i > p.L ? p.M : min(max(static_cast<int64_t>(__ldcg(p.offsets + i)), int64_t{0}), p.M); };
    const int64_t lo = offset(a), skip = static_cast<int64_t>(z - first[a]) * most;
    return {a, static_cast<int32_t>(min(max(offset(a + 1) - lo - skip, int64_t{0}), static_cast<int64_t>(most))), lo + skip};
}

// Eight neighbouring outputs of a row: out = y + d.
template <bool kF32>
struct LoraPiece {
    uint4 v[kF32 ? 2 : 1];
    __device__ __forceinline__ void load(const char *y, bool on) {
        if (!on) return;
#pragma unroll
        for (int i = 0; i < (kF32 ? 2 : 1); ++i) v[i] = __ldcg(reinterpret_cast<const uint4 *>(y) + i);
    }
    // columns 2 i and 2 i + 1: what their sums start from, and their results
    __device__ __forceinline__ void start(int i, float &a, float &b) const {
        if constexpr (kF32) {
            a = b = 0.0f;
        } else {
            const uint32_t w = reinterpret_cast<const uint32_t *>(v)[i];
            a = __uint_as_float(w << 16), b = __uint_as_float(w & 0xFFFF0000u);
        }
    }
    __device__ __forceinline__ void finish(int i, float a, float b) {
        uint32_t *w = reinterpret_cast<uint32_t *>(v);
        if constexpr (kF32) {
            w[2 * i] = __float_as_uint(__uint_as_float(w[2 * i]) + a);
            w[2 * i + 1] = __float_as_uint(__uint_as_float(w[2 * i + 1]) + b);
        } else {
            const __nv_bfloat162 o = __floats2bfloat162_rn(a, b);
            w[i] = *reinterpret_cast<const uint32_t *>(&o);
        }
    }
    __device__ __forceinline__ void store(char *out, bool on) const {
        if (!on) return;
#pragma unroll
        for (int i = 0; i < (kF32 ? 2 : 1); ++i) reinterpret_cast<uint4 *>(out)[i] = v[i];
    }
};

// Grid: `slices` CTAs per chunk: clusters of eight (kFused), one cluster of 1 to 8 (kShrink), without clusters (kExpand).
// slices = 0, for calls whose adapters may mostly have no rows: a CTA for every chunk that there can be, and for one round at
// least, in clusters of eight; the device counts the chunks and gives each as many neighbouring CTAs as that leaves, up to a
// cluster's eight (then whole clusters) for V. kSteps: 32-wide steps of the rank.
template <int kSteps, bool kF32, LoraMode kMode>
__global__ void __launch_bounds__(kLoraThreads, 2) lora_add_kernel(LoraArgs p) {
    constexpr int kMt = lora_tiles(kMode);   // m16 tiles of a chunk
    constexpr int kRows = 16 * kMt, kParts = lora_parts(kF32), kElement = kF32 ? 4 : 2;
    extern __shared__ __align__(16) uint8_t s_lora[];
    __shared__ int32_t s_off[kRouteMaxExperts + 2];
    __shared__ const uint16_t *s_x[kRows];   // the rows' places in X, Y and out, null for none
    __shared__ const char *s_y[kRows];
    __shared__ char *s_out[kRows];
    // The first launch of two waits for everything before it and only then lets the second start, so the plan, Y and B are
    // complete for both; the second waits for V.
    if constexpr (kMode != kExpand) griddep_wait();
    griddep_launch_dependents();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, t = lane & 3;
    int cluster = kMode == kFused ? kLoraCluster : p.slices;   // CTAs that make a chunk's V: a power of two
    int slices = p.slices, rank, first_rank = 0, z, slice;
    LoraChunk ch{0, 0, 0};
    if (slices > 0) {
        rank = blockIdx.x & (cluster - 1), z = blockIdx.x / slices, slice = blockIdx.x % slices;
        ch = lora_find_chunk(p, z, kRows, s_off);
    } else {
        __shared__ int64_t s_sum[kLoraWarps];
        lora_scan_chunks(p, kRows, s_off, s_sum);
        const int steps = static_cast<int>((p.N + 31) / 32);
        const int chunks = min(s_off[kMode == kShrink || p.out == p.y ? p.L : p.L + 1], p.chunks);   // rows of no adapter: copied
        cluster = kMode == kExpand ? 1 : kLoraCluster;
        while (cluster > 1 && chunks > p.room / cluster) cluster /= 2;
        const int share = kMode == kShrink ? 1 : max(1, min(p.room / (cluster * max(chunks, 1)), steps / (kLoraWarps * cluster)));
        slices = share * cluster;
        rank = blockIdx.x & (cluster - 1), z = blockIdx.x / slices, slice = blockIdx.x % slices;
        first_rank = (blockIdx.x & (kLoraCluster - 1)) - rank;
        if (z < chunks) ch = lora_chunk_at(p, z, kRows, s_off);
    }
    // A CTA without work: the same for all of a chunk's CTAs, but others of the cluster may have some (slices = 0)
    auto leave = [&]() {
        if constexpr (kMode == kExpand) {
            griddep_wait();
        } else if (p.slices == 0) {
            cluster_sync();
            cluster_sync();
        }
    };
    if (ch.rows == 0 || (ch.a == p.L && (kMode == kShrink || p.out == p.y))) {
        leave();
        return;
    }
    const int log2_cluster = 31 - __clz(cluster);
    const int r = p.r;
    // this CTA's columns, in steps of 32, and k, in steps of 32 or 64
    const int64_t nsteps = (p.N + 31) / 32, n_begin = nsteps * slice / slices, n_end = nsteps * (slice + 1) / slices;
    constexpr int kWide = kMode == kShrink ? 64 : 32;
    const int64_t ksteps = (p.K + kWide - 1) / kWide, k_begin = ksteps * rank >> log2_cluster, k_end = ksteps * (rank + 1) >> log2_cluster;
    for (int i = threadIdx.x; i < kRows; i += kLoraThreads) {
        int64_t m = -1;
        if (i < ch.rows) m = p.row_index ? static_cast<int64_t>(__ldcg(p.row_index + ch.row0 + i)) : ch.row0 + i;
        const bool on = m >= 0 && m < p.M;
        s_x[i] = on ? p.x + m * p.ldx : nullptr;
        s_y[i] = on ? static_cast<const char *>(p.y) + m * p.ldy * kElement : nullptr;
        s_out[i] = on ? static_cast<char *>(p.out) + m * p.ldo * kElement : nullptr;
    }
    __syncthreads();

    if (ch.a == p.L) {   // rows of no adapter
        leave();         // kExpand: out may still be in use
        // a warp per row, eight pieces of it in flight
        constexpr int kAhead = 8;
        const int64_t stop = min(n_end * 32, p.N);
        for (int row = warp; row < ch.rows; row += kLoraWarps) {
            if (s_y[row] == nullptr) continue;
            for (int64_t n = n_begin * 32 + 8 * lane; n < stop; n += 256 * kAhead) {
                LoraPiece<kF32> y[kAhead];
#pragma unroll
                for (int k = 0; k < kAhead; ++k) y[k].load(s_y[row] + (n + 256 * k) * kElement, n + 256 * k < stop);
#pragma unroll
                for (int k = 0; k < kAhead; ++k) y[k].store(s_out[row] + (n + 256 * k) * kElement, n + 256 * k < stop);
            }
        }
        return;
    }

    const uint16_t *A = p.A + static_cast<int64_t>(ch.a) * r * p.K, *B = p.B + static_cast<int64_t>(ch.a) * p.N * r;
    float *part = reinterpret_cast<float *>(s_lora);                                                   // [split][row][r]
    float *mine = reinterpret_cast<float *>(s_lora + (kMode == kFused ? lora_sum_offset(r, kSteps, kF32) : 0));  // [row][r]
    const int vs = lora_v_stride(r);
    uint16_t *v_s = reinterpret_cast<uint16_t *>(s_lora + lora_v_offset(r, kSteps, kF32, kMode));      // [part][row][vs]
    if constexpr (kMode == kFused) {   // this CTA's part of B, towards L2
        const char *from = reinterpret_cast<const char *>(B + n_begin * 32 * r);
        const int64_t bytes = (min(n_end * 32, p.N) - n_begin * 32) * r * 2;
        for (int64_t i = threadIdx.x * 128; i < bytes; i += kLoraThreads * 128)
            asm volatile("prefetch.global.L2 [%0];" ::"l"(from + i));
    }

    if constexpr (kMode == kFused) {
        // V = X A^T: a warp takes every eighth k step of the CTA's part
        constexpr int kTiles = kSteps == 1 ? 4 : 8;   // n8 tiles of V at a time
        for (int j0 = 0; j0 < r; j0 += 8 * kTiles) {
            float acc[kTiles][4] = {};
            int k = static_cast<int>(k_begin + warp) * 32 + 8 * t;   // this lane's first
            const int k_stop = static_cast<int>(min(k_end * 32, p.K));
            const uint16_t *a_row[kTiles], *x_row[2];
#pragma unroll
            for (int j = 0; j < kTiles; ++j) a_row[j] = j0 + 8 * j < r ? A + (j0 + 8 * j + g) * p.K + k : nullptr;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const uint16_t *row = s_x[8 * h + g];
                x_row[h] = row == nullptr ? nullptr : row + k;
            }
            uint4 x[2];
            auto load_x = [&](bool on) {
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    x[h] = lora_ld(x_row[h], on && x_row[h] != nullptr);
                    if (x_row[h] != nullptr) x_row[h] += 32 * kLoraWarps;
                }
            };
            load_x(k < k_stop);
#pragma unroll 1
            for (int s = static_cast<int>(k_begin) + warp; s < static_cast<int>(k_end); s += kLoraWarps) {
                uint4 b[kTiles];
#pragma unroll
                for (int j = 0; j < kTiles; ++j) {
                    b[j] = lora_ld(a_row[j], k < k_stop && a_row[j] != nullptr);
                    if (a_row[j] != nullptr) a_row[j] += 32 * kLoraWarps;
                }
                const uint4 lo = x[0], hi = x[1];
                k += 32 * kLoraWarps;
                load_x(k < k_stop);   // the next step's rows of X, from further away than A
#pragma unroll
                for (int j = 0; j < kTiles; ++j) {
                    if (j0 + 8 * j >= r) break;
                    mma_bf16(acc[j], lo.x, hi.x, lo.y, hi.y, b[j].x, b[j].y);
                    mma_bf16(acc[j], lo.z, hi.z, lo.w, hi.w, b[j].z, b[j].w);
                }
            }
#pragma unroll
            for (int j = 0; j < kTiles; ++j)
                if (j0 + 8 * j < r) {
                    float *dst = part + (warp * kRows + g) * r + j0 + 8 * j + 2 * t;
                    *reinterpret_cast<float2 *>(dst) = make_float2(acc[j][0], acc[j][1]);
                    *reinterpret_cast<float2 *>(dst + 8 * r) = make_float2(acc[j][2], acc[j][3]);
                }
        }
        // the parts of V are zero where nothing is written: past r, and in rows past the chunk's
        for (int i = threadIdx.x; i < lora_v_bytes(r, kMt, kParts) / 16; i += kLoraThreads)
            reinterpret_cast<uint4 *>(v_s)[i] = make_uint4(0u, 0u, 0u, 0u);
        __syncthreads();
        for (int i = threadIdx.x; i < ch.rows * r; i += kLoraThreads) {
            float v = 0.0f;
#pragma unroll
            for (int s = 0; s < kLoraWarps; ++s) v += part[s * kRows * r + i];
            mine[i] = v;
        }
    }
    if constexpr (kMode == kShrink) {
        // V = X A^T: tiles of 64 k of both operands through a ring in shared memory, rows of 128 bytes whose 16-byte pieces are
        // exchanged by row % 8. A warp has one m16 tile of the rows and half of the rank.
        constexpr int kStages = lora_shrink_stages(kSteps), kStage = lora_shrink_stage(kSteps), kTiles = 2 * kSteps;
        const uint32_t ring = smem_u32(s_lora);
        const int piece = threadIdx.x & 7, row = threadIdx.x >> 3;   // this thread copies this piece of every 32nd row
        const uint16_t *x_row[2] = {s_x[row], s_x[row + 32]}, *a_row = A + static_cast<int64_t>(row) * p.K;
        const int64_t a_step = 32 * p.K;
        auto issue = [&](int64_t step, int stage) {
            if (step < k_end) {
                const int64_t k = step * 64 + 8 * piece;
                const bool in = k < p.K;
                const uint32_t dst = ring + stage * kStage + row * 128 + ((piece ^ (row & 7)) << 4);
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const bool on = in && x_row[i] != nullptr;
                    lora_copy16(dst + i * 4096, on ? x_row[i] + k : p.x, on);
                }
#pragma unroll
                for (int i = 0; i < kSteps; ++i) {
                    const bool on = in && row + 32 * i < r;
                    lora_copy16(dst + 8192 + i * 4096, on ? a_row + i * a_step + k : A, on);
                }
            }
            cp_async_commit();   // an empty group keeps groups and stages in step
        };
#pragma unroll
        for (int i = 0; i < kStages - 1; ++i) issue(k_begin + i, i);
        const int mt = warp % 4, tile0 = warp / 4 * kTiles;
        const uint32_t x_at = ring + (16 * mt + (lane & 15)) * 128, a_at = ring + 8192 + (8 * tile0 + 8 * (lane >> 4) + (lane & 7)) * 128;
        float acc[kTiles][4] = {};
        int stage = 0;
#pragma unroll 1
        for (int64_t step = k_begin; step < k_end; ++step) {
            cp_async_wait<kStages - 2>();
            __syncthreads();   // the step's tiles are complete, and nobody reads those of the step before
            issue(step + kStages - 1, stage == 0 ? kStages - 1 : stage - 1);
            if (16 * mt < ch.rows) {
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    uint32_t x[4];
                    ldmatrix_x4(x, x_at + stage * kStage + (((2 * c + (lane >> 4)) ^ (lane & 7)) << 4));
#pragma unroll
                    for (int j = 0; j < kTiles; j += 2) {
                        uint32_t b[4];
                        ldmatrix_x4(b, a_at + stage * kStage + j * 1024 + (((2 * c + ((lane >> 3) & 1)) ^ (lane & 7)) << 4));
                        mma_bf16(acc[j], x[0], x[1], x[2], x[3], b[0], b[1]);
                        mma_bf16(acc[j + 1], x[0], x[1], x[2], x[3], b[2], b[3]);
                    }
                }
            }
            stage = stage == kStages - 1 ? 0 : stage + 1;
        }
        __syncthreads();   // the sums lie over the ring
#pragma unroll
        for (int j = 0; j < kTiles; ++j)
            if (8 * (tile0 + j) < r) {
                float *dst = mine + (16 * mt + g) * r + 8 * (tile0 + j) + 2 * t;
                *reinterpret_cast<float2 *>(dst) = make_float2(acc[j][0], acc[j][1]);
                *reinterpret_cast<float2 *>(dst + 8 * r) = make_float2(acc[j][2], acc[j][3]);
            }
    }
    // The second product's loads. A warp takes every eighth 32-column step; the first copies set out here, before V is complete.
    // Logical column c of n8 tile i is column 8 (c / 2) + 2 i + c % 2 of the step.
    constexpr int kStages = lora_ring_stages(kMt, kSteps, kF32), kPieces = lora_ring_pieces(kMt, kSteps, kF32);
    constexpr int kYPieces = kF32 ? 2 : 1;   // of a lane's eight columns
    const int N = static_cast<int>(p.N), s_end = static_cast<int>(n_end), n_lane = 8 * (g >> 1) + (g & 1);
    int s = static_cast<int>(n_begin) + warp;
    const uint16_t *b_lane = B + static_cast<int64_t>(n_lane) * r + 8 * t;
    uint8_t *ring = s_lora + (warp * kStages * kPieces * 32 + lane) * 16;   // this lane's piece 0 of stage 0
    uint32_t k_on = 0;   // steps of the rank that this lane has
#pragma unroll
    for (int ks = 0; ks < kSteps; ++ks) k_on |= 32 * ks + 8 * t < r ? 1u << ks : 0u;
    auto b_on = [&](int step, int ks, int i) { return step < s_end && step * 32 + n_lane + 2 * i < N && ((k_on >> ks) & 1); };
    auto b_at = [&](int step, int ks, int i) { return b_lane + (static_cast<int64_t>(step) * 32 + 2 * i) * r + 32 * ks; };
    auto issue = [&](int step, int stage) {
        const uint32_t dst = smem_u32(ring) + stage * kPieces * 512;
        if (step < s_end) {
#pragma unroll
            for (int k = 0; k < 2 * kMt; ++k) {
                if (kMt == 1 && 8 * k >= ch.rows) break;
                const int row = 8 * k + g;
                const char *src = s_y[row];
                if (src != nullptr && step * 32 + 8 * t < N) {
                    src += (step * 32 + 8 * t) * kElement;
#pragma unroll
                    for (int c = 0; c < kYPieces; ++c) lora_copy16(dst + (k * kYPieces + c) * 512, src + 16 * c, true);
                }
            }
            if constexpr (kMt == 1) {
#pragma unroll
                for (int k = 0; k < 4 * kSteps; ++k) {
                    const bool on = b_on(step, k / 4, k % 4);
                    lora_copy16(dst + (2 * kYPieces + k) * 512, on ? b_at(step, k / 4, k % 4) : B, on);
                }
            }
        }
        cp_async_commit();   // an empty group keeps groups and steps in step
    };
    uint4 b[kSteps][4];   // a second set for the next step's, loaded ahead, cost registers and time (2048 rows: 5 us)
    auto load_b = [&](int step, uint4 (&to)[kSteps][4]) {
#pragma unroll
        for (int ks = 0; ks < kSteps; ++ks)
#pragma unroll
            for (int i = 0; i < 4; ++i) to[ks][i] = lora_ld(b_at(step, ks, i), b_on(step, ks, i));
    };
    if constexpr (kMode != kShrink) {
        if constexpr (kMode == kFused) __syncthreads();   // the partial sums are read: the ring lies over them
#pragma unroll
        for (int k = 0; k < kStages - 1; ++k) issue(s + k * kLoraWarps, k);
        if constexpr (kMt > 1) load_b(s, b);
    }
    if constexpr (kMode != kExpand) {
        // Entries in pairs: sum over the cluster, times scale, in bf16 parts. A chunk of 16 rows is small enough for every CTA to
        // sum all of it for itself; of 64 rows each sums its share, for the workspace.
        constexpr bool kAll = kMode == kFused;
        cluster_sync();
        const float scale = p.scale ? __ldg(p.scale + ch.a) : 1.0f;
        const int pairs = (kAll ? ch.rows : kRows) * r / 2, at0 = kAll ? 0 : rank * pairs >> log2_cluster,
                  at1 = kAll ? pairs : (rank + 1) * pairs >> log2_cluster;
        for (int i = at0 + threadIdx.x; i < at1; i += kLoraThreads) {
            float a0[kLoraCluster], a1[kLoraCluster], v0 = 0.0f, v1 = 0.0f;
#pragma unroll
            for (int c = 0; c < kLoraCluster; ++c) {
                a0[c] = a1[c] = 0.0f;
                if (c >= cluster) continue;
                asm volatile("ld.shared::cluster.v2.f32 {%0, %1}, [%2];"
                             : "=f"(a0[c]), "=f"(a1[c])
                             : "r"(map_to_rank(smem_u32(mine + 2 * i), first_rank + c))
                             : "memory");
            }
#pragma unroll
            for (int c = 0; c < kLoraCluster; ++c) v0 += a0[c], v1 += a1[c];
            v0 *= scale, v1 *= scale;
            const int row = 2 * i / r, col = 2 * i - row * r;
#pragma unroll
            for (int k = 0; k < kParts; ++k) {   // each part is the rounding of what the ones before leave
                const __nv_bfloat162 b = __floats2bfloat162_rn(v0, v1);
                const uint32_t w = *reinterpret_cast<const uint32_t *>(&b);
                const float h0 = __uint_as_float(w << 16), h1 = __uint_as_float(w & 0xFFFF0000u);
                v0 = isinf(h0) ? 0.0f : v0 - h0, v1 = isinf(h1) ? 0.0f : v1 - h1;   // an infinity stays one
                const int at = (k * kRows + row) * vs + col;
                if constexpr (kAll) *reinterpret_cast<uint32_t *>(v_s + at) = w;
                else *reinterpret_cast<uint32_t *>(p.v + static_cast<int64_t>(z) * kParts * kRows * vs + at) = w;
            }
        }
        if constexpr (kAll) {
            cluster_arrive();   // waited for at the end
            __syncthreads();
        } else {
            cluster_sync();   // no CTA leaves while another reads its sums
        }
        if constexpr (kMode == kShrink) return;
    } else {
        griddep_wait();
        const uint4 *src = reinterpret_cast<const uint4 *>(p.v + static_cast<int64_t>(z) * kParts * kRows * vs);
        const int per_row = vs / 8;
        for (int i = threadIdx.x; i < kParts * kRows * per_row; i += kLoraThreads) {
            uint4 w = __ldcg(src + i);
            if (i % per_row * 8 >= r) w = make_uint4(0u, 0u, 0u, 0u);   // past the rank nothing was written
            reinterpret_cast<uint4 *>(v_s)[i] = w;
        }
        __syncthreads();
    }

    // out = Y + V B^T, all rows of 32 columns at a time, tile by tile of 16 rows
    int stage = 0;
#pragma unroll 1
    for (; s < s_end; s += kLoraWarps) {
        issue(s + (kStages - 1) * kLoraWarps, stage == 0 ? kStages - 1 : stage - 1);
        cp_async_wait<kStages - 1>();   // this lane's copies of the step have landed
        const uint4 *piece = reinterpret_cast<const uint4 *>(ring + stage * kPieces * 512);
        stage = stage == kStages - 1 ? 0 : stage + 1;
        if constexpr (kMt == 1) {
#pragma unroll
            for (int k = 0; k < 4 * kSteps; ++k) b[k / 4][k % 4] = piece[(2 * kYPieces + k) * 32];
        }
#pragma unroll
        for (int mt = 0; mt < kMt; ++mt) {
            if (16 * mt >= ch.rows) break;
            // For bf16 the sums start from Y. For fp32 Y is added last, once: an MMA that adds to it would cut at its last bit
            // every time.
            LoraPiece<kF32> y[2];
            float acc[4][4] = {};
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                if (kMt == 1 && h == 1 && ch.rows <= 8) break;   // rows 8 .. 15: none (their sums are not looked at)
#pragma unroll
                for (int c = 0; c < kYPieces; ++c) y[h].v[c] = piece[((2 * mt + h) * kYPieces + c) * 32];
#pragma unroll
                for (int i = 0; i < 4; ++i) y[h].start(i, acc[i][2 * h], acc[i][2 * h + 1]);
            }
#pragma unroll
            for (int ks = 0; ks < kSteps; ++ks)
#pragma unroll
                for (int q = 0; q < kParts; ++q) {
                    const uint16_t *v = v_s + (q * kRows + 16 * mt + g) * vs + 32 * ks + 8 * t;
                    const uint4 lo = *reinterpret_cast<const uint4 *>(v), hi = *reinterpret_cast<const uint4 *>(v + 8 * vs);
#pragma unroll
                    for (int i = 0; i < 4; ++i) mma_bf16(acc[i], lo.x, hi.x, lo.y, hi.y, b[ks][i].x, b[ks][i].y);
#pragma unroll
                    for (int i = 0; i < 4; ++i) mma_bf16(acc[i], lo.z, hi.z, lo.w, hi.w, b[ks][i].z, b[ks][i].w);
                }
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                if (kMt == 1 && h == 1 && ch.rows <= 8) break;
#pragma unroll
                for (int i = 0; i < 4; ++i) y[h].finish(i, acc[i][2 * h], acc[i][2 * h + 1]);
                char *dst = s_out[16 * mt + 8 * h + g];
                y[h].store(dst + (s * 32 + 8 * t) * kElement, dst != nullptr && s * 32 + 8 * t < N);
            }
        }
        if constexpr (kMt > 1) load_b(s + kLoraWarps, b);
    }
    if constexpr (kMode == kFused) {
        cluster_wait();   // no CTA leaves while another reads its sums
    }
}

}  // namespace macaq
