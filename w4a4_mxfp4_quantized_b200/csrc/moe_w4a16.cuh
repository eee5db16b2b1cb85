// moe_w4a16.cuh -- a whole mixture-of-experts layer for few tokens: MXFP4 weights, bf16 activations.
//
//   x'  = x diag(1/s_e) H_b                        (fp32 butterflies; the weight-only mode's transform)
//   g, u = gate and up rows of x' dq(W'_gu,e)^T    (64-row interleaved blocks)
//   h   = silu(g) u,  h' = h diag(1/s_down,e) H_b'
//   out[t] = sum_j weights[t, j] * (h'_{pos[t, j]} dq(W'_down,e)^T)
//
// Bound by HBM: every active expert's codes and scales are read once (17/32 byte a weight), and an expert has a handful of
// rows, so the two products are streams of weights against a small operand that stays in shared memory.
//
// Plan. The rows of an expert are cut into chunks of up to 8 or 16 (8 when experts average four rows or fewer, so that
// one n8 tile nearly always does). Kernel 1 takes (chunk, 128 intermediate channels), kernel 2 (chunk, 128 output
// channels); a cluster of CTAs may share one such block, each with a part of the K tiles (128 channels), and adds its
// partial sums through distributed shared memory. A CTA keeps its rows' operand as fp16 in shared memory (the
// panel). Each warp streams 32 weight rows (8 rows g of each of the four 32-row quarters of a scale tile, so one
// 16-byte scale chunk serves a lane's four rows) through its own ring of cp.async stages: no barrier between warps.
//
// Arithmetic. m16n8k16 fp16 MMAs with weights as the 16-row operand: a lane's 32-bit word of a row (8 codes of
// one MX group) becomes four fp16 pairs with one conversion instruction each, exactly, and needs no pass through shared or
// tensor memory; tcgen05 would need the codes expanded there first. ldmatrix hands lane (g, t) word t of row g, so
// the K order inside a group is the codes' own and the operand panel is read 16 bytes at a time. Each group's two
// MMAs start from zero and their fp32 sums are scaled by the group's 2^(E - 127) as they are added: scales never
// touch fp16. The panel holds, per row and 32 channels, fp16(x' s) with s a power of two: 1 when the group's largest
// value is in [2^-10, 2^15), else what brings it there. A tile whose groups all have s = 1 (the usual case) is added
// without looking at them; otherwise 1/s joins the weights' scale of the group. fp16's 11 bits round x' and h' 8 times
// finer than the output's bf16.
//
// Kernel 2 starts (programmatic launch) while kernel 1 drains: its CTAs find their chunk and fill their rings with weights,
// which no kernel in flight writes, before they wait for kernel 1's rows. A token's choices are
// added in the order j = 0, 1, ... by the CTA that writes the last of their rows (a counter per token and 128 outputs,
// zeroed by kernel 1), so results do not depend on timing.
// Sources: glonce.com page on MACaQ, paragraph 3 (weight-only serving) and paragraph 5 (grouped matmul);
// aipolix.com page, paragraph 2 (the transform at the input of every linear).
#pragma once

#include <cooperative_groups.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "groups.cuh"
#include "ptx.cuh"
#include "quant.cuh"
#include "route.cuh"

namespace macaq {

constexpr int kMoeMaxT = 64;
constexpr int kMoeThreads = 256;
constexpr int kMoeWarps = kMoeThreads / 32;
constexpr int kMoeStages = 3;
constexpr int kMoeStageBytes = 2048 + 128;  // 32 rows x 64 code bytes, 8 scale chunks
constexpr int kMoeMaxPartTiles = 16;        // K tiles of one CTA: a 16-row panel takes 64 KB

struct MoeArgs {
    const uint16_t *x;            // bf16 [T, K]
    const float *weights;         // [T, topk]
    const int32_t *offsets;       // [E + 1]
    const int32_t *row_index;     // [R]
    const int32_t *pos;           // [T, topk]
    const uint8_t *wq_gu, *wsf_gu;
    const uint8_t *wq_dn, *wsf_dn;
    const float *inv_gu, *inv_dn; // [E, K], [E, I] or nullptr
    uint16_t *h;                  // workspace: fp16 [R, I]
    float *hs;                    // workspace: [R, I / 32], 1 / s of every group of h
    float *y;                     // workspace: [R, N]
    int32_t *counts;              // workspace: [N / 128, T]
    uint16_t *out;                // bf16 [T, N]
    int32_t T, topk, E, K, I, N, R, b_gu, b_dn;
    int32_t part_tiles;           // the most K tiles a CTA of the launched kernel takes
};

// Dynamic shared memory of a CTA whose part has up to `tiles` K tiles and whose chunk has up to `rows` rows: panel, 1 / s
// [tile][group][row], a flag per tile (some s is not 1), rings.
__host__ __device__ constexpr int moe_panel_stride(int tiles) { return tiles * 256 + 64; }   // bytes; 64 mod 128: no bank conflicts
__host__ __device__ constexpr int moe_ring_offset(int tiles, int rows) {
    return rows * moe_panel_stride(tiles) + tiles * 4 * rows * 4 + kMoeMaxPartTiles * 4;
}
__host__ __device__ constexpr int moe_smem_bytes(int tiles, int rows) {
    return moe_ring_offset(tiles, rows) + kMoeWarps * kMoeStages * kMoeStageBytes;
}

__device__ __forceinline__ void cp_async16(uint32_t dst, const void *src) {
    asm volatile("cp.async.cg.shared.global.L2::128B [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int kLeft>
__device__ __forceinline__ void cp_async_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(kLeft) : "memory"); }

__device__ __forceinline__ void ldmatrix_x4(uint32_t (&r)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}

// Eight E2M1 codes (low nibble first) -> four fp16 pairs, exact.
__device__ __forceinline__ void e2m1x8_to_half(uint32_t w, uint32_t (&h)[4]) {
    asm("{\n\t.reg .b8 a, b, c, d;\n\t"
        "mov.b32 {a, b, c, d}, %4;\n\t"
        "cvt.rn.f16x2.e2m1x2 %0, a;\n\t"
        "cvt.rn.f16x2.e2m1x2 %1, b;\n\t"
        "cvt.rn.f16x2.e2m1x2 %2, c;\n\t"
        "cvt.rn.f16x2.e2m1x2 %3, d;\n\t}"
        : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
        : "r"(w));
}

// d += A (16 x 16 fp16, rows g and g + 8 per lane) x B (16 x 8 fp16)
__device__ __forceinline__ void mma_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                        uint32_t b1) {
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
                 "{%0, %1, %2, %3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// d = A x B
__device__ __forceinline__ void mma_f16_zero(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                             uint32_t b1) {
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
                 "{%10, %10, %10, %10};"
                 : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
                 : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.0f));
}

// 2^(E - 127) of the four scale bytes of a word.
__device__ __forceinline__ void moe_scales(uint32_t word, float (&s)[4]) {
    uint32_t lo, hi;
    asm("{\n\t.reg .b16 a, b;\n\t"
        "mov.b32 {a, b}, %2;\n\t"
        "cvt.rn.bf16x2.ue8m0x2 %0, a;\n\t"
        "cvt.rn.bf16x2.ue8m0x2 %1, b;\n\t}"
        : "=r"(lo), "=r"(hi)
        : "r"(word));
    s[0] = __uint_as_float(lo << 16);
    s[1] = __uint_as_float(lo & 0xFFFF0000u);
    s[2] = __uint_as_float(hi << 16);
    s[3] = __uint_as_float(hi & 0xFFFF0000u);
}

struct MoeChunk {
    int32_t e, row0, rows;   // expert, first sorted row, rows; e < 0: there is no such chunk
};

// The z-th chunk of the plan: per expert ceil(rows / kRows), in expert order. Offsets are clamped into [0, R], so rows of a
// malformed plan stay inside the workspace. Called by the whole CTA; the plan is read past L1.
template <int kRows>
__device__ __forceinline__ MoeChunk moe_find_chunk(const MoeArgs &a, int z) {
    __shared__ int32_t s_sum[kMoeWarps];
    __shared__ MoeChunk s_chunk;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    constexpr int kPer = kRouteMaxExperts / kMoeThreads;
    const int per = (a.E + kMoeThreads - 1) / kMoeThreads;   // experts per thread, in order
    int32_t first[kPer], rows[kPer], mine = 0;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
        const int e = threadIdx.x * per + i;
        rows[i] = 0;
        if (i < per && e < a.E) {
            const int32_t lo = min(max(__ldcg(a.offsets + e), 0), a.R), hi = min(max(__ldcg(a.offsets + e + 1), 0), a.R);
            first[i] = lo;
            rows[i] = max(hi - lo, 0);
        }
        mine += (rows[i] + kRows - 1) / kRows;
    }
    int32_t x = mine;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const int32_t y = __shfl_up_sync(0xffffffffu, x, d);
        if (lane >= d) x += y;
    }
    if (lane == 31) s_sum[warp] = x;
    if (threadIdx.x == 0) s_chunk.e = -1;
    __syncthreads();
    int32_t at = x - mine;
    for (int w = 0; w < warp; ++w) at += s_sum[w];
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
        const int32_t n = (rows[i] + kRows - 1) / kRows;
        if (z >= at && z < at + n) {
            const int32_t skip = (z - at) * kRows;
            s_chunk = {static_cast<int32_t>(threadIdx.x * per + i), first[i] + skip, min(rows[i] - skip, kRows)};
        }
        at += n;
    }
    __syncthreads();
    return s_chunk;
}

// Four neighbouring channels per lane, 128 per warp: the block Hadamard of order b (stages h = 1, 2, ... in order).
__device__ __forceinline__ void moe_rotate(float (&v)[4], int b, int lane) {
    if (b == 1) return;
    float a0 = v[0] + v[1], a1 = v[0] - v[1], a2 = v[2] + v[3], a3 = v[2] - v[3];
    v[0] = a0 + a2, v[1] = a1 + a3, v[2] = a0 - a2, v[3] = a1 - a3;
#pragma unroll
    for (int h = 4; h < 128; h <<= 1) {
        if (h >= b) break;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float o = __shfl_xor_sync(0xffffffffu, v[i], h / 4);
            v[i] = (lane & (h / 4)) ? o - v[i] : v[i] + o;
        }
    }
}

// log2 of the power of two s that a group is scaled by before fp16, from its largest magnitude: 0 when that is in
// [2^-10, 2^15) or zero, else what brings it to the range's nearer end.
__device__ __forceinline__ int moe_shift(float top) {
    const int e = static_cast<int>(__float_as_uint(top) >> 23);
    const int shift = e < 117 ? 117 - e : (e > 141 ? 141 - e : 0);
    return top == 0.0f ? 0 : min(shift, 112);
}

__device__ __forceinline__ float moe_pow2(int e) { return __uint_as_float(static_cast<uint32_t>(127 + e) << 23); }

__device__ __forceinline__ uint32_t half2_bits(float a, float b) {
    const __half2 h = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t *>(&h);
}

// One 32-channel group per thread: x (bf16), multipliers, the block Hadamard of order kB, fp16 into the panel.
// For kB > 32 the neighbouring lanes hold the neighbouring groups; the whole warp calls it. Returns 1 / s.
template <int kB>
__device__ __forceinline__ float moe_group_to_half(const uint16_t *x, const float *mul, bool on, uint8_t *dst) {
    uint4 raw[4];
    load_group_global(x, raw);
    uint64_t p[16];
    unpack_bf16x32(raw, p);
    if (mul != nullptr) {
        uint64_t mv[16];
        load_mul(mul, mv);
#pragma unroll
        for (int i = 0; i < 16; ++i) p[i] = mul2(p[i], mv[i]);
    }
    fwht_in_thread<kB>(p);
    if constexpr (kB >= 64) fwht_cross_lane(p, 1);
    if constexpr (kB >= 128) fwht_cross_lane(p, 2);
    float top = 0.0f;
#pragma unroll
    for (int i = 0; i < 16; ++i) {
        float a, b;
        upk2(p[i], a, b);
        top = fmaxf(top, fmaxf(fabsf(a), fabsf(b)));
    }
    const int shift = moe_shift(top);
    const float s = moe_pow2(shift);
    const uint64_t s2 = pk2(s, s);
    uint32_t h[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) {
        float a, b;
        upk2(mul2(p[i], s2), a, b);
        h[i] = half2_bits(a, b);
    }
    if (on)
#pragma unroll
        for (int i = 0; i < 4; ++i)
            *reinterpret_cast<uint4 *>(dst + 16 * i) = make_uint4(h[4 * i], h[4 * i + 1], h[4 * i + 2], h[4 * i + 3]);
    return moe_pow2(-shift);
}

// The weight stream of one warp: 32 rows of a 128-row tile (rows 8 p + g + 32 q) over K tiles.
struct MoeStream {
    const uint8_t *codes;   // this lane's first 16 bytes: row 8 p + lane / 4, chunk lane % 4, of the first tile
    const uint8_t *sf;      // this lane's scale chunk (lanes 0 .. 7) of the first tile
    int64_t q_stride;       // 32 rows of codes
    uint32_t ring;          // shared address of the warp's ring
    uint32_t st;            // this lane's offset inside a stage for its stores
    int lane;

    __device__ __forceinline__ MoeStream(const uint8_t *wq, const uint8_t *wsf, int64_t row_tile, int K, int first_tile, int p,
                                         uint32_t ring_, int lane_) {
        lane = lane_;
        const int g = lane >> 2, c = lane & 3;
        codes = wq + (row_tile * 128 + 8 * p + g) * (K / 2) + first_tile * 64 + 16 * c;
        sf = wsf + (row_tile * (K / 128) + first_tile) * 512 + (8 * p + (lane & 7)) * 16;
        q_stride = 32 * static_cast<int64_t>(K / 2);
        ring = ring_;
        st = g * 64 + ((c ^ ((g >> 1) & 3)) << 4);
    }
    __device__ __forceinline__ void issue(int tile, int tiles) const {
        if (tile < tiles) {
            const uint32_t dst = ring + (tile % kMoeStages) * kMoeStageBytes;
            const uint8_t *src = codes + tile * 64;
#pragma unroll
            for (int q = 0; q < 4; ++q) cp_async16(dst + 512 * q + st, src + q * q_stride);
            if (lane < 8) cp_async16(dst + 2048 + 16 * lane, sf + static_cast<int64_t>(tile) * 512);
        }
        cp_async_commit();   // an empty group keeps the count of groups equal to the count of tiles
    }
};

// One K tile: acc += the stage's 32 rows x the panel's columns. kScaled: some group of the tile has s != 1.
template <int kNt, bool kScaled>
__device__ __forceinline__ void moe_tile_mma(const uint32_t (&code)[4][4], const float (&sf)[4][4], uint32_t bcol, int stride,
                                             const float *xs, float (&acc)[2][kNt][4]) {
#pragma unroll
    for (int c = 0; c < 4; ++c) {
        uint32_t a[4][4];
#pragma unroll
        for (int q = 0; q < 4; ++q) e2m1x8_to_half(code[q][c], a[q]);
#pragma unroll
        for (int n = 0; n < kNt; ++n) {
            uint32_t b[4];
            asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                         : "=r"(b[0]), "=r"(b[1]), "=r"(b[2]), "=r"(b[3])
                         : "r"(bcol + n * 8 * stride + c * 64)
                         : "memory");
            float2 x = make_float2(1.0f, 1.0f);
            if constexpr (kScaled) x = *reinterpret_cast<const float2 *>(xs + c * 8 * kNt + 8 * n);
#pragma unroll
            for (int m = 0; m < 2; ++m) {
                float d[4];
                mma_f16_zero(d, a[2 * m][0], a[2 * m + 1][0], a[2 * m][1], a[2 * m + 1][1], b[0], b[1]);
                mma_f16(d, a[2 * m][2], a[2 * m + 1][2], a[2 * m][3], a[2 * m + 1][3], b[2], b[3]);
                const float s0 = sf[2 * m][c], s1 = sf[2 * m + 1][c];
                if constexpr (kScaled) {
                    acc[m][n][0] = fmaf(d[0], s0 * x.x, acc[m][n][0]);
                    acc[m][n][1] = fmaf(d[1], s0 * x.y, acc[m][n][1]);
                    acc[m][n][2] = fmaf(d[2], s1 * x.x, acc[m][n][2]);
                    acc[m][n][3] = fmaf(d[3], s1 * x.y, acc[m][n][3]);
                } else {
                    acc[m][n][0] = fmaf(d[0], s0, acc[m][n][0]);
                    acc[m][n][1] = fmaf(d[1], s0, acc[m][n][1]);
                    acc[m][n][2] = fmaf(d[2], s1, acc[m][n][2]);
                    acc[m][n][3] = fmaf(d[3], s1, acc[m][n][3]);
                }
            }
        }
    }
}

// acc[2 row tiles][kNt column tiles][4] += the warp's 32 rows x the panel's columns over `tiles` K tiles. panel: shared address
// of the first of these tiles; xs: 1 / s [tile][group][8 kNt]; scaled: the tiles' flags.
template <int kNt>
__device__ __forceinline__ void moe_stream_mma(const MoeStream &w, int tiles, uint32_t panel, int stride, const float *xs,
                                               const int32_t *scaled, float (&acc)[2][kNt][4]) {
    const int lane = w.lane, g = lane >> 2, t = lane & 3;
    const uint32_t ld = (lane & 7) * 64 + (((lane >> 3) ^ ((lane >> 1) & 3)) << 4);   // ldmatrix: chunk lane / 8 of row lane % 8
    const uint32_t bcol = panel + g * stride + t * 16;
    const float *xcol = xs + 2 * t;
#pragma unroll 1
    for (int i = 0; i < tiles; ++i) {
        cp_async_wait<kMoeStages - 2>();
        __syncwarp();   // every lane's copies of tile i have landed, and every lane is done with tile i - 1
        w.issue(i + kMoeStages - 1, tiles);
        const uint32_t stage = w.ring + (i % kMoeStages) * kMoeStageBytes;
        uint32_t code[4][4];
#pragma unroll
        for (int q = 0; q < 4; ++q) ldmatrix_x4(code[q], stage + 512 * q + ld);
        uint32_t word[4];
        asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                     : "=r"(word[0]), "=r"(word[1]), "=r"(word[2]), "=r"(word[3])
                     : "r"(stage + 2048 + 16 * g)
                     : "memory");
        float sf[4][4];
#pragma unroll
        for (int q = 0; q < 4; ++q) moe_scales(word[q], sf[q]);
        if (scaled[i]) moe_tile_mma<kNt, true>(code, sf, bcol + i * 256, stride, xcol + i * 32 * kNt, acc);
        else moe_tile_mma<kNt, false>(code, sf, bcol + i * 256, stride, xcol, acc);
    }
}

// A float4 of the same shared variable in another CTA of the cluster.
__device__ __forceinline__ float4 cluster_ld4(const float *p, uint32_t rank) {
    uint32_t addr;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(addr) : "r"(smem_u32(p)), "r"(rank));
    float4 v;
    asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                 : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
                 : "r"(addr)
                 : "memory");
    return v;
}

__device__ __forceinline__ void add4(float4 &a, const float4 &b) {
    a.x += b.x, a.y += b.y, a.z += b.z, a.w += b.w;
}

template <int kB>
__device__ __forceinline__ void moe_fill_panel(const MoeArgs &a, const MoeChunk &ch, const int32_t *token, int tile0, int tiles,
                                               uint8_t *panel, int stride, float *xs, int32_t *scaled, int panel_rows) {
    const int lane = threadIdx.x & 31, groups = tiles * 4, total = ch.rows * groups;
    for (int base = threadIdx.x & ~31; base < total; base += kMoeThreads) {
        const int u = min(base + lane, total - 1);
        const int row = u / groups, gr = u - row * groups;
        const int64_t k = tile0 * 128 + gr * 32;
        const float inv = moe_group_to_half<kB>(a.x + static_cast<int64_t>(token[row]) * a.K + k,
                                                a.inv_gu == nullptr ? nullptr : a.inv_gu + static_cast<int64_t>(ch.e) * a.K + k,
                                                base + lane < total, panel + row * stride + gr * 64);
        if (base + lane < total) {
            xs[gr * panel_rows + row] = inv;
            if (inv != 1.0f) scaled[gr >> 2] = 1;
        }
    }
}

// Kernel 1. Grid (parts of K = cluster, I / 128, chunks).
template <int kNt>
__global__ void __launch_bounds__(kMoeThreads, kNt == 1 ? 3 : 2) moe_gate_up_kernel(MoeArgs a) {
    extern __shared__ __align__(16) uint8_t s_raw[];
    constexpr int kRows = 8 * kNt;
    __shared__ int32_t s_token[kRows];
    griddep_wait();   // the plan, X and the workspace may belong to the previous kernel in the stream
    griddep_launch_dependents();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int parts = gridDim.x, part = blockIdx.x;
    if (part == 0 && blockIdx.y == 0 && blockIdx.z == 0)
        for (int i = threadIdx.x; i < a.T * (a.N / 128); i += kMoeThreads) a.counts[i] = 0;
    const int stride = moe_panel_stride(a.part_tiles);
    float *xs = reinterpret_cast<float *>(s_raw + kRows * stride);
    int32_t *scaled = reinterpret_cast<int32_t *>(xs + a.part_tiles * 4 * kRows);
    uint8_t *rings = s_raw + moe_ring_offset(a.part_tiles, kRows);
    if (threadIdx.x < kMoeMaxPartTiles) scaled[threadIdx.x] = 0;
    const MoeChunk ch = moe_find_chunk<kRows>(a, blockIdx.z);
    if (ch.e < 0) return;   // the same for the whole cluster
    const int kt = a.K / 128;
    const int tile0 = part * kt / parts, tiles = (part + 1) * kt / parts - tile0;
    const int64_t row_tiles = 2 * a.I / 128;
    const MoeStream w(a.wq_gu, a.wsf_gu, ch.e * row_tiles + 2 * blockIdx.y + (warp >> 2), a.K, tile0, warp & 3,
                      smem_u32(rings) + warp * kMoeStages * kMoeStageBytes, lane);
#pragma unroll
    for (int i = 0; i < kMoeStages - 1; ++i) w.issue(i, tiles);
    if (threadIdx.x < kRows)
        s_token[threadIdx.x] =
            threadIdx.x < ch.rows ? min(max(__ldcg(a.row_index + ch.row0 + threadIdx.x), 0), a.T - 1) : 0;
    __syncthreads();
    switch (a.b_gu) {
        case 1: moe_fill_panel<1>(a, ch, s_token, tile0, tiles, s_raw, stride, xs, scaled, kRows); break;
        case 16: moe_fill_panel<16>(a, ch, s_token, tile0, tiles, s_raw, stride, xs, scaled, kRows); break;
        case 32: moe_fill_panel<32>(a, ch, s_token, tile0, tiles, s_raw, stride, xs, scaled, kRows); break;
        case 64: moe_fill_panel<64>(a, ch, s_token, tile0, tiles, s_raw, stride, xs, scaled, kRows); break;
        default: moe_fill_panel<128>(a, ch, s_token, tile0, tiles, s_raw, stride, xs, scaled, kRows); break;
    }
    __syncthreads();
    float acc[2][kNt][4] = {};
    moe_stream_mma<kNt>(w, tiles, smem_u32(s_raw), stride, xs, scaled, acc);
    cp_async_wait<0>();
    __syncthreads();
    // partial sums [column][gate, up][128 channels], over the rings. Quarters 0, 1 of a warp's rows are gate channels
    // c, c + 32; quarters 2, 3 the up rows of the same channels.
    float *part_sums = reinterpret_cast<float *>(rings);
    const int channel = 64 * (warp >> 2) + 8 * (warp & 3) + (lane >> 2);
#pragma unroll
    for (int n = 0; n < kNt; ++n)
#pragma unroll
        for (int m = 0; m < 2; ++m)
#pragma unroll
            for (int k = 0; k < 4; ++k)
                part_sums[(8 * n + 2 * (lane & 3) + (k & 1)) * 256 + m * 128 + channel + 32 * (k >> 1)] = acc[m][n][k];
    if (parts > 1) cluster_sync();
    else __syncthreads();
    // rows part, part + parts, ... : one per warp and step, four channels per lane
    for (int row = part + parts * warp; row < ch.rows; row += parts * kMoeWarps) {
        const float *p = part_sums + row * 256 + 4 * lane;
        float4 g = make_float4(0.0f, 0.0f, 0.0f, 0.0f), u = g;
        for (int r = 0; r < parts; ++r) {
            add4(g, parts > 1 ? cluster_ld4(p, r) : *reinterpret_cast<const float4 *>(p));
            add4(u, parts > 1 ? cluster_ld4(p + 128, r) : *reinterpret_cast<const float4 *>(p + 128));
        }
        float v[4] = {g.x / (1.0f + expf(-g.x)) * u.x, g.y / (1.0f + expf(-g.y)) * u.y, g.z / (1.0f + expf(-g.z)) * u.z,
                      g.w / (1.0f + expf(-g.w)) * u.w};
        const int i = 128 * blockIdx.y + 4 * lane;
        if (a.inv_dn != nullptr) {
            const float4 f = *reinterpret_cast<const float4 *>(a.inv_dn + static_cast<int64_t>(ch.e) * a.I + i);
            v[0] *= f.x, v[1] *= f.y, v[2] *= f.z, v[3] *= f.w;
        }
        moe_rotate(v, a.b_dn, lane);
        float top = fmaxf(fmaxf(fabsf(v[0]), fabsf(v[1])), fmaxf(fabsf(v[2]), fabsf(v[3])));
#pragma unroll
        for (int d = 1; d < 8; d <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));   // 8 lanes: a group
        const int shift = moe_shift(top);
        const float s = moe_pow2(shift);
        const int64_t r = ch.row0 + row;
        *reinterpret_cast<uint2 *>(a.h + r * a.I + i) = make_uint2(half2_bits(v[0] * s, v[1] * s), half2_bits(v[2] * s, v[3] * s));
        if ((lane & 7) == 0) a.hs[r * (a.I / 32) + i / 32] = moe_pow2(-shift);
    }
    if (parts > 1) cluster_sync();   // no CTA leaves while another reads its sums
}

// The sum of a token's choices for 128 outputs, four per lane, in the order of the choices.
__device__ __forceinline__ void moe_combine_token(const MoeArgs &a, int t, int n, int lane) {
    const int32_t live = min(max(__ldcg(a.offsets + a.E), 0), a.R);
    int32_t p = -1;
    float wt = 0.0f;
    if (lane < a.topk) {
        p = __ldcg(a.pos + t * a.topk + lane);
        wt = __ldcg(a.weights + t * a.topk + lane);
        if (p >= live) p = -1;
    }
    float4 s = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll 8
    for (int j = 0; j < a.topk; ++j) {
        const int32_t r = __shfl_sync(0xffffffffu, p, j);
        const float w = __shfl_sync(0xffffffffu, wt, j);
        if (r >= 0) {
            const float4 v = __ldcg(reinterpret_cast<const float4 *>(a.y + static_cast<int64_t>(r) * a.N + n + 4 * lane));
            s.x = fmaf(w, v.x, s.x), s.y = fmaf(w, v.y, s.y), s.z = fmaf(w, v.z, s.z), s.w = fmaf(w, v.w, s.w);
        }
    }
    const __nv_bfloat162 lo = __floats2bfloat162_rn(s.x, s.y), hi = __floats2bfloat162_rn(s.z, s.w);
    *reinterpret_cast<uint2 *>(a.out + static_cast<int64_t>(t) * a.N + n + 4 * lane) =
        make_uint2(*reinterpret_cast<const uint32_t *>(&lo), *reinterpret_cast<const uint32_t *>(&hi));
}

// Live choices of token t (whole warp): how many rows its counter waits for.
__device__ __forceinline__ int moe_live_choices(const MoeArgs &a, int t, int32_t live, int lane) {
    const int32_t p = lane < a.topk ? __ldcg(a.pos + t * a.topk + lane) : -1;
    return __popc(__ballot_sync(0xffffffffu, p >= 0 && p < live));
}

// Kernel 2. Grid (parts of I = cluster, N / 128, chunks). Warps 0-3 and 4-7 take the halves of the part's tiles for the same
// 128 rows.
template <int kNt>
__global__ void __launch_bounds__(kMoeThreads, kNt == 1 ? 3 : 2) moe_down_kernel(MoeArgs a) {
    constexpr int kRows = 8 * kNt;
    extern __shared__ __align__(16) uint8_t s_raw[];
    __shared__ int32_t s_token[kRows];
    __shared__ int32_t s_need[kRows];
    __shared__ int32_t s_last[kRows];
    griddep_launch_dependents();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int parts = gridDim.x, part = blockIdx.x;
    // Kernel 1 let this grid start only after its own wait for everything before it, so the plan and the weights are
    // complete; only kernel 1's rows are not.
    const MoeChunk ch = moe_find_chunk<kRows>(a, blockIdx.z);
    const int32_t live = min(max(__ldcg(a.offsets + a.E), 0), a.R);
    if (part == 0 && blockIdx.z == 0)   // tokens whose choices are all dropped
        for (int t = warp; t < a.T; t += kMoeWarps)
            if (moe_live_choices(a, t, live, lane) == 0) {
                griddep_wait();
                *reinterpret_cast<uint2 *>(a.out + static_cast<int64_t>(t) * a.N + 128 * blockIdx.y + 4 * lane) = make_uint2(0u, 0u);
            }
    if (ch.e < 0) {
        griddep_wait();
        return;
    }
    const int kt = a.I / 128;
    const int tile0 = part * kt / parts, tiles = (part + 1) * kt / parts - tile0;
    const int half0 = (warp >> 2) ? tiles / 2 : 0, halves = (warp >> 2) ? tiles - tiles / 2 : tiles / 2;
    const int stride = moe_panel_stride(a.part_tiles);
    float *xs = reinterpret_cast<float *>(s_raw + kRows * stride);
    int32_t *scaled = reinterpret_cast<int32_t *>(xs + a.part_tiles * 4 * kRows);
    uint8_t *rings = s_raw + moe_ring_offset(a.part_tiles, kRows);
    if (threadIdx.x < kMoeMaxPartTiles) scaled[threadIdx.x] = 0;
    const MoeStream w(a.wq_dn, a.wsf_dn, ch.e * static_cast<int64_t>(a.N / 128) + blockIdx.y, a.I, tile0 + half0, warp & 3,
                      smem_u32(rings) + warp * kMoeStages * kMoeStageBytes, lane);
#pragma unroll
    for (int i = 0; i < kMoeStages - 1; ++i) w.issue(i, halves);
    for (int row = warp; row < ch.rows; row += kMoeWarps) {
        const int t = min(max(__ldcg(a.row_index + ch.row0 + row), 0), a.T - 1);
        const int need = moe_live_choices(a, t, live, lane);
        if (lane == 0) {
            s_token[row] = t;
            s_need[row] = need;
        }
    }
    griddep_wait();
    __syncthreads();
    for (int i = threadIdx.x; i < ch.rows * tiles * 16; i += kMoeThreads) {
        const int row = i / (tiles * 16), c = i - row * tiles * 16;
        *reinterpret_cast<uint4 *>(s_raw + row * stride + c * 16) =
            __ldcg(reinterpret_cast<const uint4 *>(a.h + static_cast<int64_t>(ch.row0 + row) * a.I + tile0 * 128 + c * 8));
    }
    for (int i = threadIdx.x; i < ch.rows * tiles * 4; i += kMoeThreads) {
        const int row = i / (tiles * 4), gr = i - row * tiles * 4;
        const float inv = __ldcg(a.hs + static_cast<int64_t>(ch.row0 + row) * (a.I / 32) + tile0 * 4 + gr);
        xs[gr * kRows + row] = inv;
        if (inv != 1.0f) scaled[gr >> 2] = 1;
    }
    __syncthreads();
    float acc[2][kNt][4] = {};
    moe_stream_mma<kNt>(w, halves, smem_u32(s_raw) + half0 * 256, stride, xs + half0 * 4 * kRows, scaled + half0, acc);
    cp_async_wait<0>();
    __syncthreads();
    float *part_sums = reinterpret_cast<float *>(rings);   // [halves][column][128]
#pragma unroll
    for (int n = 0; n < kNt; ++n)
#pragma unroll
        for (int m = 0; m < 2; ++m)
#pragma unroll
            for (int k = 0; k < 4; ++k)   // quarter 2 m + k / 2, column 2 t + k % 2
                part_sums[((warp >> 2) * kRows + 8 * n + 2 * (lane & 3) + (k & 1)) * 128 + 8 * (warp & 3) + (lane >> 2) +
                          32 * (2 * m + (k >> 1))] = acc[m][n][k];
    if (parts > 1) cluster_sync();
    else __syncthreads();
    const int n = 128 * blockIdx.y;
    for (int row = part + parts * warp; row < ch.rows; row += parts * kMoeWarps) {
        const float *p = part_sums + row * 128 + 4 * lane;
        float4 s = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        for (int r = 0; r < parts; ++r) {
            add4(s, parts > 1 ? cluster_ld4(p, r) : *reinterpret_cast<const float4 *>(p));
            add4(s, parts > 1 ? cluster_ld4(p + kRows * 128, r) : *reinterpret_cast<const float4 *>(p + kRows * 128));
        }
        *reinterpret_cast<float4 *>(a.y + static_cast<int64_t>(ch.row0 + row) * a.N + n + 4 * lane) = s;
    }
    // whoever counts a token's last row adds its choices: rows are visible on the device before they are counted
    __threadfence();
    __syncthreads();
    if (threadIdx.x < ch.rows && threadIdx.x % parts == part) {
        const int t = s_token[threadIdx.x];
        s_last[threadIdx.x] = atomicAdd(a.counts + static_cast<int64_t>(blockIdx.y) * a.T + t, 1) + 1 == s_need[threadIdx.x];
    }
    __syncthreads();
    for (int row = part + parts * warp; row < ch.rows; row += parts * kMoeWarps)
        if (s_last[row]) {
            __threadfence();
            moe_combine_token(a, s_token[row], n, lane);
        }
    if (parts > 1) cluster_sync();
}

}  // namespace macaq
