// moe_w4a16.cuh -- a whole mixture-of-experts layer for few tokens: MXFP4 weights, bf16 activations.
//
//   x'  = x diag(1/s_e) H_b                        (fp32 butterflies; the weight-only mode's transform)
//   g, u = gate and up rows of x' dq(W'_gu,e)^T    (64-row interleaved blocks)
//   h   = silu(g) u,  h' = h diag(1/s_down,e) H_b'
//   out[t] = sum_j weights[t, j] * (h'_{pos[t, j]} dq(W'_down,e)^T)
//
// Bound by HBM: every active expert's codes and scales (17/32 byte a weight), and an expert has a handful of rows, so the
// two products are streams of weights against a small operand that stays in shared memory. They are read once per chunk of
// an expert's rows: once in all up to 8 (16) rows, as long as panels of so many rows fit: K and I up to 6,144 (2,560). Wider
// layers have smaller chunks (I = 14336: 2 rows), and experts with more rows than that stream their weights several times.
//
// Plan. Three launches: gate, up and SwiGLU (kernel 1); down (kernel 2); the weighted sum of each token's choices (for few
// rows one kernel does the last two, see moe_down_sum_kernel). The rows of an expert are cut into chunks of up to 8 or 16 (8
// when experts average four rows or fewer, so that one n8 tile nearly always does). An item is (chunk, 32 weight rows):
// rows 8 p + g of each of the four 32-row quarters of a scale tile, so one 16-byte scale chunk serves a lane's four rows,
// and gate and up rows of a channel meet in one lane.
// CTAs, one per SM, take equal contiguous ranges of the items, chunk by chunk, and cut theirs into equal runs of K tiles
// (128 channels), one per warp, wherever the cuts fall: every warp streams the same number of weights, for one token as
// for 64. The pieces of a cut item meet in shared memory once the CTA's warps are done. The chunks' operands are
// fp16 panels in shared memory, made before the CTA streams; each warp streams through its own ring of cp.async stages,
// without a barrier.
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
// Measured on B200 (128 experts, top-8, 2048 x 768; a graph that cycles three layers): one token 15.7 us (20.2 MB), 8 tokens
// 35.5 us (130 MB), 64 tokens 72.2 us (318 MB, 4.4 TB/s). With 64 tokens the two weight streams themselves run at 5.9 and
// 5.8 TB/s (36 and 18 us) of the 6.5 that a copy reaches; the rest is three starts (plan 1.3 us, first loads and panel 3 to
// 5 us, a launch's end to the next one's first instruction 1 to 1.5 us) and the closing of cut items (1 us). One token is
// made of those latencies alone. Wider layers (top-8 of 128, 4096 x 1536): one token 29.7 us (80 MB), 8 tokens 110 us (541
// MB), 64 tokens 261 us (1273 MB, 4.9 TB/s); top-8 of 256, 7168 x 2048: 50.8 (187 MB), 253 (1310 MB), 1010 us (5147 MB);
// top-2 of 8, 4096 x 14336: 47.3 (187 MB), 150 (749 MB), and 64 tokens, whose experts have 16 rows in chunks of 2, 720 us
// (749 MB).
// Sources: glonce.com page on MACaQ, paragraph 3 (weight-only serving) and paragraph 5 (grouped matmul);
// aipolix.com page, paragraph 2 (the transform at the input of every linear).
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "groups.cuh"
#include "ptx.cuh"
#include "quant.cuh"
#include "route.cuh"

namespace macaq {

constexpr int kMoeMaxT = 64;
constexpr int kMoeThreads = 512;
constexpr int kMoeWarps = kMoeThreads / 32;
constexpr int kMoeStages = 3;
constexpr int kMoeStageBytes = 2048 + 128;  // 32 rows x 64 code bytes, 8 scale chunks
constexpr int kMoeMaxPanels = 8;
constexpr int kMoeFewRows = 16, kMoeFewTokens = 8;   // of moe_down_sum_kernel
constexpr int kMoeGroupUnroll = 4;         // MX groups of a tile in straight code

struct MoeArgs {
    const uint16_t *x;            // bf16 [T, K]
    const float *weights;         // [T, topk]
    const int32_t *offsets;       // [E + 1]
    const int32_t *row_index;     // [R]
    const int32_t *pos;           // [T, topk]
    const uint8_t *wq_gu, *wsf_gu;
    const uint8_t *wq_dn, *wsf_dn;
    const float *inv_gu, *inv_dn; // [E, K], [E, I] or nullptr
    float *h;                     // workspace: [R, I]
    float *y;                     // workspace: [R, N]
    uint16_t *out;                // bf16 [T, N]
    int32_t T, topk, E, K, I, N, R, b_gu, b_dn;
    int32_t chunk_rows;           // rows of a chunk: 8 or 16, fewer where a panel of so many does not fit
    int32_t panel_rows;           // rows whose panels a CTA holds at a time
    int32_t max_chunks;           // room for the chunks of a CTA's items
};

struct MoeChunk {
    int32_t e, row0, rows;        // expert, first sorted row, rows
};

// A panel row of `tiles` K tiles: fp16 values, then 1 / s of its groups (kept apart, after all rows).
__host__ __device__ constexpr int moe_panel_stride(int tiles) { return tiles * 256 + 64; }   // bytes; 64 mod 128: no bank conflicts
__host__ __device__ constexpr int moe_row_bytes(int tiles) { return moe_panel_stride(tiles) + tiles * 16; }
// Dynamic shared memory: rings, first pieces of cut items (one per warp), panel rows, their 1 / s, flags [panel][tile] (some s
// of the tile is not 1), chunk table.
__host__ __device__ constexpr int moe_heads_offset() { return kMoeWarps * kMoeStages * kMoeStageBytes; }
__host__ __device__ constexpr int moe_panels_offset(int nt) { return moe_heads_offset() + kMoeWarps * 1024 * nt; }
__host__ __device__ constexpr int moe_flags_offset(int nt, int tiles, int rows) {
    return moe_panels_offset(nt) + rows * moe_row_bytes(tiles);
}
__host__ __device__ constexpr int moe_table_offset(int nt, int tiles, int rows) {
    return moe_flags_offset(nt, tiles, rows) + kMoeMaxPanels * tiles * 4;
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
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
                 "{%0, %1, %2, %3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// d = A x B
__device__ __forceinline__ void mma_f16_zero(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                             uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
                 "{%10, %10, %10, %10};"
                 : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
                 : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.0f));
}

// 2^(E - 127) for the scale byte c of two words.
__device__ __forceinline__ void moe_scales(uint32_t w0, uint32_t w1, int c, float &s0, float &s1) {
    const uint32_t two = __byte_perm(w0, w1, 0x0040u + 0x0011u * c);
    uint32_t r;
    asm("{\n\t.reg .b16 a, b;\n\t"
        "mov.b32 {a, b}, %1;\n\t"
        "cvt.rn.bf16x2.ue8m0x2 %0, a;\n\t}"
        : "=r"(r)
        : "r"(two));
    s0 = __uint_as_float(r << 16);
    s1 = __uint_as_float(r & 0xFFFF0000u);
}

// The plan's chunks, per expert ceil(rows / chunk_rows) of them in expert order, make `blocks` items each. Returns the item
// range of CTA c of `ctas` and the number of its first item in that item's chunk, and fills table[] with the chunks that
// it meets. Offsets are clamped into [0, R], so rows of a malformed plan stay inside the workspace; they are read past
// L1, once per CTA into `off_s` (all CTAs read the same few lines). Every warp scans them, with the same result.
__device__ __forceinline__ void moe_find_items(const MoeArgs &a, int c, int ctas, int blocks, int32_t *off_s, MoeChunk *table,
                                               int &begin, int &end, int &first) {
    const int lane = threadIdx.x & 31, per = a.chunk_rows;
    for (int e = threadIdx.x; e <= a.E; e += blockDim.x) off_s[e] = min(max(__ldcg(a.offsets + e), 0), a.R);
    __syncthreads();
    int total = 0;
    const int passes = a.E <= 128 ? 1 : 2;   // up to 128 experts one pass knows the total; else count first
#pragma unroll 1
    for (int pass = 0; pass < passes; ++pass) {
        int before = 0;
#pragma unroll 1
        for (int base = 0; base < a.E; base += 128) {
            int32_t off[5], n = 0;
#pragma unroll
            for (int i = 0; i < 5; ++i) off[i] = off_s[min(base + 4 * lane + i, a.E)];
#pragma unroll
            for (int i = 0; i < 4; ++i) n += (max(off[i + 1] - off[i], 0) + per - 1) / per;
            int32_t x = n;
#pragma unroll
            for (int d = 1; d < 32; d <<= 1) {
                const int32_t y = __shfl_up_sync(0xffffffffu, x, d);
                if (lane >= d) x += y;
            }
            int32_t at = before + x - n;
            before += __shfl_sync(0xffffffffu, x, 31);
            if (pass == 0) total = min(before, 60000);   // a sound plan has fewer; keeps item numbers in 31 bits
            if (pass == passes - 1) {
                const int items = total * blocks, share = items / ctas, rest = items - share * ctas;
                begin = c * share + min(c, rest);
                end = begin + share + (c < rest ? 1 : 0);
                const int z0 = begin / blocks;
                first = begin - z0 * blocks;
                end = min(end, (z0 + a.max_chunks) * blocks);   // more only where a plan lists a row twice
                const int z1 = begin < end ? (end - 1) / blocks : -1;
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    for (int rows = off[i + 1] - off[i]; rows > 0; rows -= per, ++at)
                        if (at >= z0 && at <= z1)
                            table[at - z0] = {base + 4 * lane + i, off[i + 1] - rows, min(rows, per)};
            }
        }
    }
    __syncthreads();   // off_s is free again
}

// log2 of the power of two s that a group is scaled by before fp16, from its largest magnitude: 0 when that is in
// [2^-10, 2^15) or zero, else what brings it to the range's nearer end. A value below the normal numbers has no exponent to
// go by: 2^126 brings it under 1, and its last bit, 2^-149, to 2^-23.
__device__ __forceinline__ int moe_shift(float top) {
    const int e = static_cast<int>(__float_as_uint(top) >> 23);
    const int shift = e < 117 ? (e == 0 ? 126 : 117 - e) : (e > 141 ? 141 - e : 0);
    return top == 0.0f ? 0 : shift;
}

__device__ __forceinline__ float moe_pow2(int e) { return __uint_as_float(static_cast<uint32_t>(127 + e) << 23); }

__device__ __forceinline__ uint32_t half2_bits(float a, float b) {
    const __half2 h = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t *>(&h);
}

// One K tile: acc += the stage's 32 rows x the panel's columns. kScaled: some group of the tile has s != 1; x0, x1: 1 / s of
// this lane's two columns per column tile.
template <int kNt, bool kScaled>
__device__ __forceinline__ void moe_tile_mma(uint32_t codes, const uint32_t (&word)[4], const uint8_t *const (&bcol)[kNt],
                                             const float *const (&x0)[kNt], const float *const (&x1)[kNt], int tile,
                                             float (&acc)[2][kNt][4]) {
#pragma unroll kMoeGroupUnroll
    for (int c = 0; c < 4; ++c) {
        uint32_t code[4], a[4][4];
        ldmatrix_x4(code, codes ^ (c << 4));
#pragma unroll
        for (int q = 0; q < 4; ++q) e2m1x8_to_half(code[q], a[q]);
        float s[4];
        moe_scales(word[0], word[1], c, s[0], s[1]);
        moe_scales(word[2], word[3], c, s[2], s[3]);
#pragma unroll
        for (int n = 0; n < kNt; ++n) {
            const uint4 b = *reinterpret_cast<const uint4 *>(bcol[n] + tile * 256 + c * 64);
            float xa = 1.0f, xb = 1.0f;
            bool beyond = false;   // a scale times 1 / s past fp32, whose sums may be in it all the same (codes of zero)
            if constexpr (kScaled) {
                xa = x0[n][tile * 4 + c], xb = x1[n][tile * 4 + c];
                beyond = isinf(fmaxf(fmaxf(s[0], s[1]), fmaxf(s[2], s[3])) * fmaxf(xa, xb));
            }
#pragma unroll
            for (int m = 0; m < 2; ++m) {
                float d[4];
                mma_f16_zero(d, a[2 * m][0], a[2 * m + 1][0], a[2 * m][1], a[2 * m + 1][1], b.x, b.y);
                mma_f16(d, a[2 * m][2], a[2 * m + 1][2], a[2 * m][3], a[2 * m + 1][3], b.z, b.w);
                if (kScaled && beyond) {
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const float w = s[2 * m + k / 2], x = k % 2 ? xb : xa;
                        acc[m][n][k] = w > 1.0f && x > 1.0f ? fmaf(d[k] * w, x, acc[m][n][k]) : fmaf(d[k], w * x, acc[m][n][k]);
                    }
                } else if constexpr (kScaled) {
                    acc[m][n][0] = fmaf(d[0], s[2 * m] * xa, acc[m][n][0]);
                    acc[m][n][1] = fmaf(d[1], s[2 * m] * xb, acc[m][n][1]);
                    acc[m][n][2] = fmaf(d[2], s[2 * m + 1] * xa, acc[m][n][2]);
                    acc[m][n][3] = fmaf(d[3], s[2 * m + 1] * xb, acc[m][n][3]);
                } else {
                    acc[m][n][0] = fmaf(d[0], s[2 * m], acc[m][n][0]);
                    acc[m][n][1] = fmaf(d[1], s[2 * m], acc[m][n][1]);
                    acc[m][n][2] = fmaf(d[2], s[2 * m + 1], acc[m][n][2]);
                    acc[m][n][3] = fmaf(d[3], s[2 * m + 1], acc[m][n][3]);
                }
            }
        }
    }
}

// Eight neighbouring channels of a panel row per lane, 16 lanes a 128-channel block: the block Hadamard of order b (stages h = 1, 2, ... in order), fp16. Returns 1 / s of the lane's group. The whole warp calls it.
__device__ __forceinline__ float moe_to_half(float (&v)[8], int b, uint4 &out) {
    if (b > 1) {
#pragma unroll
        for (int h = 1; h < 8; h <<= 1)
#pragma unroll
            for (int i = 0; i < 8; ++i)
                if ((i & h) == 0) {
                    const float p = v[i], q = v[i + h];
                    v[i] = p + q;
                    v[i + h] = p - q;
                }
#pragma unroll 1
        for (int d = 1; 8 * d < b; d <<= 1) {   // stage h = 8 d
            const float sign = (threadIdx.x & d) ? -1.0f : 1.0f;
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] = fmaf(v[i], sign, __shfl_xor_sync(0xffffffffu, v[i], d));
        }
    }
    float top = 0.0f;
#pragma unroll
    for (int i = 0; i < 8; ++i) top = fmaxf(top, fabsf(v[i]));
    top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
    top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
    const int shift = moe_shift(top);
    const float s = moe_pow2(shift);
    out = make_uint4(half2_bits(v[0] * s, v[1] * s), half2_bits(v[2] * s, v[3] * s), half2_bits(v[4] * s, v[5] * s),
                     half2_bits(v[6] * s, v[7] * s));
    return moe_pow2(-shift);
}

// The panel rows of a phase from X (kernel 1) or from h (kernel 2). rows: per panel row the chunk (its number in the
// phase) and the row of X or h.
struct MoeRow {
    int32_t panel, source;
};

// after_loads() runs once the first loads are on their way.
template <bool kDown, typename AfterLoads>
__device__ __forceinline__ void moe_fill_panels(const MoeArgs &a, const MoeChunk *chunks, const MoeRow *rows, int count, uint8_t *panel,
                                                float *xs, int32_t *flags, AfterLoads after_loads) {
    const int width = kDown ? a.I : a.K, units = width / 8, total = count * units, lane = threadIdx.x & 31;
    const int stride = moe_panel_stride(width / 128);
    const float *inv_s = kDown ? a.inv_dn : a.inv_gu;
    constexpr int kAtOnce = 2;   // units whose loads are in flight
    bool first = true;
#pragma unroll 1
    for (int base = threadIdx.x & ~31; base < total; base += kAtOnce * kMoeThreads) {
        float4 f[kAtOnce][2], m[kAtOnce][2];
        int row[kAtOnce], c[kAtOnce], chunk[kAtOnce];
#pragma unroll
        for (int k = 0; k < kAtOnce; ++k) {
            const int u = min(base + k * kMoeThreads + lane, total - 1);
            row[k] = u / units;
            c[k] = u - row[k] * units;
            const MoeRow r = rows[row[k]];
            chunk[k] = r.panel;
            if constexpr (kDown) {
                const float4 *src = reinterpret_cast<const float4 *>(a.h + static_cast<int64_t>(r.source) * a.I + 8 * c[k]);
                f[k][0] = __ldcg(src), f[k][1] = __ldcg(src + 1);
            } else {
                f[k][0] = __ldcg(reinterpret_cast<const float4 *>(a.x + static_cast<int64_t>(r.source) * a.K + 8 * c[k]));
            }
            m[k][0] = m[k][1] = make_float4(1.0f, 1.0f, 1.0f, 1.0f);
            if (inv_s != nullptr) {
                const float4 *mul = reinterpret_cast<const float4 *>(inv_s + static_cast<int64_t>(chunks[r.panel].e) * width + 8 * c[k]);
                m[k][0] = __ldg(mul), m[k][1] = __ldg(mul + 1);
            }
        }
        if (first) after_loads();
        first = false;
#pragma unroll
        for (int k = 0; k < kAtOnce; ++k) {
            if (base + k * kMoeThreads >= total) break;
            float v[8];
            if constexpr (kDown) {
                v[0] = f[k][0].x, v[1] = f[k][0].y, v[2] = f[k][0].z, v[3] = f[k][0].w;
                v[4] = f[k][1].x, v[5] = f[k][1].y, v[6] = f[k][1].z, v[7] = f[k][1].w;
            } else {
                const uint32_t w[4] = {__float_as_uint(f[k][0].x), __float_as_uint(f[k][0].y), __float_as_uint(f[k][0].z),
                                       __float_as_uint(f[k][0].w)};
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    v[2 * i] = __uint_as_float(w[i] << 16);
                    v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
                }
            }
            v[0] *= m[k][0].x, v[1] *= m[k][0].y, v[2] *= m[k][0].z, v[3] *= m[k][0].w;
            v[4] *= m[k][1].x, v[5] *= m[k][1].y, v[6] *= m[k][1].z, v[7] *= m[k][1].w;
            uint4 h;
            const float inv = moe_to_half(v, kDown ? a.b_dn : a.b_gu, h);
            if (base + k * kMoeThreads + lane < total) {
                *reinterpret_cast<uint4 *>(panel + row[k] * stride + c[k] * 16) = h;
                if ((lane & 3) == 0) {
                    xs[row[k] * (width / 32) + c[k] / 4] = inv;
                    if (inv != 1.0f) flags[chunk[k] * (width / 128) + c[k] / 16] = 1;
                }
            }
        }
    }
    if (first) after_loads();
}

// The weight stream of one warp: the K tiles of consecutive items, or (kAcross) of the same weight rows of consecutive chunks.
// issue() starts the copies of the next tile.
template <bool kAcross>
struct MoeStream {
    const uint8_t *wq, *wsf;
    const MoeChunk *table;
    const uint8_t *codes;   // this lane's 16 bytes: row 8 p + lane / 4, chunk lane % 4
    const uint8_t *sf;      // this lane's scale chunk (lanes 0 .. 7)
    uint32_t ring, st;      // shared address of the warp's ring; this lane's place in a stage
    int K, tiles, per_chunk;
    int z, r, tile, left, slot;

    __device__ __forceinline__ void point() {   // item r of chunk z: 128-row tile r / 4, p = r % 4
        const int lane = threadIdx.x & 31;
        const int64_t rt = static_cast<int64_t>(table[z].e) * (per_chunk / 4) + (r >> 2);
        codes = wq + (rt * 128 + 8 * (r & 3) + (lane >> 2)) * (K / 2) + tile * 64 + 16 * (lane & 3);
        sf = wsf + (rt * tiles + tile) * 512 + (8 * (r & 3) + (lane & 7)) * 16;
    }
    // `count` tiles from tile `tile_` of item r_ of chunk z_ on
    __device__ __forceinline__ void start(int z_, int r_, int tile_, int count) {
        z = z_, r = r_, tile = tile_, left = count, slot = 0;
        if (left > 0) point();
#pragma unroll 1
        for (int i = 0; i < kMoeStages - 1; ++i) issue();
    }
    __device__ __forceinline__ void issue() {
        const int lane = threadIdx.x & 31;
        if (left > 0) {
            const uint32_t dst = ring + slot * kMoeStageBytes;
#pragma unroll
            for (int q = 0; q < 4; ++q) cp_async16(dst + 512 * q + st, codes + q * (16 * static_cast<int64_t>(K)));
            if (lane < 8) cp_async16(dst + 2048 + 16 * lane, sf);
            codes += 64;
            sf += 512;
            --left;
            if (++tile == tiles) {
                tile = 0;
                if (kAcross || ++r == per_chunk) {
                    if (!kAcross) r = 0;
                    ++z;
                }
                if (left > 0) point();
            }
        }
        slot = slot == kMoeStages - 1 ? 0 : slot + 1;
        cp_async_commit();   // an empty group keeps groups and stages in step
    }
};

// An item's sums, to h (kernel 1) or y (kernel 2). A lane holds rows g of quarters 2 m + k / 2, columns 8 n + 2 t + k % 2.
template <bool kDown, int kNt>
__device__ __forceinline__ void moe_store_item(const MoeArgs &a, const MoeChunk &ch, int r, const float (&acc)[2][kNt][4], int lane) {
    const int base = (kDown ? 128 : 64) * (r >> 2) + 8 * (r & 3) + (lane >> 2);
#pragma unroll
    for (int n = 0; n < kNt; ++n)
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const int col = 8 * n + 2 * (lane & 3) + (k & 1);
            if (col >= ch.rows) continue;
            const int64_t row = ch.row0 + col;
            if constexpr (kDown) {
#pragma unroll
                for (int m = 0; m < 2; ++m) a.y[row * a.N + base + 32 * (2 * m + (k >> 1))] = acc[m][n][k];
            } else {   // quarters 0, 1: gate rows of channels c, c + 32; quarters 2, 3: their up rows
                const float v = acc[0][n][k];
                a.h[row * a.I + base + 32 * (k >> 1)] = v / (1.0f + expf(-v)) * acc[1][n][k];
            }
        }
}

// kDown = false: kernel 1; true: kernel 2.
template <bool kDown, int kNt>
__global__ void __launch_bounds__(kMoeThreads, 1) moe_w4a16_kernel(MoeArgs a) {
    extern __shared__ __align__(128) uint8_t s_moe[];
    __shared__ MoeRow s_rows[kMoeMaxPanels * 8 * kNt];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, t = lane & 3;
    // Kernel 1 waits for everything before it and only then lets kernel 2 start, so the plan and the weights are complete
    // for both; kernel 2 waits for kernel 1's rows before it reads them.
    if constexpr (!kDown) griddep_wait();
    griddep_launch_dependents();

    const int kt = (kDown ? a.I : a.K) / 128, stride = moe_panel_stride(kt);
    float *heads = reinterpret_cast<float *>(s_moe + moe_heads_offset());
    uint8_t *panel = s_moe + moe_panels_offset(kNt);
    float *xs = reinterpret_cast<float *>(panel + a.panel_rows * stride);   // [row][group]
    int32_t *flags = reinterpret_cast<int32_t *>(s_moe + moe_flags_offset(kNt, kt, a.panel_rows));
    MoeChunk *table = reinterpret_cast<MoeChunk *>(s_moe + moe_table_offset(kNt, kt, a.panel_rows));

    MoeStream<false> w;
    w.wq = kDown ? a.wq_dn : a.wq_gu;
    w.wsf = kDown ? a.wsf_dn : a.wsf_gu;
    w.table = table;
    w.ring = smem_u32(s_moe) + warp * kMoeStages * kMoeStageBytes;
    w.st = g * 64 + ((t ^ ((g >> 1) & 3)) << 4);
    w.K = 128 * kt;
    w.tiles = kt;
    w.per_chunk = (kDown ? a.N : 2 * a.I) / 32;
    const uint32_t ld = (lane >> 3) * 512 + (lane & 7) * 64 + (((lane >> 1) & 3) << 4);   // ldmatrix: row lane % 8 of quarter lane / 8

    int begin, end, r, z = 0;   // the CTA's items; the next one is number r of the table's chunk z
    moe_find_items(a, blockIdx.x, gridDim.x, w.per_chunk, reinterpret_cast<int32_t *>(panel), table, begin, end, r);
    if constexpr (kDown)
        if (begin >= end) griddep_wait();   // nothing after this grid runs before kernel 1 ends
    for (int from = begin; from < end;) {
        // a phase: the items of as many chunks as have their panel rows in shared memory at a time
        int chunks = 0, rows = 0, to = from;
        while (to < end && chunks < kMoeMaxPanels && rows + table[z + chunks].rows <= a.panel_rows) {
            rows += table[z + chunks].rows;
            to = min(end, to + w.per_chunk - (chunks == 0 ? r : 0));
            ++chunks;
        }
        const int total = (to - from) * kt;
        auto cut = [&](int i) { return static_cast<int>(static_cast<int64_t>(total) * i / kMoeWarps); };
        const int first = cut(warp), last = cut(warp + 1);
        int item_z = z, item_r = first / kt;   // where this warp starts
        int tile = first - item_r * kt;
        item_r += r;
        for (; item_r >= w.per_chunk; item_r -= w.per_chunk) ++item_z;
        if constexpr (kDown) w.start(item_z, item_r, tile, last - first);
        for (int i = threadIdx.x; i < chunks * 8 * kNt; i += kMoeThreads) {
            int at = i % (8 * kNt);
            const MoeChunk ch = table[z + i / (8 * kNt)];
            if (at >= ch.rows) continue;
            const int src = kDown ? ch.row0 + at : min(max(__ldcg(a.row_index + ch.row0 + at), 0), a.T - 1);
            for (int c = 0; c < i / (8 * kNt); ++c) at += table[z + c].rows;
            s_rows[at] = {i / (8 * kNt), src};
        }
        for (int i = threadIdx.x; i < chunks * kt; i += kMoeThreads) flags[i] = 0;
        if constexpr (kDown)
            if (from == begin) griddep_wait();
        __syncthreads();
        // kernel 1 has its operands on their way before the weights queue up behind them
        moe_fill_panels<kDown>(a, table + z, s_rows, rows, panel, xs, flags, [&] {
            if (!kDown) w.start(item_z, item_r, tile, last - first);
        });
        __syncthreads();

        float acc[2][kNt][4] = {};
        bool whole = tile == 0;   // the piece in acc starts its item
        const uint8_t *bcol[kNt];
        const float *x0[kNt], *x1[kNt];
        const int32_t *flag = nullptr;
        auto open = [&]() {
            int base = 0;
            for (int c = z; c < item_z; ++c) base += table[c].rows;
            const int most = table[item_z].rows - 1;   // columns past the chunk's rows read its last row and go nowhere
#pragma unroll
            for (int n = 0; n < kNt; ++n) {
                bcol[n] = panel + (base + min(8 * n + g, most)) * stride + t * 16;
                x0[n] = xs + (base + min(8 * n + 2 * t, most)) * kt * 4;
                x1[n] = xs + (base + min(8 * n + 2 * t + 1, most)) * kt * 4;
            }
            flag = flags + (item_z - z) * kt;
        };
        if (first < last) open();
        int slot = 0;
#pragma unroll 1
        for (int j = first; j < last; ++j) {
            cp_async_wait<kMoeStages - 2>();
            __syncwarp();   // every lane's copies of this tile have landed, and every lane is done with the tile before
            w.issue();
            const uint32_t stage = w.ring + slot * kMoeStageBytes;
            slot = slot == kMoeStages - 1 ? 0 : slot + 1;
            uint32_t word[4];
            asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                         : "=r"(word[0]), "=r"(word[1]), "=r"(word[2]), "=r"(word[3])
                         : "r"(stage + 2048 + 16 * g)
                         : "memory");
            if (flag[tile]) moe_tile_mma<kNt, true>(stage + ld, word, bcol, x0, x1, tile, acc);
            else moe_tile_mma<kNt, false>(stage + ld, word, bcol, x0, x1, tile, acc);
            if (++tile == kt) {
                if (whole) {
                    moe_store_item<kDown, kNt>(a, table[item_z], item_r, acc, lane);
                } else {
#pragma unroll
                    for (int i = 0; i < 8 * kNt; ++i) heads[(warp * 8 * kNt + i) * 32 + lane] = acc[i / (4 * kNt)][i / 4 % kNt][i % 4];
                }
#pragma unroll
                for (int i = 0; i < 8 * kNt; ++i) acc[i / (4 * kNt)][i / 4 % kNt][i % 4] = 0.0f;
                tile = 0;
                whole = true;
                if (++item_r == w.per_chunk) {
                    item_r = 0;
                    ++item_z;
                    if (j + 1 < last) open();
                }
            }
        }
        float *tails = reinterpret_cast<float *>(s_moe + warp * kMoeStages * kMoeStageBytes);
        cp_async_wait<0>();
        __syncwarp();
        // a piece that its item's end does not close: the warp's first if it starts inside the item, else over its ring
        if (tile != 0 && first < last) {
            float *dst = whole ? tails : heads + warp * 8 * kNt * 32;
#pragma unroll
            for (int i = 0; i < 8 * kNt; ++i) dst[i * 32 + lane] = acc[i / (4 * kNt)][i / 4 % kNt][i % 4];
        }
        __syncthreads();
        // a cut item is closed by the first warp that starts inside it: the piece before, its own, and those after
        const int whole_items = first / kt;
        if (first != whole_items * kt && warp > 0 && cut(warp - 1) <= whole_items * kt) {
            const int stop = (whole_items + 1) * kt;
            const float *before = reinterpret_cast<const float *>(s_moe + (warp - 1) * kMoeStages * kMoeStageBytes);
#pragma unroll
            for (int i = 0; i < 8 * kNt; ++i) acc[i / (4 * kNt)][i / 4 % kNt][i % 4] = before[i * 32 + lane];
            for (int v = warp; v < kMoeWarps && cut(v) < stop; ++v) {
                if (cut(v) == cut(v + 1)) continue;
#pragma unroll
                for (int i = 0; i < 8 * kNt; ++i) acc[i / (4 * kNt)][i / 4 % kNt][i % 4] += heads[(v * 8 * kNt + i) * 32 + lane];
            }
            int it = r + whole_items, iz = z;
            for (; it >= w.per_chunk; it -= w.per_chunk) ++iz;
            moe_store_item<kDown, kNt>(a, table[iz], it, acc, lane);
        }
        r += to - from - (chunks - 1) * w.per_chunk;   // in the phase's last chunk
        z += chunks - 1;
        if (r == w.per_chunk) {
            r = 0;
            ++z;
        }
        from = to;
        if (from < end) __syncthreads();   // panels and pieces are read before the next phase writes them
    }
}

// Down and the weighted sum in one launch, for few rows: a cluster of `ranks` CTAs has 32 weight rows of every chunk's expert
// and sums its outputs over the chunks itself. The K tiles of all chunks, one chunk after the other, are cut into equal
// runs for the cluster's warps; a warp adds its pieces, times the rows' weights, to sums of its own per token, which
// meet through shared memory, then through distributed shared memory, always in the same order. It saves a launch, 2 us of the
// host's time, and for one token some of the GPU's (top-8: 15.7 against 16.0 us; two experts of 4096 x 2048 17.1 against 18.1);
// but every CTA makes the panels of all its chunks, so that with 24 rows it is slower (25.1 against 23.9), with 16 even.
__global__ void __launch_bounds__(kMoeThreads, 1) moe_down_sum_kernel(MoeArgs a, int ranks) {
    extern __shared__ __align__(128) uint8_t s_moe[];
    __shared__ MoeRow s_rows[kMoeFewRows];
    __shared__ int32_t s_token[kMoeFewRows];   // of a sorted row, -1 for none
    __shared__ float s_weight[kMoeFewRows];
    __shared__ __align__(8) float s_sum[kMoeFewTokens * 32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, t = lane & 3;
    griddep_launch_dependents();   // kernel 1 has waited for everything before it: the plan and the weights are complete
    const int rank = blockIdx.x % ranks, item = blockIdx.x / ranks;
    const int kt = a.I / 128, stride = moe_panel_stride(kt);
    float *part = reinterpret_cast<float *>(s_moe + moe_heads_offset()) + warp * kMoeFewTokens * 32;   // [token][weight row]
    uint8_t *panel = s_moe + moe_panels_offset(1);
    float *xs = reinterpret_cast<float *>(panel + a.R * stride);
    int32_t *flags = reinterpret_cast<int32_t *>(panel + a.R * moe_row_bytes(kt));   // [chunk][tile]
    MoeChunk *table = reinterpret_cast<MoeChunk *>(flags + a.R * kt);
    if (threadIdx.x < kMoeFewRows) {
        s_rows[threadIdx.x] = {0, 0};
        s_token[threadIdx.x] = -1;
    }
    for (int i = threadIdx.x; i < a.R * kt; i += kMoeThreads) flags[i] = 0;
    for (int i = lane; i < kMoeFewTokens * 32; i += 32) part[i] = 0.0f;

    int begin, chunks, none;
    moe_find_items(a, 0, 1, 1, reinterpret_cast<int32_t *>(s_moe), table, begin, chunks, none);   // every chunk
    const int units = chunks * kt, u0 = units * rank / ranks, u1 = units * (rank + 1) / ranks;
    const int first = u0 + (u1 - u0) * warp / kMoeWarps, last = u0 + (u1 - u0) * (warp + 1) / kMoeWarps;
    const int z0 = u0 / kt, z1 = u1 > u0 ? (u1 - 1) / kt : z0 - 1;   // the chunks of this CTA
    int z = first / kt, tile = first - z * kt;
    MoeStream<true> w;
    w.wq = a.wq_dn, w.wsf = a.wsf_dn, w.table = table;
    w.ring = smem_u32(s_moe) + warp * kMoeStages * kMoeStageBytes;
    w.st = g * 64 + ((t ^ ((g >> 1) & 3)) << 4);
    w.K = a.I, w.tiles = kt, w.per_chunk = a.N / 32;
    w.start(z, item, tile, last - first);
    // panel rows are the chunks' rows, from the first chunk's on (kept in range where a plan's offsets overlap)
    auto panel_row = [&](int row) { return min(max(row - table[z0].row0, 0), a.R - 1); };
    for (int i = threadIdx.x; i < (z1 - z0 + 1) * 8; i += kMoeThreads) {
        const MoeChunk ch = table[z0 + i / 8];
        if (i % 8 < ch.rows) s_rows[panel_row(ch.row0 + i % 8)] = {i / 8, ch.row0 + i % 8};
    }
    const int32_t live = min(max(__ldcg(a.offsets + a.E), 0), a.R);
    for (int i = threadIdx.x; i < a.R; i += kMoeThreads) {
        const int32_t row = __ldcg(a.pos + i);
        if (row >= 0 && row < live) {
            s_token[row] = i / a.topk;
            s_weight[row] = __ldcg(a.weights + i);
        }
    }
    griddep_wait();   // kernel 1's rows; out may still be in use
    __syncthreads();
    const int rows = z1 < z0 ? 0 : panel_row(table[z1].row0 + table[z1].rows - 1) + 1;
    moe_fill_panels<true>(a, table + z0, s_rows, rows, panel, xs, flags, [] {});
    __syncthreads();

    float acc[2][1][4] = {};
    const uint8_t *bcol[1];
    const float *x0[1], *x1[1];
    const uint32_t ld = (lane >> 3) * 512 + (lane & 7) * 64 + (((lane >> 1) & 3) << 4);
    auto open = [&]() {
        const int base = table[z].row0, most = table[z].rows - 1;
        bcol[0] = panel + panel_row(base + min(g, most)) * stride + t * 16;
        x0[0] = xs + panel_row(base + min(2 * t, most)) * kt * 4;
        x1[0] = xs + panel_row(base + min(2 * t + 1, most)) * kt * 4;
    };
    if (first < last) open();
    int slot = 0;
#pragma unroll 1
    for (int j = first; j < last; ++j) {
        cp_async_wait<kMoeStages - 2>();
        __syncwarp();   // every lane's copies of this tile have landed, and every lane is done with the tile before
        w.issue();
        const uint32_t stage = w.ring + slot * kMoeStageBytes;
        slot = slot == kMoeStages - 1 ? 0 : slot + 1;
        uint32_t word[4];
        asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                     : "=r"(word[0]), "=r"(word[1]), "=r"(word[2]), "=r"(word[3])
                     : "r"(stage + 2048 + 16 * g)
                     : "memory");
        if (flags[(z - z0) * kt + tile]) moe_tile_mma<1, true>(stage + ld, word, bcol, x0, x1, tile, acc);
        else moe_tile_mma<1, false>(stage + ld, word, bcol, x0, x1, tile, acc);
        if (++tile < kt && j + 1 < last) continue;
        // the end of the chunk or of the run. Row by row, since a token may have chosen an expert twice.
        const MoeChunk ch = table[z];
        for (int c = 0; c < ch.rows; ++c) {
            const int token = s_token[ch.row0 + c];
            if (t == c >> 1 && token >= 0) {
                const float weight = s_weight[ch.row0 + c];
#pragma unroll
                for (int m = 0; m < 2; ++m)
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        float *at = part + token * 32 + 8 * (2 * m + h) + g;
                        *at = fmaf(weight, (c & 1) ? acc[m][0][2 * h + 1] : acc[m][0][2 * h], *at);
                    }
            }
            __syncwarp();
        }
#pragma unroll
        for (int m = 0; m < 2; ++m)
#pragma unroll
            for (int k = 0; k < 4; ++k) acc[m][0][k] = 0.0f;
        tile = 0;
        ++z;
        if (j + 1 < last) open();
    }
    cp_async_wait<0>();
    __syncthreads();
    const float *parts = reinterpret_cast<const float *>(s_moe + moe_heads_offset());
    if (threadIdx.x < a.T * 32) {
        float sum = 0.0f;
#pragma unroll
        for (int v = 0; v < kMoeWarps; ++v) sum += parts[v * kMoeFewTokens * 32 + threadIdx.x];
        s_sum[threadIdx.x] = sum;
    }
    cluster_sync();
    if (const int i = threadIdx.x; rank == 0 && i < a.T * 16) {   // two outputs each
        float v0 = 0.0f, v1 = 0.0f;
        for (int c = 0; c < ranks; ++c) {
            float a0, a1;
            asm volatile("ld.shared::cluster.v2.f32 {%0, %1}, [%2];"
                         : "=f"(a0), "=f"(a1)
                         : "r"(map_to_rank(smem_u32(s_sum + 2 * i), c))
                         : "memory");
            v0 += a0, v1 += a1;
        }
        const int token = i / 16, q = i % 16 / 4, at = 2 * (i % 4);
        const __nv_bfloat162 o = __floats2bfloat162_rn(v0, v1);
        *reinterpret_cast<__nv_bfloat162 *>(a.out + static_cast<int64_t>(token) * a.N + 128 * (item >> 2) + 32 * q + 8 * (item & 3) + at) = o;
    }
    cluster_sync();   // no CTA leaves while another reads its sums
}

// The weighted sum of each token's choices, in the order j = 0, 1, ...: a warp takes 128 outputs of a token.
constexpr int kMoeSumWarps = 4;
__global__ void __launch_bounds__(32 * kMoeSumWarps) moe_sum_kernel(MoeArgs a) {
    griddep_launch_dependents();
    const int lane = threadIdx.x & 31, blocks = a.N / 128;
    const int id = blockIdx.x * kMoeSumWarps + (threadIdx.x >> 5);
    if (id >= a.T * blocks) {
        griddep_wait();
        return;
    }
    const int t = id / blocks, n = 128 * (id - t * blocks) + 4 * lane;
    const int32_t live = min(max(__ldcg(a.offsets + a.E), 0), a.R);
    int32_t p = -1;
    float wt = 0.0f;
    if (lane < a.topk) {
        p = __ldcg(a.pos + t * a.topk + lane);
        wt = __ldcg(a.weights + t * a.topk + lane);
        if (p >= live) p = -1;
    }
    griddep_wait();   // the rows of kernel 2; the plan is older
    float s[4] = {};
    for (int j0 = 0; j0 < a.topk; j0 += 8) {
        float4 u[8];
        float wj[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {   // eight rows in flight
            const int32_t r = __shfl_sync(0xffffffffu, p, (j0 + j) & 31);
            wj[j] = __shfl_sync(0xffffffffu, wt, (j0 + j) & 31);
            u[j] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
            if (j0 + j < a.topk && r >= 0) u[j] = __ldcg(reinterpret_cast<const float4 *>(a.y + static_cast<int64_t>(r) * a.N + n));
            else wj[j] = 0.0f;
        }
#pragma unroll
        for (int j = 0; j < 8; ++j)
            s[0] = fmaf(wj[j], u[j].x, s[0]), s[1] = fmaf(wj[j], u[j].y, s[1]), s[2] = fmaf(wj[j], u[j].z, s[2]),
            s[3] = fmaf(wj[j], u[j].w, s[3]);
    }
    const __nv_bfloat162 lo = __floats2bfloat162_rn(s[0], s[1]), hi = __floats2bfloat162_rn(s[2], s[3]);
    *reinterpret_cast<uint2 *>(a.out + static_cast<int64_t>(t) * a.N + n) =
        make_uint2(*reinterpret_cast<const uint32_t *>(&lo), *reinterpret_cast<const uint32_t *>(&hi));
}

}  // namespace macaq
