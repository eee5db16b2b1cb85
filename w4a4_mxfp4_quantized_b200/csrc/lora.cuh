// lora.cuh -- low-rank adapters of many requests beside a shared projection.
//
//   out[m, :] = Y[m, :] + scale[a] * (X[m, :] A[a]^T) B[a]^T     for the rows m of adapter a
//
// Rows come sorted by adapter through group_offsets and row_index (a row plan); rows of no adapter are copied when
// out is not Y. X A^T is held in fp32.
#pragma once

#include <cuda_bf16.h>

#include "groups.cuh"
#include "ptx.cuh"
#include "route.cuh"

namespace macaq {

constexpr int kLoraThreads = 256;
constexpr int kLoraMaxRank = 128;

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
    int32_t r, L, f32;
};

__device__ __forceinline__ float bf16_value(uint16_t v) { return __uint_as_float(static_cast<uint32_t>(v) << 16); }

__global__ void __launch_bounds__(kLoraThreads) lora_add_kernel(LoraArgs p) {
    __shared__ float s_v[kLoraMaxRank];
    griddep_wait();
    griddep_launch_dependents();
    const int64_t s = blockIdx.x;
    int a = -1;
    int64_t lo = 0;
    for (int g = 0; g < p.L; ++g) {
        int64_t hi = p.offsets[g + 1];
        hi = hi < lo ? lo : (hi > p.M ? p.M : hi);
        if (s >= lo && s < hi) a = g;
        lo = hi;
    }
    const int64_t m = p.row_index ? p.row_index[s] : s;
    if (m < 0 || m >= p.M || (a < 0 && p.out == p.y)) return;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (a >= 0)
        for (int j = warp; j < p.r; j += kLoraThreads / 32) {
            const uint16_t *row = p.A + (static_cast<int64_t>(a) * p.r + j) * p.K;
            float v = 0.0f;
            for (int64_t k = lane; k < p.K; k += 32) v = fmaf(bf16_value(p.x[m * p.ldx + k]), bf16_value(row[k]), v);
            v = warp_sum(v);
            if (lane == 0) s_v[j] = p.scale ? v * p.scale[a] : v;
        }
    __syncthreads();
    for (int64_t n = threadIdx.x; n < p.N; n += kLoraThreads) {
        float v = p.f32 ? static_cast<const float *>(p.y)[m * p.ldy + n]
                        : bf16_value(static_cast<const uint16_t *>(p.y)[m * p.ldy + n]);
        if (a >= 0) {
            const uint16_t *row = p.B + (static_cast<int64_t>(a) * p.N + n) * p.r;
            float d = 0.0f;
            for (int j = 0; j < p.r; ++j) d = fmaf(s_v[j], bf16_value(row[j]), d);
            v += d;
        }
        if (p.f32) static_cast<float *>(p.out)[m * p.ldo + n] = v;
        else static_cast<__nv_bfloat16 *>(p.out)[m * p.ldo + n] = __float2bfloat16_rn(v);
    }
}

}  // namespace macaq
