// moe_w4a16.cuh -- a whole mixture-of-experts layer for few tokens: MXFP4 weights, bf16 activations.
//
//   x'  = x diag(1/s_e) H_b                      (fp32; the weight-only mode's transform without its bf16 step)
//   g, u = gate and up rows of x' dq(W'_gu,e)^T    (64-row interleaved blocks)
//   h   = silu(g) u,  h' = h diag(1/s_down,e) H_b'
//   out[t] = sum_j weights[t, j] * (h'_{pos[t, j]} dq(W'_down,e)^T)
//
// First kernel: h of every routed row to the workspace (fp32). Second kernel: the down projection and the
// weighted sum of each token's choices, in the order j = 0, 1, ...
// Sources: glonce.com page on MACaQ, paragraph 3 (weight-only serving) and paragraph 5 (grouped matmul);
// aipolix.com page, paragraph 2 (the transform at the input of every linear).
#pragma once

#include <cuda_bf16.h>

#include "groups.cuh"
#include "ptx.cuh"
#include "route.cuh"
#include "w4a16.cuh"

namespace macaq {

constexpr int kMoeMaxT = 64;
constexpr int kMoeThreads = 128;

struct MoeArgs {
    const uint16_t *x;            // bf16 [T, K]
    const float *weights;         // [T, topk]
    const int32_t *offsets;       // [E + 1]
    const int32_t *row_index;     // [R]
    const int32_t *pos;           // [T, topk]
    const uint8_t *wq_gu, *wsf_gu;
    const uint8_t *wq_dn, *wsf_dn;
    const float *inv_gu, *inv_dn; // [E, K], [E, I] or nullptr
    float *h;                     // workspace [R, I]
    uint16_t *out;                // bf16 [T, N]
    int32_t T, topk, E, K, I, N, R, b_gu, b_dn;
};

// Expert of sorted row r by a linear look at the offsets (clamped to [0, R] as everywhere), or -1.
__device__ __forceinline__ int moe_expert(const MoeArgs &a, int32_t r) {
    int32_t lo = 0, found = -1;
    for (int e = 0; e < a.E; ++e) {
        int32_t hi = a.offsets[e + 1];
        hi = hi < lo ? lo : (hi > a.R ? a.R : hi);
        if (r >= lo && r < hi) found = e;
        lo = hi;
    }
    return found;
}

// In-place block Hadamard of v[0..n) in shared memory, order h = 1, 2, ..., b / 2.
__device__ __forceinline__ void fwht_shared(float *v, int n, int b) {
    for (int h = 1; h < b; h <<= 1) {
        for (int i = threadIdx.x; i < n / 2; i += blockDim.x) {
            const int k = (i / h) * 2 * h + i % h;
            const float p = v[k], q = v[k + h];
            v[k] = p + q;
            v[k + h] = p - q;
        }
        __syncthreads();
    }
}

// sum_k v[k] dq(W[n, k]) by one warp; code bytes of the row, its tiled scales.
__device__ __forceinline__ float mx_row_dot(const float *v, const uint8_t *codes, const uint8_t *sf, int n, int K, int lane) {
    float s = 0.0f;
    for (int g = lane; g < K / 32; g += 32) {
        const uint32_t E = sf[sf_offset(n, g, K / 128)];
        const float scale = E ? __uint_as_float(E << 23) : __uint_as_float(0x00400000u);
        const uint8_t *c = codes + static_cast<int64_t>(n) * (K / 2) + g * 16;
        float d = 0.0f;
        for (int i = 0; i < 16; ++i) {
            d = fmaf(v[32 * g + 2 * i], e2m1_to_float(c[i] & 15u), d);
            d = fmaf(v[32 * g + 2 * i + 1], e2m1_to_float(c[i] >> 4), d);
        }
        s = fmaf(d, scale, s);
    }
    return warp_sum(s);
}

__global__ void __launch_bounds__(kMoeThreads) moe_gate_up_kernel(MoeArgs a) {
    extern __shared__ float s_v[];
    griddep_wait();
    griddep_launch_dependents();
    const int r = blockIdx.x;
    const int e = moe_expert(a, r);
    if (e < 0) return;
    const int t = min(max(a.row_index[r], 0), a.T - 1);
    for (int k = threadIdx.x; k < a.K; k += blockDim.x) {
        const float x = __uint_as_float(static_cast<uint32_t>(a.x[static_cast<int64_t>(t) * a.K + k]) << 16);
        s_v[k] = a.inv_gu ? x * a.inv_gu[static_cast<int64_t>(e) * a.K + k] : x;
    }
    __syncthreads();
    fwht_shared(s_v, a.K, a.b_gu);
    const int64_t rows = 2 * static_cast<int64_t>(a.I);
    const uint8_t *codes = a.wq_gu + e * rows * (a.K / 2);
    const uint8_t *sf = a.wsf_gu + e * rows * (a.K / 32);
    const int lane = threadIdx.x & 31;
    for (int i = threadIdx.x >> 5; i < 64; i += kMoeThreads / 32) {
        const int n = 128 * blockIdx.y + i;
        const float g = mx_row_dot(s_v, codes, sf, n, a.K, lane);
        const float u = mx_row_dot(s_v, codes, sf, n + 64, a.K, lane);
        if (lane == 0) a.h[static_cast<int64_t>(r) * a.I + 64 * blockIdx.y + i] = g / (1.0f + expf(-g)) * u;
    }
}

__global__ void __launch_bounds__(kMoeThreads) moe_down_kernel(MoeArgs a) {
    extern __shared__ float s_v[];
    __shared__ float s_out[128];
    griddep_wait();
    griddep_launch_dependents();
    const int t = blockIdx.x;
    s_out[threadIdx.x] = 0.0f;
    for (int j = 0; j < a.topk; ++j) {
        const int32_t r = a.pos[t * a.topk + j];
        const int e = r >= 0 && r < a.R ? moe_expert(a, r) : -1;
        if (e < 0) continue;
        __syncthreads();
        for (int k = threadIdx.x; k < a.I; k += blockDim.x) {
            const float h = a.h[static_cast<int64_t>(r) * a.I + k];
            s_v[k] = a.inv_dn ? h * a.inv_dn[static_cast<int64_t>(e) * a.I + k] : h;
        }
        __syncthreads();
        fwht_shared(s_v, a.I, a.b_dn);
        const uint8_t *codes = a.wq_dn + static_cast<int64_t>(e) * a.N * (a.I / 2);
        const uint8_t *sf = a.wsf_dn + static_cast<int64_t>(e) * a.N * (a.I / 32);
        const float w = a.weights[t * a.topk + j];
        const int lane = threadIdx.x & 31;
        for (int i = threadIdx.x >> 5; i < 128; i += kMoeThreads / 32) {
            const float y = mx_row_dot(s_v, codes, sf, 128 * blockIdx.y + i, a.I, lane);
            if (lane == 0) s_out[i] += w * y;
        }
    }
    __syncthreads();
    const __nv_bfloat16 o = __float2bfloat16_rn(s_out[threadIdx.x]);
    a.out[static_cast<int64_t>(t) * a.N + 128 * blockIdx.y + threadIdx.x] = *reinterpret_cast<const uint16_t *>(&o);
}

}  // namespace macaq
