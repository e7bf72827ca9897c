// Dense product of bf16 activations and weights with bias, activation, gate
// and residual in its epilogue (k3moe_linear).
#pragma once

#include "common.cuh"

namespace k3 {

struct LinearParams {
    const uint16_t *x;         // bf16, T rows, ldx elements apart
    const uint16_t *w, *wg;    // bf16, N rows, ldw elements apart (wg: null, or the gate's)
    const float *bias, *bias_g;
    const void *resid;         // T rows, ldr elements apart, or null
    void *out;                 // T rows, ldo elements apart
    long long ldx, ldw, ldr, ldo;
    int T, N, K, act, out_fp32;
};

// The activation of one pre-activation value, in fp32.
__device__ __forceinline__ float linear_act(float v, int act) {
    switch (act) {
        case K3MOE_ACT_RELU: return fmaxf(v, 0.f) + (v != v ? v : 0.f);
        case K3MOE_ACT_SILU: return v / (1.0f + expf(-v));
        case K3MOE_ACT_GELU: return 0.5f * v * erfcf(-0.70710678118654752f * v);
        case K3MOE_ACT_GELU_TANH:
            return 0.5f * v * (1.0f + tanhf(0.79788456080286536f * (v + 0.044715f * v * v * v)));
        default: return v;
    }
}

// Tiles of 64 tokens x 64 columns, K in steps of 16 through shared memory,
// 4 x 4 outputs per thread in fp32.
constexpr int kLinT = 64, kLinN = 64, kLinK = 16;
__global__ void __launch_bounds__(256) linear_kernel(const __grid_constant__ LinearParams p) {
    __shared__ float xs[kLinK][kLinT + 4], ws[2][kLinK][kLinN + 4];
    const int n0 = blockIdx.x * kLinN;
    const long long t0 = (long long)blockIdx.y * kLinT;
    const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
    float v[4][4] = {}, g[4][4] = {};
    for (int k0 = 0; k0 < p.K; k0 += kLinK) {
        for (int i = threadIdx.x; i < 64 * kLinK; i += 256) {
            const int r = i / kLinK, kk = i % kLinK;
            const bool kin = k0 + kk < p.K;
            xs[kk][r] = kin && t0 + r < p.T ? bf16_lo(p.x[(t0 + r) * p.ldx + k0 + kk]) : 0.f;
            const bool win = kin && n0 + r < p.N;
            ws[0][kk][r] = win ? bf16_lo(p.w[(n0 + r) * p.ldw + k0 + kk]) : 0.f;
            ws[1][kk][r] = win && p.wg ? bf16_lo(p.wg[(n0 + r) * p.ldw + k0 + kk]) : 0.f;
        }
        __syncthreads();
        for (int kk = 0; kk < kLinK; ++kk)
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    v[i][j] = fmaf(xs[kk][4 * ty + i], ws[0][kk][4 * tx + j], v[i][j]);
                    g[i][j] = fmaf(xs[kk][4 * ty + i], ws[1][kk][4 * tx + j], g[i][j]);
                }
        __syncthreads();
    }
    for (int i = 0; i < 4; ++i)
        for (int j = 0; j < 4; ++j) {
            const long long t = t0 + 4 * ty + i;
            const int n = n0 + 4 * tx + j;
            if (t >= p.T || n >= p.N) continue;
            float a = v[i][j] + (p.bias ? p.bias[n] : 0.f);
            if (p.wg)
                a = linear_act(g[i][j] + (p.bias_g ? p.bias_g[n] : 0.f), p.act) * a;
            else
                a = linear_act(a, p.act);
            if (p.resid)
                a += p.out_fp32 ? reinterpret_cast<const float *>(p.resid)[t * p.ldr + n]
                                : bf16_lo(reinterpret_cast<const uint16_t *>(p.resid)[t * p.ldr + n]);
            if (p.out_fp32)
                reinterpret_cast<float *>(p.out)[t * p.ldo + n] = a;
            else
                reinterpret_cast<uint16_t *>(p.out)[t * p.ldo + n] = __bfloat16_as_ushort(__float2bfloat16_rn(a));
        }
}

}  // namespace k3
