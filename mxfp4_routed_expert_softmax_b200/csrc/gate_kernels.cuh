// Routing from given logits (k3moe_gate): scores, balance bias, groups, top-k.
#pragma once

#include "common.cuh"

namespace k3 {

constexpr int kGateMaxE = 1024;
constexpr int kGateMaxK = 32;

struct GateParams {
    const void *logits;  // fp32 or bf16, T rows, ld elements apart
    long long ld;
    int T, E, k;
    const float *bias;   // fp32 [E] or null
    int sigmoid, groups, kept, group_top, renorm, bf16;
    float scale;
    int32_t *idx;        // [T][k]
    float *weight;       // [T][k]
};

// One warp per token, the values it ranks by in shared memory as 64-bit
// numbers; every pick is a warp-wide maximum over them.
__global__ void __launch_bounds__(32) gate_kernel(const __grid_constant__ GateParams p) {
    __shared__ double s_order[kGateMaxE];  // c_e, or the logit where there is no bias; -inf: out
    __shared__ float s_l[kGateMaxE];
    __shared__ double s_group[32];
    __shared__ float s_w[kGateMaxK];
    const int lane = threadIdx.x;
    const double ninf = -INFINITY;
    for (long long t = blockIdx.x; t < p.T; t += gridDim.x) {
        float mx = -INFINITY;
        bool any_nan = false;
        for (int e = lane; e < p.E; e += 32) {
            const float l = p.bf16 ? __bfloat162float(reinterpret_cast<const __nv_bfloat16 *>(p.logits)[t * p.ld + e])
                                   : reinterpret_cast<const float *>(p.logits)[t * p.ld + e];
            s_l[e] = l;
            any_nan |= l != l;
            mx = fmaxf(mx, l);
        }
        for (int o = 16; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
        const bool bad = __any_sync(0xffffffffu, any_nan) || mx == INFINITY;  // the softmax is NaN
        double sum = 0.0;
        if (!p.sigmoid) {
            for (int e = lane; e < p.E; e += 32)
                if (s_l[e] > -INFINITY) sum += exp((double)s_l[e] - (double)mx);
            for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
        }
        auto score = [&](int e) -> double {
            const double l = s_l[e];
            if (p.sigmoid) return 1.0 / (1.0 + exp(-l));
            return bad ? (double)NAN : exp(l - (double)mx) / sum;
        };
        for (int e = lane; e < p.E; e += 32) {
            double c = s_l[e];
            if (p.bias && c > ninf) c = score(e) + (double)p.bias[e];
            s_order[e] = c > ninf && s_l[e] > -INFINITY ? c : ninf;
        }
        __syncwarp();
        if (p.groups > 1) {
            const int gs = p.E / p.groups;
            if (lane < p.groups) {
                double a = ninf, b = ninf;
                for (int e = lane * gs; e < (lane + 1) * gs; ++e) {
                    double c = s_order[e];
                    if (c > ninf && !p.bias && p.group_top > 1) {
                        c = score(e);
                        if (!(c > ninf)) c = ninf;
                    }
                    if (c > a) {
                        b = a;
                        a = c;
                    } else if (c > b) {
                        b = c;
                    }
                }
                s_group[lane] = p.group_top > 1 ? (b > ninf ? a + b : ninf) : a;
            }
            __syncwarp();
            bool keep = false;
            if (lane < p.groups) {
                int r = 0;
                for (int g = 0; g < p.groups; ++g)
                    r += s_group[g] > s_group[lane] || (s_group[g] == s_group[lane] && g < lane) ? 1 : 0;
                keep = r < p.kept;
                if (!keep)
                    for (int e = lane * gs; e < (lane + 1) * gs; ++e) s_order[e] = ninf;
            }
            __syncwarp();
        }
        int mine = -1;  // lane j: pick j
        for (int j = 0; j < p.k; ++j) {
            double best = ninf;
            int at = 0x7FFFFFFF;
            for (int e = lane; e < p.E; e += 32)
                if (s_order[e] > best) {
                    best = s_order[e];
                    at = e;
                }
            for (int o = 16; o > 0; o >>= 1) {
                const double v = __shfl_xor_sync(0xffffffffu, best, o);
                const int a = __shfl_xor_sync(0xffffffffu, at, o);
                if (v > best || (v == best && a < at)) {
                    best = v;
                    at = a;
                }
            }
            if (!(best > ninf)) break;
            if (lane == j) mine = at;
            if (lane == (at & 31)) s_order[at] = ninf;
            __syncwarp();
        }
        const double w = mine >= 0 ? score(mine) : 0.0;
        double z = w;
        for (int o = 16; o > 0; o >>= 1) z += __shfl_xor_sync(0xffffffffu, z, o);
        if (lane < p.k) {
            p.idx[t * p.k + lane] = mine;
            p.weight[t * p.k + lane] = (float)((p.renorm ? (z == 0.0 ? 0.0 : w / z) : w) * (double)p.scale);
        }
        __syncwarp();
    }
}

}  // namespace k3
