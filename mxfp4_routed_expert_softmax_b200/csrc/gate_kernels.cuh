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
    int vec;             // four logits of a row (and the bias) can be loaded at once
    int gsize, glanes_log2;  // experts of a group; log2 of the lanes that scan one (groups << it at most 32)
    uint32_t gmul;           // e / gsize = e gmul >> 20 for e < 1024
    float scale;
    int32_t *idx;        // [T][k]
    float *weight;       // [T][k]
};

__device__ __forceinline__ float gate_logit(const GateParams &p, long long t, int e) {
    return p.bf16 ? __bfloat162float(reinterpret_cast<const __nv_bfloat16 *>(p.logits)[t * p.ld + e])
                  : reinterpret_cast<const float *>(p.logits)[t * p.ld + e];
}

__device__ __forceinline__ double warp_sum(double v) {
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

// One token in 64 bits throughout, by one warp: what the definition says, one
// pick after the other.  The tokens that gate_kernel cannot settle in 32 bits
// come here.
struct GateExact {
    double order[kGateMaxE];  // c_e, or the logit where there is no bias; -inf: out
    float l[kGateMaxE];
    double group[32];
};
__device__ __noinline__ void gate_exact(const GateParams &p, long long t, GateExact &s) {
    const int lane = threadIdx.x & 31;
    const double ninf = -INFINITY;
    float mx = -INFINITY;
    bool any_nan = false;
    for (int e = lane; e < p.E; e += 32) {
        const float l = gate_logit(p, t, e);
        s.l[e] = l;
        any_nan |= l != l;
        mx = fmaxf(mx, l);
    }
    for (int o = 16; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
    const bool bad = __any_sync(0xffffffffu, any_nan) || mx == INFINITY;  // the softmax is NaN
    double sum = 0.0;
    if (!p.sigmoid) {
        for (int e = lane; e < p.E; e += 32)
            if (s.l[e] > -INFINITY) sum += exp((double)s.l[e] - (double)mx);
        sum = warp_sum(sum);
    }
    auto score = [&](int e) -> double {
        const double l = s.l[e];
        if (p.sigmoid) return 1.0 / (1.0 + exp(-l));
        return bad ? (double)NAN : exp(l - (double)mx) / sum;
    };
    for (int e = lane; e < p.E; e += 32) {
        double c = s.l[e];
        if (p.bias && c > ninf) c = score(e) + (double)p.bias[e];
        s.order[e] = c > ninf && s.l[e] > -INFINITY ? c : ninf;
    }
    __syncwarp();
    if (p.groups > 1) {
        const int gs = p.E / p.groups;
        if (lane < p.groups) {
            double a = ninf, b = ninf;
            for (int e = lane * gs; e < (lane + 1) * gs; ++e) {
                double c = s.order[e];
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
            s.group[lane] = p.group_top > 1 ? (b > ninf ? a + b : ninf) : a;
        }
        __syncwarp();
        if (lane < p.groups) {
            int r = 0;
            for (int g = 0; g < p.groups; ++g)
                r += s.group[g] > s.group[lane] || (s.group[g] == s.group[lane] && g < lane) ? 1 : 0;
            if (r >= p.kept)
                for (int e = lane * gs; e < (lane + 1) * gs; ++e) s.order[e] = ninf;
        }
        __syncwarp();
    }
    int mine = -1;  // lane j: pick j
    for (int j = 0; j < p.k; ++j) {
        double best = ninf;
        int at = 0x7FFFFFFF;
        for (int e = lane; e < p.E; e += 32)
            if (s.order[e] > best) {
                best = s.order[e];
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
        if (lane == (at & 31)) s.order[at] = ninf;
        __syncwarp();
    }
    const double w = mine >= 0 ? score(mine) : 0.0;
    const double z = warp_sum(w);
    if (lane < p.k) {
        p.idx[t * p.k + lane] = mine;
        p.weight[t * p.k + lane] = (float)((p.renorm ? (z == 0.0 ? 0.0 : w / z) : w) * (double)p.scale);
    }
}

// One warp per token, its logits in registers (lane l holds ids 128 i + 4 l
// to + 3): no exchange between warps, and 4096 tokens fill the device once.  The selection is a filter with an error bound:
//   - without a bias the ranking is the logits' own and exact; with one the
//     values c_e are formed in 32 bits, each within eps of the true one
//     (sigmoid scores first by the hardware's tanh, within 2^-10);
//   - the k-th largest of the 32 lanes' maxima is a value that at least k
//     values reach, so only those no more than 2 eps below it can be among the
//     k largest (about 22 of 896 for k = 16): they go to a list, where sigmoid
//     scores are formed again more exactly;
//   - each candidate's place is the number of larger ones (ties to the lower
//     id); where two neighbours of the list are within 2 eps, the candidates'
//     values are formed again in 64 bits and placed by those.
// What cannot be settled so (groups whose values are within the error, more
// than kGateCap candidates, infinite biases, scores below 2^-100) goes through
// gate_exact, so the result is that of the 64-bit definition in every case.
// Weights are 32-bit: the scores of the picks from expf, the softmax's argument
// l - max with its rounding error carried along.
//
// Bound by one wave's load and chain of steps as much as by instruction issue:
// about 1000 instructions a token of 896 experts (3.6 kB), half of the issue
// slots filled, so 4096 tokens, softmax, top 16, take 6.7 us where their
// instructions take 3.5 and their bytes 2.3 (8.0 us with a compare and a store
// per logit, 45 us with a warp-wide maximum per pick over 64-bit values in
// shared memory).  8191 tokens, sigmoid with a bias: 15.5 us (bytes 4.6), of
// which one in some hundred tokens needs 64 bits.  A single token: 3.0 us, the
// chain of the steps above.
constexpr int kGateWarps = 4;
constexpr int kGateCap = 160;  // a multiple of 8
struct alignas(16) GateWarp {
    uint64_t key[kGateCap];   // value (order-preserving bits) above the inverted id
    double exact[kGateCap];
    uint32_t top[32];
    float sorted[kGateMaxK + 1];
    int32_t id[kGateMaxK + 1];
};
static_assert(sizeof(GateWarp) % 16 == 0, "16-byte parts of shared memory");

__host__ __device__ inline int gate_smem(int ni) {
    const int warps = kGateWarps * ((int)sizeof(GateWarp) + ni * 512);
    return warps > (int)sizeof(GateExact) ? warps : (int)sizeof(GateExact);
}

__device__ __forceinline__ uint32_t order_bits(float v) {
    const uint32_t b = __float_as_uint(v);
    return b ^ ((uint32_t)((int32_t)b >> 31) | 0x80000000u);
}
__device__ __forceinline__ float from_order_bits(uint32_t b) {
    return __uint_as_float(b & 0x80000000u ? b ^ 0x80000000u : ~b);
}
__device__ __forceinline__ float ex2_approx(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ float rcp_approx(float x) {
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ float tanh_approx(float x) {
    float y;
    asm("tanh.approx.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

template <int NI, bool BIAS>
__global__ void __launch_bounds__(32 * kGateWarps) gate_kernel(const __grid_constant__ GateParams p) {
    extern __shared__ __align__(16) uint8_t gate_raw[];
    constexpr int N = 4 * NI;
    constexpr float kLog2e = 1.44269504088896341f;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    GateWarp &s = *reinterpret_cast<GateWarp *>(gate_raw + warp * (sizeof(GateWarp) + NI * 512));
    float *val = reinterpret_cast<float *>(&s + 1);  // [128 NI] what the experts are ranked by
    const long long t = (long long)blockIdx.x * kGateWarps + warp;
    const float ninf = -INFINITY;
    const uint32_t all = 0xffffffffu;
    pdl_wait();
    pdl_trigger();
    bool unsettled = false;
    if (t < p.T) {
        float o[N], b[BIAS ? N : 1];  // o: the logits, then what the experts are ranked by
#pragma unroll
        for (int i = 0; i < NI; ++i) {
            const int e = 128 * i + 4 * lane;
            if (p.vec && e + 4 <= p.E) {
                if (p.bf16) {
                    const uint2 v = *reinterpret_cast<const uint2 *>(reinterpret_cast<const uint16_t *>(p.logits) + t * p.ld + e);
                    o[4 * i] = bf16_lo(v.x), o[4 * i + 1] = bf16_hi(v.x), o[4 * i + 2] = bf16_lo(v.y), o[4 * i + 3] = bf16_hi(v.y);
                } else {
                    const float4 v = *reinterpret_cast<const float4 *>(reinterpret_cast<const float *>(p.logits) + t * p.ld + e);
                    o[4 * i] = v.x, o[4 * i + 1] = v.y, o[4 * i + 2] = v.z, o[4 * i + 3] = v.w;
                }
            } else {
#pragma unroll
                for (int c = 0; c < 4; ++c) o[4 * i + c] = e + c < p.E ? gate_logit(p, t, e + c) : ninf;
            }
            if constexpr (BIAS) {
                if (p.vec && e + 4 <= p.E) {
                    const float4 v = *reinterpret_cast<const float4 *>(p.bias + e);
                    b[4 * i] = v.x, b[4 * i + 1] = v.y, b[4 * i + 2] = v.z, b[4 * i + 3] = v.w;
                } else {
#pragma unroll
                    for (int c = 0; c < 4; ++c) b[4 * i + c] = e + c < p.E ? p.bias[e + c] : 0.f;
                }
            }
        }
        float lm = ninf, mx = ninf, sum = 0.f, inv = 0.f;  // lm: the lane's largest
        if (!BIAS || !p.sigmoid) {
#pragma unroll
            for (int i = 0; i < N; ++i) lm = fmaxf(lm, o[i]);  // passes over NaN
        }
        if (!p.sigmoid) {
            mx = from_order_bits(__reduce_max_sync(all, order_bits(lm)));
            // NaN and +inf logits make the sum NaN, as the formula does; the
            // exponential's error (2 units and |x| half units) is small where
            // the term is
            if (mx > ninf) {
                float part[4] = {};
#pragma unroll
                for (int i = 0; i < N; ++i) part[i % 4] += ex2_approx((o[i] - mx) * kLog2e);
                sum = (part[0] + part[1]) + (part[2] + part[3]);
                for (int q = 16; q > 0; q >>= 1) sum += __shfl_xor_sync(all, sum, q);
                inv = 1.0f / sum;  // the largest score
            }
        }
        // A score in 32 bits: within 2^-20 (sigmoid) or 2^-18 of the largest (softmax).
        auto rough = [&](float v) {
            return p.sigmoid ? rcp_approx(1.0f + ex2_approx(-v * kLog2e)) : ex2_approx((v - mx) * kLog2e) * inv;
        };
        const float fine = p.sigmoid ? 0x1p-20f : inv * 0x1p-18f;
        const bool scores = !BIAS && p.groups > 1 && p.group_top > 1;  // groups are compared by scores
        const bool coarse = BIAS && p.sigmoid && p.groups == 1;
        if constexpr (BIAS) {
            if (coarse) {
#pragma unroll
                for (int i = 0; i < N; ++i) {
                    const float c = fmaf(0.5f, tanh_approx(0.5f * o[i]), 0.5f + b[i]);
                    o[i] = o[i] > ninf ? fmaxf(c, ninf) : ninf;  // NaN: out
                }
            } else {
#pragma unroll
                for (int i = 0; i < N; ++i) {
                    const float c = rough(o[i]) + b[i];
                    o[i] = o[i] > ninf ? fmaxf(c, ninf) : ninf;
                }
            }
        } else {
#pragma unroll
            for (int i = 0; i < N; ++i) o[i] = fmaxf(o[i], ninf);  // NaN: out
        }
        if (p.groups > 1) {
            // lp lanes scan a group for its one or two largest values
            const int gs = p.gsize, lp = 1 << p.glanes_log2;
            float amax = 0.f;
#pragma unroll
            for (int i = 0; i < NI; ++i) {
                float v[4];
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    v[c] = o[4 * i + c];
                    if (scores && v[c] > ninf) v[c] = fmaxf(rough(v[c]), ninf);
                    if (v[c] > ninf) amax = fmaxf(amax, fabsf(v[c]));
                }
                *reinterpret_cast<float4 *>(val + 128 * i + 4 * lane) = make_float4(v[0], v[1], v[2], v[3]);
            }
            __syncwarp();
            const int g = lane >> p.glanes_log2;
            float x1 = ninf, x2 = ninf;
            if (g < p.groups)
                for (int e = lane & (lp - 1); e < gs; e += 4 * lp) {
                    float v[4];
#pragma unroll
                    for (int c = 0; c < 4; ++c) v[c] = e + c * lp < gs ? val[g * gs + e + c * lp] : ninf;
#pragma unroll
                    for (int c = 0; c < 4; ++c) {
                        x2 = fmaxf(x2, fminf(x1, v[c]));
                        x1 = fmaxf(x1, v[c]);
                    }
                }
            for (int q = 1; q < lp; q <<= 1) {
                const float y1 = __shfl_xor_sync(all, x1, q), y2 = __shfl_xor_sync(all, x2, q);
                x2 = fmaxf(fmaxf(x2, y2), fminf(x1, y1));
                x1 = fmaxf(x1, y1);
            }
            float v = p.group_top > 1 ? (x2 > ninf ? x1 + x2 : ninf) : x1;
            v = __shfl_sync(all, v, (lane * lp) & 31);
            int r = 0;
            for (int h0 = 0; h0 < p.groups; h0 += 8) {
#pragma unroll
                for (int h = 0; h < 8; ++h) {
                    const float x = __shfl_sync(all, v, (h0 + h) & 31);
                    r += h0 + h < p.groups && (x > v || (x == v && h0 + h < lane)) ? 1 : 0;
                }
            }
            const bool is = lane < p.groups;
            const uint32_t keep = __ballot_sync(all, is && r < p.kept);
            if (BIAS || scores) {
                // the last group kept and the first one dropped must differ by more than their errors
                amax = __uint_as_float(__reduce_max_sync(all, __float_as_uint(amax)));  // not negative: in the order of its bits
                const float vk = __shfl_sync(all, v, __ffs(__ballot_sync(all, is && r == p.kept - 1)) - 1);
                const float vd = __shfl_sync(all, v, __ffs(__ballot_sync(all, is && r == p.kept)) - 1);
                const float geps = p.group_top * (fine + 0x1p-22f * amax);
                if (vk > ninf && vd > ninf && !(vk - vd > 2.f * geps)) unsettled = true;
                if (amax == INFINITY) unsettled = true;
            }
#pragma unroll
            for (int i = 0; i < N; ++i) {
                const uint32_t e = 128 * (i / 4) + 4 * lane + i % 4;
                if (!((keep >> ((e * p.gmul) >> 20 & 31)) & 1u)) o[i] = ninf;
            }
        }
        if (BIAS || p.groups > 1) {
            lm = ninf;
#pragma unroll
            for (int i = 0; i < N; ++i) lm = fmaxf(lm, o[i]);
            __syncwarp();
        }
#pragma unroll
        for (int i = 0; i < NI; ++i)
            *reinterpret_cast<float4 *>(val + 128 * i + 4 * lane) = make_float4(o[4 * i], o[4 * i + 1], o[4 * i + 2], o[4 * i + 3]);
        // The k-th largest lane maximum, from below: the keys leave out the
        // last 5 bits, which tell the lanes apart.
        const uint32_t mine_key = (order_bits(lm) & ~31u) | (31u - lane);
        s.top[lane] = mine_key;
        __syncwarp();
        int r = 0;
#pragma unroll
        for (int j = 0; j < 32; j += 4) {
            const uint4 v = *reinterpret_cast<const uint4 *>(&s.top[j]);
            r += (v.x > mine_key) + (v.y > mine_key) + (v.z > mine_key) + (v.w > mine_key);
        }
        const int at = __ffs(__ballot_sync(all, r == p.k - 1)) - 1;
        const float low = __shfl_sync(all, lm, at);
        const float top = __shfl_sync(all, lm, __ffs(__ballot_sync(all, r == 0)) - 1);
        float th = low > ninf ? from_order_bits(order_bits(low) & ~31u) : ninf;
        float eps = 0.f;
        if (BIAS && top > ninf) {
            // values of larger size than both are far below the threshold
            const float size = 0x1p-22f * fmaxf(fabsf(top), low > ninf ? fabsf(low) : 0.f);
            eps = fine + size;
            th -= 2.f * ((coarse ? 0x1p-10f : fine) + size);
            if (!(eps < 0x1p100f)) unsettled = true;  // infinite biases
        }
        th = fmaxf(th, -3.402823466e38f);  // -inf is out
        uint32_t mask = 0u;
#pragma unroll
        for (int i = 0; i < N; ++i) mask |= o[i] >= th ? 1u << i : 0u;
        const int cnt = __popc(mask);
        int pos = cnt;
#pragma unroll
        for (int q = 1; q < 32; q <<= 1) {
            const int v = __shfl_up_sync(all, pos, q);
            if (lane >= q) pos += v;
        }
        const int C = __shfl_sync(all, pos, 31);
        pos -= cnt;
        if (C > kGateCap) unsettled = true;
        if (!unsettled) {  // alike in all lanes
            while (mask) {
                const int i = __ffs(mask) - 1;
                mask &= mask - 1u;
                const int e = 128 * (i >> 2) + 4 * lane + (i & 3);
                s.key[pos++] = (uint64_t)order_bits(val[e] + 0.f) << 32 | (uint32_t)~e;  // -0 ranks as 0
            }
            if (lane < 8 && C + lane < ((C + 7) & ~7)) s.key[C + lane] = 0ull;  // up to a multiple of 8: below every key
            __syncwarp();
            if (coarse) {
                for (int c = lane; c < C; c += 32) {
                    const uint32_t inv_id = (uint32_t)s.key[c];
                    const float v = rough(gate_logit(p, t, (int)~inv_id)) + p.bias[(int)~inv_id];
                    s.key[c] = (uint64_t)order_bits(v + 0.f) << 32 | inv_id;
                }
                __syncwarp();
            }
            for (int c = lane; c < C; c += 32) {
                const uint64_t key = s.key[c];
                int place = 0;
                for (int j = 0; j < C; j += 8) {
#pragma unroll
                    for (int i = 0; i < 8; i += 2) {
                        const ulonglong2 x = *reinterpret_cast<const ulonglong2 *>(&s.key[j + i]);
                        place += (x.x > key ? 1 : 0) + (x.y > key ? 1 : 0);
                    }
                }
                if (place <= p.k) {
                    s.sorted[place] = from_order_bits((uint32_t)(key >> 32));
                    s.id[place] = (int32_t)~(uint32_t)key;
                }
            }
            __syncwarp();
            const int got = min(C, p.k);
            if (BIAS) {
                const float v0 = s.sorted[min(lane, got)], v1 = s.sorted[min(lane + 1, p.k)];
                const bool close = lane < got && lane + 1 < C && !(v0 - v1 > 2.f * (eps + 0x1p-22f * fmaxf(fabsf(v0), fabsf(v1))));
                if (__any_sync(all, close)) {
                    double sum64 = 0.0;
                    if (!p.sigmoid) {
                        // in gate_exact's order: ids lane, lane + 32, ...
                        for (int e = lane; e < p.E; e += 32) {
                            const float v = gate_logit(p, t, e);
                            if (v > ninf) sum64 += exp((double)v - (double)mx);
                        }
                        sum64 = warp_sum(sum64);
                    }
                    for (int c = lane; c < C; c += 32) {
                        const int e = (int32_t)~(uint32_t)s.key[c];
                        const double v = gate_logit(p, t, e);
                        s.exact[c] = (p.sigmoid ? 1.0 / (1.0 + exp(-v)) : exp(v - (double)mx) / sum64) + (double)p.bias[e];
                    }
                    __syncwarp();
                    for (int c = lane; c < C; c += 32) {
                        const double v = s.exact[c];
                        const uint32_t inv_id = (uint32_t)s.key[c];  // larger: lower id
                        int place = 0;
                        for (int j = 0; j < C; ++j)
                            place += s.exact[j] > v || (s.exact[j] == v && (uint32_t)s.key[j] > inv_id) ? 1 : 0;
                        if (place < p.k) s.id[place] = (int32_t)~inv_id;
                    }
                    __syncwarp();
                }
            }
            int mine = -1;
            float w = 0.f;
            if (lane < got) {
                mine = s.id[lane];
                const float v = BIAS ? gate_logit(p, t, mine) : s.sorted[lane];
                if (p.sigmoid) {
                    w = 1.0f / (1.0f + expf(-v));
                } else {
                    const float d = v - mx, y = d - v, x = (v - (d - y)) - (mx + y);  // d + x = v - mx exactly
                    w = d < -100.f ? 0.f : expf(d) * (1.0f + x) / sum;
                }
            }
            if (__any_sync(all, mine >= 0 && w < 0x1p-100f)) {
                unsettled = true;
            } else {
                float z = w;
                for (int q = 16; q > 0; q >>= 1) z += __shfl_xor_sync(all, z, q);
                if (lane < p.k) {
                    p.idx[t * p.k + lane] = mine;
                    p.weight[t * p.k + lane] = (p.renorm ? (z == 0.f ? 0.f : w / z) : w) * p.scale;
                }
            }
        }
    }
    if (__syncthreads_or(unsettled)) {
        GateExact &slow = *reinterpret_cast<GateExact *>(gate_raw);  // over the warps' parts, which are done with
        for (int w = 0; w < kGateWarps; ++w) {
            if (w == warp && unsettled) gate_exact(p, t, slow);
            __syncthreads();
        }
    }
}

}  // namespace k3
