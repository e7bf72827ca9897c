// Dense product of bf16 activations and weights with bias, activation, gate
// and residual in its epilogue (k3moe_linear).
#pragma once

#include "common.cuh"
#include "layout.cuh"
#include "umma.cuh"

namespace k3 {

struct LinearParams {
    const uint16_t *x;         // bf16, T rows, ldx elements apart
    const uint16_t *w, *wg;    // bf16, N rows, ldw elements apart (wg: null, or the gate's)
    const float *bias, *bias_g;
    const void *resid;         // T rows, ldr elements apart, or null
    void *out;                 // T rows, ldo elements apart
    long long ldx, ldw, ldr, ldo;
    int T, N, K, act, out_fp32;
    int vec;                   // out's and resid's rows are 16-byte aligned
};

// The activation of NV values.  One branch for all of them: a switch inside
// the unrolled loops of the epilogues made code of some 100 KB, and fetching
// it took longer than the product (down projection of 4095 tokens: 326 us).
template <int NV>
__device__ __forceinline__ void linear_act(float (&v)[NV], int act) {
    if (act == K3MOE_ACT_RELU) {
#pragma unroll
        for (int i = 0; i < NV; ++i) v[i] = v[i] < 0.f ? 0.f : v[i];  // NaN stays NaN
    } else if (act == K3MOE_ACT_SILU) {
#pragma unroll
        for (int i = 0; i < NV; ++i) v[i] = __fdividef(v[i], 1.0f + __expf(-v[i]));  // within 4 units in the last place + |v| 2^-24
    } else if (act == K3MOE_ACT_GELU) {
#pragma unroll
        for (int i = 0; i < NV; ++i) v[i] = 0.5f * v[i] * erfcf(-0.70710678118654752f * v[i]);
    } else if (act == K3MOE_ACT_GELU_TANH) {
#pragma unroll
        for (int i = 0; i < NV; ++i)
            v[i] = __fdividef(v[i], 1.0f + __expf(-1.5957691216057308f * (v[i] + 0.044715f * v[i] * v[i] * v[i])));  // (1 + tanh u) / 2
    }
}

__device__ __forceinline__ uint16_t bf16_bits(float v) { return __bfloat16_as_ushort(__float2bfloat16_rn(v)); }

// A thread finishes NV outputs: element i is column n + i dn of token t + i dt.
// Where the rows of the output and the residual are 16-byte aligned, NV
// neighbouring columns of one token (dn = 1), in one access of 8 or 16 bytes
// (bf16, NV = 4 or 8); elsewhere the lanes of a warp have neighbouring columns
// and a thread walks over others.  (2-byte accesses to aligned rows: the down
// projection of 4095 tokens took 114 us; NV neighbouring columns of unaligned
// ones: 1245 tokens of 2553 columns 33 us.)
struct LinearWalk {
    int dt, dn;
    long long tend;  // tokens up to here
};
template <int NV>
struct Residual {
    uint32_t w[NV];  // fp32 bits, or NV bf16 in the first half
};

// Loads only: nothing here waits for them.  (t, n) exists; elements that do
// not are read as the last ones.
template <int NV>
__device__ __forceinline__ void linear_resid(const LinearParams &p, long long t, int n, Residual<NV> &r, bool out_fp32,
                                             const LinearWalk &k) {
    if (!p.resid) return;
    const bool wide = p.vec && k.dn == 1 && n + NV <= p.N;
    auto at = [&](int i) { return min(t + i * k.dt, k.tend - 1) * p.ldr + min(n + i * k.dn, p.N - 1); };
    if (out_fp32) {
        const float *q = reinterpret_cast<const float *>(p.resid);
        if (NV % 4 == 0 && wide) {
#pragma unroll
            for (int i = 0; i < NV; i += 4) {
                const uint4 v = *reinterpret_cast<const uint4 *>(q + t * p.ldr + n + i);
                r.w[i] = v.x, r.w[i + 1] = v.y, r.w[i + 2] = v.z, r.w[i + 3] = v.w;
            }
        } else {
#pragma unroll
            for (int i = 0; i < NV; ++i) r.w[i] = __float_as_uint(q[at(i)]);
        }
    } else {
        const uint16_t *q = reinterpret_cast<const uint16_t *>(p.resid);
        if (NV == 8 && wide) {
            const uint4 v = *reinterpret_cast<const uint4 *>(q + t * p.ldr + n);
            r.w[0] = v.x, r.w[1 % NV] = v.y, r.w[2 % NV] = v.z, r.w[3 % NV] = v.w;
        } else if (NV == 4 && wide) {
            const uint2 v = *reinterpret_cast<const uint2 *>(q + t * p.ldr + n);
            r.w[0] = v.x, r.w[1 % NV] = v.y;
        } else {
            uint16_t h[NV];
#pragma unroll
            for (int i = 0; i < NV; ++i) h[i] = q[at(i)];
#pragma unroll
            for (int i = 0; i < NV; i += 2) r.w[i / 2] = h[i] | (uint32_t)(NV > 1 ? h[(i + 1) % NV] : 0) << 16;
        }
    }
}

// v, g: the sums; b, bg: the columns' biases.  Bias, activation, gate and
// residual in fp32, one rounding.
template <int NV>
__device__ __forceinline__ void linear_finish(const LinearParams &p, long long t, int n, float (&v)[NV], float (&g)[NV],
                                              const float (&b)[NV], const float (&bg)[NV], const Residual<NV> &r,
                                              bool gated, bool resid, bool out_fp32, const LinearWalk &k) {
    const bool wide = p.vec && k.dn == 1 && n + NV <= p.N;
#pragma unroll
    for (int i = 0; i < NV; ++i) v[i] += b[i];
    if (gated) {
#pragma unroll
        for (int i = 0; i < NV; ++i) g[i] += bg[i];
        linear_act(g, p.act);
#pragma unroll
        for (int i = 0; i < NV; ++i) v[i] *= g[i];
    } else {
        linear_act(v, p.act);
    }
    if (resid) {
        if (out_fp32) {
#pragma unroll
            for (int i = 0; i < NV; ++i) v[i] += __uint_as_float(r.w[i]);
        } else {
#pragma unroll
            for (int i = 0; i < NV; ++i) v[i] += i % 2 ? bf16_hi(r.w[i / 2]) : bf16_lo(r.w[i / 2]);
        }
    }
    if (out_fp32) {
        float *q = reinterpret_cast<float *>(p.out) + t * p.ldo + n;
        if (NV % 4 == 0 && wide) {
#pragma unroll
            for (int i = 0; i < NV; i += 4)
                *reinterpret_cast<float4 *>(q + i) = make_float4(v[i], v[(i + 1) % NV], v[(i + 2) % NV], v[(i + 3) % NV]);
        } else {
#pragma unroll
            for (int i = 0; i < NV; ++i)
                if (t + i * k.dt < k.tend && n + i * k.dn < p.N) q[(long long)(i * k.dt) * p.ldo + i * k.dn] = v[i];
        }
    } else {
        uint16_t *q = reinterpret_cast<uint16_t *>(p.out) + t * p.ldo + n;
        uint16_t h[NV];
#pragma unroll
        for (int i = 0; i < NV; ++i) h[i] = bf16_bits(v[i]);
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) w[i] = h[2 * i % NV] | (uint32_t)h[(2 * i + 1) % NV] << 16;
        if (NV == 8 && wide) {
            *reinterpret_cast<uint4 *>(q) = make_uint4(w[0], w[1], w[2], w[3]);
        } else if (NV == 4 && wide) {
            *reinterpret_cast<uint2 *>(q) = make_uint2(w[0], w[1]);
        } else {
#pragma unroll
            for (int i = 0; i < NV; ++i)
                if (t + i * k.dt < k.tend && n + i * k.dn < p.N) q[(long long)(i * k.dt) * p.ldo + i * k.dn] = h[i];
        }
    }
}

template <int NV>
__device__ __forceinline__ void linear_bias(const float *bias, int n, int dn, int N, float (&b)[NV]) {
#pragma unroll
    for (int i = 0; i < NV; ++i) b[i] = bias && n < N ? __ldg(bias + min(n + i * dn, N - 1)) : 0.f;
}

// ------------------------------------------------------ few tokens: stream --
// Up to 16 tokens: the weights are read once from memory and little else
// counts.  TMA brings a chunk of kc columns of the CTA's weight rows and of the
// tokens into a ring of stages of each warp (chunk c belongs to warp c %
// warps; zeros past the last row and column); the warp multiplies it
// with warp-level MMAs (m16n8k16: A = 16 tokens, B = 8 weight rows), whose few
// cycles do not show, so a tensor-memory round trip would only add to the
// latency.  A lane's 16 bytes hold 8 consecutive k of one row; the same k
// order is used for weights and tokens, so the order of k inside a step is
// free and two MMAs take them as they are.  (Loads straight into the operand
// registers, 8 lines each: one token's 896 x 7168 took 4.4 us to arrive; bulk
// copies of 512-byte rows: 4.7 us; this: 3.3 us.)  Bound by memory where K and n
// are large (7168 x 7168: 19 us, 5.4 TB/s), by latency below (4 tokens, 680 x
// 680: 2.1 us in a captured graph).
constexpr int kLsMaxT = 16;
constexpr int kLsWarps = 8;
constexpr int kLsMaxStages = 4;

struct LinearStreamParams {
    alignas(64) uint4 tw[8];
    alignas(64) uint4 twg[8];
    alignas(64) uint4 tx[8];
    LinearParams p;
    int kc, ns;  // columns per chunk (a multiple of 64), stages per warp
    WsHeader *hdr;
    uint64_t wait_ns;
};

__device__ __forceinline__ void mma_16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                          uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// NM groups of 8 weight rows (gated: all of w's, then w_gate's), TG 8-token halves.
__host__ __device__ constexpr int ls_red_bytes(int nm, int tg) { return kLsWarps * nm * tg * 64 * 4; }
__host__ __device__ constexpr int ls_stage_bytes(int nm, int tg, int kc) { return (nm + tg) * 8 * kc * 2; }
__host__ __device__ constexpr int ls_smem_bytes(int nm, int tg, int kc, int ns) {
    return 1024 + 2 * ls_red_bytes(nm, tg) + kLsWarps * ns * ls_stage_bytes(nm, tg, kc);
}

// RG: groups of 8 output columns per CTA.
// INJECT: failure-path tests, one warp makes no copies (a kernel of its own: a
// parameter for it cost 0.05 to 0.2 us at the start).
template <int RG, bool GATED, int TG, bool INJECT = false>
__global__ void __launch_bounds__(32 * kLsWarps) linear_stream_kernel(const __grid_constant__ LinearStreamParams a) {
    constexpr int NM = RG * (GATED ? 2 : 1), TT = 8 * TG;
    extern __shared__ __align__(128) uint8_t ls_raw[];
    uint64_t *bars = reinterpret_cast<uint64_t *>(ls_raw);  // [warp][stage]
    volatile int *s_abort = reinterpret_cast<volatile int *>(ls_raw + 512);
    float *red = reinterpret_cast<float *>(ls_raw + 1024);  // [2][warp][NM][TT tokens][8 rows]
    const LinearParams &p = a.p;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int g = lane >> 2, q = lane & 3;
    const int T = p.T, rowb = a.kc * 2, stageb = (NM + TG) * 8 * rowb;
    uint8_t *ring = ls_raw + 1024 + 2 * ls_red_bytes(NM, TG) + warp * a.ns * stageb;
    uint64_t *bar = bars + warp * kLsMaxStages;
    if (lane == 0) {
        for (int s = 0; s < a.ns; ++s) mbar_init(&bar[s], 1);
        fence_mbar_init();
        if (warp == 0) {
            *s_abort = 0;
            umma::prefetch_tmap(a.tw);
            if (GATED) umma::prefetch_tmap(a.twg);
            umma::prefetch_tmap(a.tx);
        }
    }
    __syncthreads();
    pdl_wait();
    pdl_trigger();
    const int chunks = ceil_div(p.K, a.kc), groups = ceil_div(p.N, RG * 8);
    // The warp's next chunk to copy: it runs on into the CTA's next groups of
    // columns while the sums of one are brought together.
    int ig = warp < chunks && !(INJECT && warp == 0) ? blockIdx.x : groups, ic = warp, issued = 0;
    auto issue = [&](int s) {
        if (ig >= groups) return;
        if (umma::elect()) {
            uint8_t *st = ring + s * stageb;
            mbar_arrive_expect_tx(&bar[s], (uint32_t)((NM * 8 + T) * rowb));  // the other token rows stay as they are
            umma::tma_load_2d(st, a.tw, ic * a.kc, ig * RG * 8, &bar[s]);
            if (GATED) umma::tma_load_2d(st + RG * 8 * rowb, a.twg, ic * a.kc, ig * RG * 8, &bar[s]);
            umma::tma_load_2d(st + NM * 8 * rowb, a.tx, ic * a.kc, 0, &bar[s]);
        }
        __syncwarp();
        ++issued;
        if ((ic += kLsWarps) >= chunks) {
            ic = warp;
            ig += gridDim.x;
        }
    };
    for (int s = 0; s < a.ns; ++s) issue(s);
    const bool odd = (g & 1) != 0;
    // 64 columns of row r of a stage, columns 8 q.. of the first and of the
    // second 32; odd rows read them in the other order (no bank conflicts)
    auto row64 = [&](const uint8_t *row, uint4 (&v)[2]) {
        const uint4 x = *reinterpret_cast<const uint4 *>(row + (odd ? 64 : 0));
        const uint4 y = *reinterpret_cast<const uint4 *>(row + (odd ? 0 : 64));
        v[0] = odd ? y : x;
        v[1] = odd ? x : y;
    };
    const int rg = threadIdx.x / (TT * 8), ot = (threadIdx.x / 8) % TT;  // this thread's output of a group
    int s = 0, par = 0;
    uint32_t ph = 0u;
    bool ok = true;
    for (int grp = blockIdx.x; grp < groups; grp += gridDim.x, par ^= 1) {
        const int on = grp * RG * 8 + rg * 8 + threadIdx.x % 8;
        const bool out = rg < RG && ot < T && on < p.N;
        float b[1], bg[1];
        Residual<1> res;
        if (out) {
            linear_bias(p.bias, on, 0, p.N, b);
            linear_bias(p.bias_g, on, 0, p.N, bg);
            linear_resid(p, ot, on, res, p.out_fp32, LinearWalk{0, 0, T});
        }
        __syncwarp();
        float sum[NM][4] = {};
        for (int c = warp; c < chunks; c += kLsWarps) {
            ok = ok && mbar_wait_warp(&bar[s], ph, a.hdr, a.wait_ns, s_abort);
            if (!ok) break;
            const uint8_t *st = ring + s * stageb + g * rowb + q * 16;
            float part[NM][4] = {};  // a chain per chunk; the chunks are added in fp32
#pragma unroll 2
            for (int k = 0; k < rowb; k += 128) {
                uint4 x[TG][2];
#pragma unroll
                for (int t = 0; t < TG; ++t) row64(st + (NM + t) * 8 * rowb + k, x[t]);
#pragma unroll
                for (int m = 0; m < NM; ++m) {
                    uint4 w[2];
                    row64(st + m * 8 * rowb + k, w);
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const uint4 &xa = x[0][h], &xb = x[TG - 1][h];
                        mma_16816(part[m], xa.x, TG == 2 ? xb.x : 0u, xa.y, TG == 2 ? xb.y : 0u, w[h].x, w[h].y);
                        mma_16816(part[m], xa.z, TG == 2 ? xb.z : 0u, xa.w, TG == 2 ? xb.w : 0u, w[h].z, w[h].w);
                    }
                }
            }
#pragma unroll
            for (int m = 0; m < NM; ++m)
#pragma unroll
                for (int e = 0; e < 4; ++e) sum[m][e] += part[m][e];
            __syncwarp();
            issue(s);
            if (++s == a.ns) {
                s = 0;
                ph ^= 1u;
            }
        }
        __syncwarp();
        float *rbuf = red + par * (ls_red_bytes(NM, TG) / 4);
#pragma unroll
        for (int m = 0; m < NM; ++m) {
            float *o = rbuf + (warp * NM + m) * TT * 8 + g * 8 + 2 * q;  // token g, rows 2q and 2q + 1
            *reinterpret_cast<float2 *>(o) = make_float2(sum[m][0], sum[m][1]);
            if (TG == 2) *reinterpret_cast<float2 *>(o + 64) = make_float2(sum[m][2], sum[m][3]);
        }
        __syncthreads();
        if (out) {
            float v[1] = {0.f}, gv[1] = {0.f};
            const float *src = rbuf + rg * TT * 8 + threadIdx.x % (TT * 8);
#pragma unroll
            for (int w = 0; w < kLsWarps; ++w) {
                v[0] += src[w * NM * TT * 8];
                if (GATED) gv[0] += src[(w * NM + RG) * TT * 8];
            }
            linear_finish(p, ot, on, v, gv, b, bg, res, GATED, p.resid != nullptr, p.out_fp32, LinearWalk{0, 0, T});
        }
        __syncwarp();
    }
    // a warp that gave up waits (bounded) for its own copies in flight
    if (!ok && lane == 0) {
        const uint64_t t0 = globaltimer();
        for (int i = 0; i < a.ns && i < issued; ++i) mbar_drain(&bar[i], (uint32_t)(((issued - 1 - i) / a.ns) & 1), t0);
    }
}

// -------------------------------------------------------- tcgen05 kernels --
// The weights are the MMA's M side (accumulator lane = output column), the
// tokens its N side, so that a warp stores 32 neighbouring columns of one
// token at once, whatever the rows' alignment, and a column's bias is one
// register.  A gated product stacks 64 rows of w and 64 of w_gate into the 128
// rows; the two are brought together through shared memory in the epilogue.
constexpr int kLtEpi = 16;                     // epilogue warps: four per lane quadrant
constexpr int kLtThreads = 32 * (kLtEpi + 2);  // and one that copies, one that issues MMAs
constexpr int kLtKStep = 64;     // bf16 per K-step: 128 bytes of every row, one swizzle atom
constexpr int kLtA = 128 * 128;  // bytes of the weight box per stage
constexpr int kLtHead = 1024;    // barriers, before the stages
constexpr int kLtMaxStages = 10;
constexpr int kLtMaxSplit = 8;
constexpr int kLtChain = 8;        // K-steps per accumulation chain of an fp32 output
constexpr int kLtChainBf16 = 256;  // and of a bf16 one; in the pair kernel that is one chain,
constexpr int kLpMaxSteps = 512;   // of K up to this many steps
constexpr int kLinearMaxT = 1 << 30;

struct LinearTcParams {
    alignas(64) uint4 tw[8];
    alignas(64) uint4 twg[8];
    alignas(64) uint4 tx[8];
    alignas(64) uint4 tx_part[8];  // pair kernel: boxes of the last wave's parts
    LinearParams p;
    int bn;          // tokens per tile (pair kernel: of the pair)
    int whole, parts;  // pair kernel: tiles run whole (the first ones); parts of bn / parts tokens of each other tile
    int nst;         // pipeline stages; from bit 8: failure-path tests, last K-steps that one CTA does not copy
                     // (with a parameter of its own 333 x 1001 x 1000 took 8.30 us, so 8.19)
    int nrb, ntt;    // row blocks, token tiles
    int split;       // tile kernel: CTAs (one cluster) that share a tile's K
    int chain;       // K-steps accumulated in tensor memory at a stretch (pair kernel: of an fp32 output)
    int tcols;       // tensor-memory columns
    int part, red;   // tile kernel: offsets of its own sums and of the other CTAs' parts
    WsHeader *hdr;
    uint64_t wait_ns;
};

// A tile of 128 weight rows x bn tokens per cluster of `split` CTAs, which
// share its K: each accumulates its part, sends every CTA of the cluster the
// columns that CTA finishes (one bulk copy each over distributed shared
// memory; stores of single values took 1.8 us for 112 columns), and finishes
// its own columns, adding the parts in rank order.  Bound by memory and the way
// in (64 bytes a clock per SM): gated 100 tokens x 1536 x 7168, K in five, 14.1 us
// for 44 MB, of which the stream takes 8.8, the exchange 1.5, the ends the rest.
//
// The tensor core cuts its running sum at every step, so a long chain drifts:
// with fp32 outputs the sum moves to shared memory (tiles of more than 128
// tokens: registers) every `chain` K-steps (two tensor-memory buffers) and the
// pieces are added there, rounded to nearest.
// A step of 16 cuts up to 2^-23 of it, towards zero.  Measured against 64 bits:
// chains of 8 K-steps 0.9e-6 of a sum of equal signs and 0.5e-6 (rms) of the
// outputs' size at random signs, whatever K; one chain of 7168 columns 2.8e-5
// and 0.8e-5, of 32768 1.8e-4 and 3.8e-5.  A bf16 output's half step is 2e-3 to
// 4e-3 of it, so it takes chains of up to kLtChainBf16 K-steps here (16384
// columns; K in S parts is in S chains), of kLpMaxSteps in the pair kernel
// (32768).
template <bool GATED, bool RESID, bool OUT32>
__global__ void __launch_bounds__(kLtThreads, 1) linear_tile_kernel(const __grid_constant__ LinearTcParams a) {
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
    const LinearParams &p = a.p;
    const int nst = a.nst & 255, bn = a.bn, S = a.split;
    const int SB = kLtA + bn * 128;
    uint64_t *full = reinterpret_cast<uint64_t *>(smem);
    uint64_t *empty = full + nst;
    uint64_t *afull = empty + nst;
    uint64_t *aempty = afull + 2;
    uint64_t *mdone = aempty + 2;
    uint64_t *rfull = mdone + 1;  // the other CTAs' parts of this CTA's columns have arrived
    uint32_t *tslot = reinterpret_cast<uint32_t *>(rfull + 1);
    volatile int *s_abort = reinterpret_cast<volatile int *>(tslot + 1);
    volatile int *s_issued = s_abort + 1;  // stages filled, once all are; -1 before
    uint8_t *stages = smem + kLtHead;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        for (int s = 0; s < nst; ++s) {
            mbar_init(&full[s], 1);
            mbar_init(&empty[s], 1);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(&afull[b], 1);
            mbar_init(&aempty[b], kLtEpi);
        }
        mbar_init(mdone, 1);
        mbar_init(rfull, 1);
        fence_mbar_init();
        *s_abort = 0;
        *s_issued = -1;
    }
    if (warp == kLtEpi && lane == 0) {
        umma::prefetch_tmap(a.tw);
        umma::prefetch_tmap(a.tx);
    }
    if (warp == 0) umma::tmem_alloc(tslot, (uint32_t)a.tcols);
    umma::fence_before();
    __syncthreads();
    if (S > 1) {  // the barriers of every CTA of the cluster are set up
        umma::cluster_arrive();
        umma::cluster_wait();
    }
    umma::fence_after();
    const uint32_t tbase = *tslot;
    const int rank = S > 1 ? (int)umma::cluster_rank() : 0;
    const int tile = blockIdx.x / S;
    const int nrow = GATED ? 64 : 128;
    const int n0 = (tile % a.nrb) * nrow, t0 = (tile / a.nrb) * bn;
    const int nkt = ceil_div(p.K, kLtKStep);
    const int kt0 = (int)((long long)nkt * rank / S), nk = (int)((long long)nkt * (rank + 1) / S) - kt0;
    const int fill = rank == 0 ? nk - (a.nst >> 8) : nk;  // K-steps copied
    const int nch = ceil_div(nk, a.chain);
    const int cpo = ceil_div(bn, S);  // columns that one CTA of the cluster finishes
    auto wait = [&](uint64_t *bar, uint32_t parity) { return mbar_wait_warp(bar, parity, a.hdr, a.wait_ns, s_abort); };
    pdl_wait();
    pdl_trigger();

    // part[column][row]: this CTA's sums (of the chains so far); red[source][
    // column][row]: the other CTAs' parts of the columns this CTA finishes.
    float *part = reinterpret_cast<float *>(smem + a.part);
    float *red = reinterpret_cast<float *>(smem + a.red);
    const int cend = min(bn, p.T - t0);                     // columns that exist
    const int jmax = max(0, min(cpo, cend - rank * cpo));   // of them, finished here
    if (S > 1 && threadIdx.x == 0 && jmax > 0) mbar_arrive_expect_tx(rfull, (uint32_t)((S - 1) * jmax * 512));
    if (warp == kLtEpi) {
        int i = 0, s = 0;
        uint32_t ph = 1u;  // of the empty barriers: the first round's waits pass at once
        for (; i < fill; ++i) {
            if (!wait(&empty[s], ph)) break;
            if (umma::elect()) {
                uint8_t *st = stages + s * SB;
                const int x = (kt0 + i) * kLtKStep;
                mbar_arrive_expect_tx(&full[s], (uint32_t)SB);
                umma::tma_load_2d(st, a.tw, x, n0, &full[s]);
                if (GATED) umma::tma_load_2d(st + kLtA / 2, a.twg, x, n0, &full[s]);
                umma::tma_load_2d(st + kLtA, a.tx, x, t0, &full[s]);
            }
            __syncwarp();
            if (++s == nst) {
                s = 0;
                ph ^= 1u;
            }
        }
        if (lane == 0) *s_issued = i;
    } else if (warp == kLtEpi + 1) {
        const uint64_t adesc = umma::smem_desc(smem_u32(stages), 16u, 1024u, umma::kLayoutSw128);
        const uint32_t idesc = umma::idesc_bf16(bn);
        int i = 0, s = 0;
        uint32_t ph = 0u;
        bool ok = true;
        for (int c = 0; c < nch && ok; ++c) {
            const int buf = c & 1;
            if (c >= 2 && !wait(&aempty[buf], (uint32_t)(((c >> 1) + 1) & 1))) break;
            const uint32_t d = tbase + (uint32_t)(buf * bn);
            const int i0 = i, i1 = min(nk, i + a.chain);
            for (; i < i1; ++i) {
                if (!wait(&full[s], ph)) {
                    ok = false;
                    break;
                }
                umma::fence_after();
                const uint64_t ad = adesc + ((uint32_t)(s * SB) >> 4), bd = ad + (kLtA >> 4);
                const int steps = ceil_div(p.K - (kt0 + i) * kLtKStep, 16);  // past K: zeros from TMA
                if (umma::elect()) {
                    umma::mma_bf16(d, ad, bd, idesc, i > i0 ? 1u : 0u);
                    if (steps > 1) umma::mma_bf16(d, ad + 2, bd + 2, idesc, 1u);
                    if (steps > 2) umma::mma_bf16(d, ad + 4, bd + 4, idesc, 1u);
                    if (steps > 3) umma::mma_bf16(d, ad + 6, bd + 6, idesc, 1u);
                    umma::commit(&empty[s]);
                    if (i + 1 == i1) umma::commit(&afull[buf]);
                }
                __syncwarp();
                if (++s == nst) {
                    s = 0;
                    ph ^= 1u;
                }
            }
        }
        if (umma::elect()) {
            umma::commit(mdone);
            mbar_drain(mdone, 0u, globaltimer());
            if (*s_abort) drain_ring(full, nst, s_issued);
        }
    } else {
        // A thread finishes 4 columns of the tokens j0, j0 + step, ... of its
        // CTA's (a warp's lanes: one token, or two of a gated product); the
        // biases and the first residual are loaded while the MMAs run.
        constexpr int lpt = GATED ? 16 : 32, step = kLtEpi * 32 / lpt;
        const LinearWalk walk{0, p.vec ? 1 : lpt, p.T};
        const int n = n0 + lane % lpt * (p.vec ? 4 : 1), j0 = threadIdx.x / lpt;
        const long long tq = (long long)t0 + rank * cpo;
        float b[4], bg[4];
        Residual<4> res;
        linear_bias(p.bias, n, walk.dn, p.N, b);
        linear_bias(p.bias_g, n, walk.dn, p.N, bg);
        if (RESID && n < p.N && j0 < jmax) linear_resid(p, tq + j0, n, res, OUT32, walk);
        __syncwarp();
        const uint32_t src0 = tbase + umma::lane_base(warp);
        float *dst = part + 32 * (warp & 3) + lane;
        auto release = [&](int buf) {
            umma::fence_before();
            __syncwarp();
            if (lane == 0)
                asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_u32(&aempty[buf])) : "memory");
            __syncwarp();
        };
        if (OUT32 && bn > 128) {
            // No room for the chains' sums in shared memory: a warp's rows and
            // its columns 16 (warp / 4) + 64 i + 0..15 in registers, over the
            // stages at the end.  (4096 x 896 x 7168 in 49 us, 88 in tiles of
            // 128 tokens.  Smaller tiles in this form took 0.4 us more to
            // fetch its code: 64 x 896 x 7168 9.0 us, 8.8.)
            float acc[4][16];
            bool ok = true;
            for (int c = 0; c < nch; ++c) {
                const int buf = c & 1;
                ok = wait(&afull[buf], (uint32_t)((c >> 1) & 1));
                if (!ok) break;
                umma::fence_after();
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int j = 16 * (warp >> 2) + 64 * i;
                    if (j < cend) {
                        uint32_t r[16];
                        umma::ld16(src0 + (uint32_t)(buf * bn + j), r);
                        umma::wait_ld();
#pragma unroll
                        for (int q = 0; q < 16; ++q)
                            acc[i][q] = c == 0 ? __uint_as_float(r[q]) : acc[i][q] + __uint_as_float(r[q]);
                    }
                }
                release(buf);
            }
            if (ok) {  // the MMAs have read every stage: the sums may lie over them
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int j = 16 * (warp >> 2) + 64 * i;
                    if (j < cend)
#pragma unroll
                        for (int q = 0; q < 16; ++q) dst[(j + q) * 128] = acc[i][q];
                }
            }
            __syncwarp();
        } else {
            for (int c = 0; c < nch; ++c) {
                const int buf = c & 1;
                if (!wait(&afull[buf], (uint32_t)((c >> 1) & 1))) break;
                umma::fence_after();
                for (int j = 16 * (warp >> 2); j < cend; j += 4 * kLtEpi) {
                    uint32_t r[16];
                    umma::ld16(src0 + (uint32_t)(buf * bn + j), r);
                    umma::wait_ld();
                    float *d = dst + j * 128;
                    if (c == 0) {
#pragma unroll
                        for (int i = 0; i < 16; ++i) d[i * 128] = __uint_as_float(r[i]);
                    } else {
#pragma unroll
                        for (int i = 0; i < 16; ++i) d[i * 128] += __uint_as_float(r[i]);
                    }
                }
                release(buf);
            }
        }
        if (S > 1) fence_proxy_async();  // the copies below read what was stored here
        umma::bar_sync(1, 32 * kLtEpi);
        if (S > 1) {
            if (threadIdx.x < S && threadIdx.x != rank) {
                const int cols = min(cpo, cend - (int)threadIdx.x * cpo);
                if (cols > 0)
                    umma::bulk_s2s(umma::mapa(smem_u32(red) + (uint32_t)(rank * cpo) * 512u, threadIdx.x),
                                   part + threadIdx.x * cpo * 128, (uint32_t)cols * 512u,
                                   umma::mapa(smem_u32(rfull), threadIdx.x));
            }
            __syncwarp();
            // Every CTA sends, one that gave up too: what is sent here lands
            // before this CTA leaves (the cluster barrier orders the sending,
            // not the landing).
            if (jmax > 0 && !wait(rfull, 0u)) mbar_drain(rfull, 0u, globaltimer());
            __syncwarp();
        }
        const float *own = part + rank * cpo * 128 + (n - n0);
        if (n < p.N) {
            for (int j = j0; j < jmax; j += step) {
                const Residual<4> r = res;
                if (RESID && j + step < jmax) linear_resid(p, tq + j + step, n, res, OUT32, walk);
                float v[4] = {}, g[4] = {};
                const float *src = red + j * 128 + (n - n0);
                for (int s = 0; s < S; ++s, src += cpo * 128) {
                    const float *q = s == rank ? own + j * 128 : src;
                    if (p.vec) {
                        const float4 x = *reinterpret_cast<const float4 *>(q);
                        v[0] += x.x, v[1] += x.y, v[2] += x.z, v[3] += x.w;
                        if (GATED) {
                            const float4 y = *reinterpret_cast<const float4 *>(q + 64);
                            g[0] += y.x, g[1] += y.y, g[2] += y.z, g[3] += y.w;
                        }
                    } else {
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            v[i] += q[i * lpt];
                            if (GATED) g[i] += q[64 + i * lpt];
                        }
                    }
                }
                linear_finish(p, tq + j, n, v, g, b, bg, r, GATED, RESID, OUT32, walk);
            }
        }
    }
    __syncwarp();
    if (S > 1) {  // no CTA leaves while a copy from or into its memory may be in flight
        umma::cluster_arrive();
        umma::cluster_wait();
    }
    umma::fence_before();
    __syncthreads();
    if (warp == 0) {
        umma::fence_after();
        umma::tmem_dealloc(tbase, (uint32_t)a.tcols);
    }
}

// Many tokens: persistent CTA pairs (cta_group::2), tiles of 256
// weight rows x bn tokens, each CTA of the pair loading its 128 weight rows
// and half of the tokens, so every operand byte a pair brings in feeds twice
// the MMA work of a single CTA's tile.  Two tensor-memory buffers: the
// epilogue of a tile runs under the next tile's MMAs.  Bound by the tensor
// cores under the power limit, and by whole waves of tiles: 4096 tokens x 7168 x
// 7168 at 1.30 to 1.46 PFLOP/s, gated 4096 x 1536 x 7168 at 1.21 to 1.28, 4095 x
// 7168 x 1536 with a residual at 1.00 to 1.06 in calls that follow one another
// for a second, at 1.25 in runs of some 10 ms.  Issue loops that keep one lane
// in a branch (without elect) ran the MMAs at two thirds of that.  fp32 outputs: the chains of the
// tile kernel, a buffer each, added in the epilogue warps' registers; a tile's
// end then covers two chains of the next tile, not all of it (4096 x 7168 x 1536
// with a residual 131 us, 4096 x 7168 x 7168 360 us).
constexpr int kLpRow = 36;                  // floats from token to token of the epilogue's buffers (4 off: no bank conflicts)
constexpr int kLpEpi = 16;                  // epilogue warps: four per lane quadrant
constexpr int kLpThreads = 32 * (kLpEpi + 2);
constexpr int kLpExch = kLpEpi * 16 * kLpRow * 4;

// drain_ring for a pair, by CTA 0's issuing role: its barriers count the copies
// of both CTAs.  What a CTA that stopped earlier will not bring is taken off,
// and the rest waited for.  CTA 1 is told to give up, and is still there (the
// closing cluster barrier).  Not inlined: in the kernel's body it changed the
// code of the loops (4095 x 7168 x 1536 with a residual 72 us, 78 with it).
__device__ __noinline__ void pair_drain(uint64_t *full, int nst, volatile int *issued, int nk, int whole, int bn, int parts) {
    const uint32_t there = umma::mapa(smem_u32(const_cast<int *>(issued)), 1u);
    umma::st_cluster(there - 4, 1u);  // its s_abort, the word before
    uint64_t t0 = globaltimer();
    int i0, i1;
    while ((i0 = *issued) < 0 || (i1 = (int)umma::ld_cluster(there)) < 0) {
        if (globaltimer() - t0 > 2 * kWaitLimitNs) return;
    }
    t0 = globaltimer();
    const int pairs = gridDim.x >> 1, end = max(i0, i1);
    for (int j = max(0, end - nst); j < end; ++j) {
        const int s = j % nst, it = (int)(blockIdx.x >> 1) + j / nk * pairs;
        const uint32_t bytes = (uint32_t)(kLtA + (it < whole ? bn : bn / parts) * 64);  // of one CTA
        if (j >= i1) umma::complete_tx(&full[s], bytes);
        if (j >= i0) mbar_arrive_expect_tx(&full[s], bytes);
        mbar_drain(&full[s], (uint32_t)((j / nst) & 1), t0);
    }
}

// OUT32: the output's type.  VEC: p.vec (a choice at run time cost the aligned
// case 2 to 4 us: 1024 x 7168 x 1536 with a residual 24.5 us, 28.3 with it).
template <bool GATED, bool RESID, bool VEC, bool OUT32>
__global__ void __launch_bounds__(kLpThreads, 1) linear_pair_kernel(const __grid_constant__ LinearTcParams a) {
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
    const LinearParams &p = a.p;
    const int nst = a.nst & 255, bn = a.bn;
    const int SB = kLtA + bn * 64;
    uint64_t *full = reinterpret_cast<uint64_t *>(smem);
    uint64_t *empty = full + nst;
    uint64_t *afull = empty + nst;
    uint64_t *aempty = afull + 2;
    uint64_t *mdone = aempty + 2;
    uint32_t *tslot = reinterpret_cast<uint32_t *>(mdone + 1);
    volatile int *s_abort = reinterpret_cast<volatile int *>(tslot + 1);
    volatile int *s_issued = s_abort + 1;  // stages that this CTA's copies filled, once all are; -1 before
    uint8_t *stages = smem + kLtHead;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int rank = (int)umma::cluster_rank();
    if (threadIdx.x == 0) {
        for (int s = 0; s < nst; ++s) {
            mbar_init(&full[s], 1);   // CTA 0's counts both CTAs' copies
            mbar_init(&empty[s], 1);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(&afull[b], 1);
            mbar_init(&aempty[b], 2 * kLpEpi);  // CTA 0's: the epilogue warps of both
        }
        mbar_init(mdone, 1);
        fence_mbar_init();
        *s_abort = 0;
        *s_issued = -1;
    }
    if (warp == kLpEpi && lane == 0) {
        umma::prefetch_tmap(a.tw);
        umma::prefetch_tmap(a.tx);
        if (a.parts > 1) umma::prefetch_tmap(a.tx_part);
    }
    if (warp == 0) umma::tmem_alloc_pair(tslot, 512u);
    umma::fence_before();
    __syncthreads();
    umma::cluster_arrive();
    umma::cluster_wait();  // both CTAs' barriers are set up
    umma::fence_after();
    const uint32_t tbase = *tslot;
    const int nrow = GATED ? 64 : 128;  // output columns of one CTA's rows
    const int nk = ceil_div(p.K, kLtKStep);
    const int chain = OUT32 ? a.chain : nk;  // K-steps per tensor-memory buffer
    const int pairs = gridDim.x >> 1, pair = blockIdx.x >> 1;
    const int items = a.whole + (a.nrb * a.ntt - a.whole) * a.parts;
    // Tiles in bands of 8 token tiles, tokens innermost: the pairs at work at
    // one time share their weight rows and their tokens through L2.
    // The tiles that would leave most pairs idle in the last wave are cut
    // into parts of fewer tokens, an item each.
    auto tile_at = [&](int it, int &n0, int &t0) {
        const bool part = it >= a.whole;
        const int tile = part ? a.whole + (it - a.whole) / a.parts : it;
        const int per = 8 * a.nrb, band = tile / per, in = tile - band * per;
        const int w = min(8, a.ntt - band * 8);
        n0 = ((in / w) * 2 + rank) * nrow;
        t0 = (band * 8 + in % w) * bn;
        if (part) t0 += (it - a.whole) % a.parts * (bn / a.parts);
        return part ? bn / a.parts : bn;  // its tokens
    };
    auto wait = [&](uint64_t *bar, uint32_t parity) { return mbar_wait_warp(bar, parity, a.hdr, a.wait_ns, s_abort); };
    pdl_wait();
    pdl_trigger();

    if (warp == kLpEpi) {
        int i = 0, s = 0;
        uint32_t ph = 1u;
        bool ok = true;
        for (int it = pair; it < items && ok; it += pairs) {
            int n0, t0;
            const int tn = tile_at(it, n0, t0), tx = t0 + rank * (tn / 2);
            const void *xmap = it < a.whole ? a.tx : a.tx_part;
            const int fill = rank == 1 && it + pairs >= items ? nk - (a.nst >> 8) : nk;
            for (int kt = 0; kt < fill; ++kt, ++i) {
                if (!wait(&empty[s], ph)) {
                    ok = false;
                    break;
                }
                if (umma::elect()) {
                    uint8_t *st = stages + s * SB;
                    const uint32_t bar = umma::mapa(smem_u32(&full[s]), 0u);
                    if (rank == 0) mbar_arrive_expect_tx(&full[s], (uint32_t)(2 * (kLtA + tn * 64)));
                    umma::tma_load_2d_pair(st, a.tw, kt * kLtKStep, n0, bar);
                    if (GATED) umma::tma_load_2d_pair(st + kLtA / 2, a.twg, kt * kLtKStep, n0, bar);
                    umma::tma_load_2d_pair(st + kLtA, xmap, kt * kLtKStep, tx, bar);
                }
                __syncwarp();
                if (++s == nst) {
                    s = 0;
                    ph ^= 1u;
                }
            }
        }
        if (lane == 0) *s_issued = i;
    } else if (warp == kLpEpi + 1) {
        if (rank == 0) {
            const uint64_t adesc = umma::smem_desc(smem_u32(stages), 16u, 1024u, umma::kLayoutSw128);
            int s = 0, q = 0;
            uint32_t ph = 0u;
            bool ok = true;
            int it = pair, kt = 0;
            for (; it < items && ok; ++q) {
                const int buf = q & 1, k0 = kt, k1 = min(nk, kt + chain);
                if (q >= 2 && !wait(&aempty[buf], (uint32_t)(((q >> 1) + 1) & 1))) break;
                const uint32_t d = tbase + (uint32_t)(buf * 256);
                const uint32_t idesc = umma::idesc_bf16_pair(it < a.whole ? bn : bn / a.parts);
                for (; kt < k1; ++kt) {
                    if (!wait(&full[s], ph)) {
                        ok = false;
                        break;
                    }
                    umma::fence_after();
                    const uint64_t ad = adesc + ((uint32_t)(s * SB) >> 4), bd = ad + (kLtA >> 4);
                    const int steps = ceil_div(p.K - kt * kLtKStep, 16);
                    if (umma::elect()) {
                        umma::mma_bf16_pair(d, ad, bd, idesc, kt > k0 ? 1u : 0u);
                        if (steps > 1) umma::mma_bf16_pair(d, ad + 2, bd + 2, idesc, 1u);
                        if (steps > 2) umma::mma_bf16_pair(d, ad + 4, bd + 4, idesc, 1u);
                        if (steps > 3) umma::mma_bf16_pair(d, ad + 6, bd + 6, idesc, 1u);
                        umma::commit_pair(&empty[s]);
                        if (kt + 1 == k1) umma::commit_pair(&afull[buf]);
                    }
                    __syncwarp();
                    if (++s == nst) {
                        s = 0;
                        ph ^= 1u;
                    }
                }
                if (kt == nk) {
                    kt = 0;
                    it += pairs;
                }
            }
            if (umma::elect()) {
                umma::commit_pair(mdone);
                if (*s_abort) pair_drain(full, nst, s_issued, nk, a.whole, a.bn, a.parts);
            }
            __syncwarp();
        }
    } else {
        // Epilogue: warp w takes lane quadrant w % 4 and every fourth group of
        // 16 tokens, through shared memory so that a thread finishes 8
        // neighbouring columns of a token.  Gated: quadrants 0, 1 hold w's rows
        // and 2, 3 w_gate's; the warps of quadrants u and u + 2 write their
        // sums of a group and finish 8 of its tokens each.
        const int quad = warp & 3, hv = warp >> 2, peer = (quad & 1) + 2 * hv;
        float *ex = reinterpret_cast<float *>(stages + nst * SB);
        float *mine = ex + warp * kLpRow * 16;  // [16 tokens][32 columns]
        const float *vs = ex + (GATED ? warp & ~2 : warp) * kLpRow * 16, *gs = ex + (warp | 2) * kLpRow * 16;
        // 8 bf16 or 4 fp32 outputs per thread and pass: 16 bytes (two stores of
        // 16 bytes each, 32 apart from lane to lane, halved the rate).
        constexpr int NV = OUT32 ? 4 : 8, LT = 32 / NV, np = (GATED ? 8 : 16) / NV;
        const LinearWalk walk{VEC ? 0 : 1, VEC ? 1 : 0, p.T};  // not VEC: a thread has one column of NV tokens
        const int tl = (GATED ? (quad >> 1) * 8 : 0) + (VEC ? lane / LT : 0);  // first token of this thread in a group
        const int nl = 32 * (GATED ? quad & 1 : quad) + (VEC ? lane % LT * NV : lane);
        int q = 0;
        for (int it = pair; it < items; it += pairs) {
            int n0, t0;
            const int tn = tile_at(it, n0, t0), n = n0 + nl;
            const int left = n < p.N ? p.T - t0 : 0;  // tokens of this tile to store
            // Residuals, one group ahead of their use (the first while the
            // tile's MMAs run).
            Residual<NV> res[np];
            auto fetch = [&](int f) {
#pragma unroll
                for (int h = 0; h < np; ++h)
                    if (RESID && f < tn && f + tl + NV * h < left) linear_resid(p, t0 + f + tl + NV * h, n, res[h], OUT32, walk);
            };
            float b[NV], bg[NV];
            auto columns = [&] {
                linear_bias(p.bias, n, walk.dn, p.N, b);
                linear_bias(p.bias_g, n, walk.dn, p.N, bg);
                fetch(hv * 16);
            };
            float acc[OUT32 ? 4 : 1][16];  // the chains' sums of this warp's groups
            bool got;
            int buf = q & 1;
            if (OUT32) {
                for (int kt = 0; kt < nk; kt += chain, ++q) {
                    buf = q & 1;
                    got = wait(&afull[buf], (uint32_t)((q >> 1) & 1));
                    __syncwarp();
                    if (!got) break;
                    umma::fence_after();
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const int f = hv * 16 + i * 4 * kLpEpi;
                        if (f < tn) {
#pragma unroll
                            for (int h = 0; h < 16; h += 8) {
                                uint32_t raw[8];
                                umma::ld8(tbase + umma::lane_base(warp) + (uint32_t)(buf * 256 + f + h), raw);
                                umma::wait_ld();
#pragma unroll
                                for (int j = 0; j < 8; ++j) {
                                    float &x = acc[OUT32 ? i : 0][h + j];
                                    x = kt == 0 ? __uint_as_float(raw[j]) : x + __uint_as_float(raw[j]);
                                }
                            }
                        }
                    }
                    umma::fence_before();
                    __syncwarp();
                    if (lane == 0) umma::arrive_cluster(umma::mapa(smem_u32(&aempty[buf]), 0u));
                    __syncwarp();
                }
                columns();
                __syncwarp();
            } else {
                columns();
                got = wait(&afull[buf], (uint32_t)((q >> 1) & 1));
                __syncwarp();
            }
            // the two warps that exchange go on together or not at all
            if (GATED) got = umma::bar_red_and(1 + peer, 64, got);
            if (!got) break;
            umma::fence_after();
            const uint32_t src = tbase + umma::lane_base(warp) + (uint32_t)(buf * 256);
#pragma unroll 1
            for (int f = hv * 16; f < tn; f += 4 * kLpEpi) {
                // opaque: no loop of a lane's own around the aligned instructions
                int lim = left;
                asm volatile("" : "+r"(lim));
                if (OUT32) {
                    // the next group's sums move up: a choice among the four
                    // would keep all of them in registers to the end
#pragma unroll
                    for (int j = 0; j < 16; ++j) mine[j * kLpRow + lane] = acc[0][j];
#pragma unroll
                    for (int i = 0; i + 1 < (OUT32 ? 4 : 1); ++i)
#pragma unroll
                        for (int j = 0; j < 16; ++j) acc[i][j] = acc[i + 1][j];
                } else {
                    uint32_t raw[16];
                    umma::ld16(src + f, raw);
                    umma::wait_ld();
#pragma unroll
                    for (int j = 0; j < 16; ++j) mine[j * kLpRow + lane] = __uint_as_float(raw[j]);
                }
                __syncwarp();
                if (GATED) umma::bar_sync(1 + peer, 64);
                float v[np][NV], g[np][NV];
                if (!VEC) {
#pragma unroll
                    for (int h = 0; h < np; ++h)
#pragma unroll
                        for (int e = 0; e < NV; ++e) {
                            v[h][e] = vs[(tl + NV * h + e) * kLpRow + lane];
                            if (GATED) g[h][e] = gs[(tl + NV * h + e) * kLpRow + lane];
                        }
                } else {
#pragma unroll
                    for (int h = 0; h < np; ++h)
#pragma unroll
                        for (int e = 0; e < NV; e += 4) {
                            const int o = (tl + NV * h) * kLpRow + lane % LT * NV + e;
                            const float4 x = *reinterpret_cast<const float4 *>(vs + o);
                            v[h][e] = x.x, v[h][e + 1] = x.y, v[h][e + 2] = x.z, v[h][e + 3] = x.w;
                            if (GATED) {
                                const float4 y = *reinterpret_cast<const float4 *>(gs + o);
                                g[h][e] = y.x, g[h][e + 1] = y.y, g[h][e + 2] = y.z, g[h][e + 3] = y.w;
                            }
                        }
                }
#pragma unroll
                for (int h = 0; h < np; ++h)
                    if (f + tl + NV * h < lim)
                        linear_finish(p, (long long)t0 + f + tl + NV * h, n, v[h], g[h], b, bg, res[h], GATED, RESID, OUT32, walk);
                fetch(f + 4 * kLpEpi);
                __syncwarp();
                if (GATED) umma::bar_sync(1 + peer, 64);
            }
            if (!OUT32) {
                umma::fence_before();
                __syncwarp();
                if (lane == 0) umma::arrive_cluster(umma::mapa(smem_u32(&aempty[buf]), 0u));
                ++q;
            }
        }
    }
    // Every role of this CTA is done: only now the wait for the last arrival
    // from the pair's MMAs, in both CTAs.  From the start its limit would be
    // one on the whole call.  (The other CTA may have two limits to go.)
    __syncthreads();
    if (warp == kLpEpi + 1) mbar_drain(mdone, 0u, globaltimer(), 4 * kWaitLimitNs);
    __syncwarp();
    umma::fence_before();
    umma::cluster_arrive();
    umma::cluster_wait();  // neither CTA leaves while the other's copies, MMAs or arrivals need it
    if (warp == 0) {
        umma::fence_after();
        umma::tmem_dealloc_pair(tbase, 512u);
    }
}

}  // namespace k3
