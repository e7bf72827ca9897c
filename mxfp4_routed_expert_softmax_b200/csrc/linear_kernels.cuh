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

// One output from its sums: bias, activation, gate and residual in fp32, one
// rounding.  b, bg: the column's biases; r: the residual.
__device__ __forceinline__ float linear_value(const LinearParams &p, float v, float g, float b, float bg, float r) {
    v += b;
    return (p.wg ? linear_act(g + bg, p.act) * v : linear_act(v, p.act)) + r;
}
__device__ __forceinline__ float linear_resid(const LinearParams &p, long long t, int n) {
    if (!p.resid) return 0.f;
    return p.out_fp32 ? reinterpret_cast<const float *>(p.resid)[t * p.ldr + n]
                      : bf16_lo(reinterpret_cast<const uint16_t *>(p.resid)[t * p.ldr + n]);
}
__device__ __forceinline__ void linear_store(const LinearParams &p, long long t, int n, float a) {
    if (p.out_fp32)
        reinterpret_cast<float *>(p.out)[t * p.ldo + n] = a;
    else
        reinterpret_cast<uint16_t *>(p.out)[t * p.ldo + n] = __bfloat16_as_ushort(__float2bfloat16_rn(a));
}

// ------------------------------------------------------ few tokens: stream --
// Up to 16 tokens: the weights are read once from memory and nothing else
// counts, so they go straight from global memory into the operand registers
// of warp-level MMAs (m16n8k16: A = 16 tokens, B = 8 weight rows), without
// shared memory or a tensor-memory round trip.  A lane's 16-byte load holds 8
// consecutive k of one weight row; the same k order is used for x, so the
// order of k inside a 32-wide step is free and two MMAs take the 16 bytes as
// they are.  Warps split K in 64-wide units (a whole 128-byte line of each
// row), their sums are added in warp order.
constexpr int kLsMaxT = 16;

__device__ __forceinline__ void mma_16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                          uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint4 ldg_once(const uint4 *p) {  // no reuse inside the kernel: past L1
    uint4 v;
    asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "l"(p));
    return v;
}

// RG: groups of 8 weight rows per CTA; TG: 8-token halves; U: 64-wide units
// whose loads are in flight together.
template <int RG, bool GATED, int TG, int U>
__global__ void __launch_bounds__(512) linear_stream_kernel(const __grid_constant__ LinearParams p) {
    constexpr int NM = RG * (GATED ? 2 : 1);
    extern __shared__ float red[];  // [warps][NM][8 * TG tokens][8 rows]
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, nw = blockDim.x >> 5;
    const int g = lane >> 2, q = lane & 3;
    const int n0 = blockIdx.x * RG * 8;
    const int units = ceil_div(p.K, 64);
    pdl_wait();
    pdl_trigger();
    const uint4 zero = make_uint4(0u, 0u, 0u, 0u);
    float sum[NM][4] = {};
    for (int u0 = warp; u0 < units; u0 += nw * U) {
        uint4 w[U][2][NM];
#pragma unroll
        for (int i = 0; i < U; ++i)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int k = (u0 + i * nw) * 64 + h * 32 + q * 8;  // below 2^25
#pragma unroll
                for (int r = 0; r < NM; ++r) {
                    const int n = n0 + (GATED ? r >> 1 : r) * 8 + g;
                    const uint16_t *row = (GATED && (r & 1) ? p.wg : p.w) + (long long)n * p.ldw;
                    w[i][h][r] = k < p.K && n < p.N ? ldg_once(reinterpret_cast<const uint4 *>(row + k)) : zero;
                }
            }
        float part[NM][4] = {};  // chains of 4 U steps at most; the rest is added in fp32
#pragma unroll
        for (int i = 0; i < U; ++i)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int k = (u0 + i * nw) * 64 + h * 32 + q * 8;
                uint4 xa = zero, xb = zero;
                if (k < p.K && g < p.T) xa = __ldg(reinterpret_cast<const uint4 *>(p.x + g * p.ldx + k));
                if (TG == 2 && k < p.K && g + 8 < p.T)
                    xb = __ldg(reinterpret_cast<const uint4 *>(p.x + (g + 8) * p.ldx + k));
#pragma unroll
                for (int r = 0; r < NM; ++r) {
                    mma_16816(part[r], xa.x, xb.x, xa.y, xb.y, w[i][h][r].x, w[i][h][r].y);
                    mma_16816(part[r], xa.z, xb.z, xa.w, xb.w, w[i][h][r].z, w[i][h][r].w);
                }
            }
#pragma unroll
        for (int r = 0; r < NM; ++r)
#pragma unroll
            for (int c = 0; c < 4; ++c) sum[r][c] += part[r][c];
    }
    constexpr int TT = 8 * TG;
#pragma unroll
    for (int r = 0; r < NM; ++r) {
        float *o = red + (warp * NM + r) * TT * 8 + g * 8 + 2 * q;  // token g, rows 2q and 2q + 1
        *reinterpret_cast<float2 *>(o) = make_float2(sum[r][0], sum[r][1]);
        if (TG == 2) *reinterpret_cast<float2 *>(o + 64) = make_float2(sum[r][2], sum[r][3]);
    }
    __syncthreads();
    for (int i = threadIdx.x; i < RG * TT * 8; i += blockDim.x) {
        const int rg = i / (TT * 8), t = (i / 8) % TT, n = n0 + rg * 8 + i % 8;
        if (t >= p.T || n >= p.N) continue;
        const float b = p.bias ? __ldg(p.bias + n) : 0.f, bg = p.bias_g ? __ldg(p.bias_g + n) : 0.f;
        const float res = linear_resid(p, t, n);
        float v = 0.f, gv = 0.f;
        const float *src = red + (GATED ? 2 * rg : rg) * TT * 8 + i % (TT * 8);
        for (int w = 0; w < nw; ++w) {
            v += src[w * NM * TT * 8];
            if (GATED) gv += src[(w * NM + 1) * TT * 8];
        }
        linear_store(p, t, n, linear_value(p, v, gv, b, bg, res));
    }
}

// -------------------------------------------------------- tcgen05 kernels --
// The weights are the MMA's M side (accumulator lane = output column), the
// tokens its N side, so that a warp stores 32 neighbouring columns of one
// token at once, whatever the rows' alignment, and a column's bias is one
// register.  A gated product stacks 64 rows of w and 64 of w_gate into the 128
// rows; the two are brought together through shared memory in the epilogue.
constexpr int kLtThreads = 320;  // warps 0-7 epilogue (two per lane quadrant), 8 copies, 9 MMA issue
constexpr int kLtKStep = 64;     // bf16 per K-step: 128 bytes of every row, one swizzle atom
constexpr int kLtA = 128 * 128;  // bytes of the weight box per stage
constexpr int kLtHead = 1024;    // barriers, before the stages
constexpr int kLtMaxStages = 10;
constexpr int kLtMaxSplit = 8;
constexpr int kLtChain = 4;      // K-steps per accumulation chain of an fp32 output
constexpr int kLinearMaxT = 1 << 30;

struct LinearTcParams {
    alignas(64) uint4 tw[8];
    alignas(64) uint4 twg[8];
    alignas(64) uint4 tx[8];
    LinearParams p;
    int bn;          // tokens per tile (pair kernel: of the pair)
    int nst;         // pipeline stages
    int nrb, ntt;    // row blocks, token tiles
    int split;       // tile kernel: CTAs (one cluster) that share a tile's K
    int chain;       // tile kernel: K-steps accumulated in tensor memory at a stretch
    int tcols;       // tensor-memory columns
    int red;         // tile kernel: offset of the reduction buffer
    WsHeader *hdr;
    uint64_t wait_ns;
};

__device__ __forceinline__ void prefetch_tmap(const void *m) { asm volatile("prefetch.tensormap [%0];" ::"l"(m) : "memory"); }

// A tile of 128 weight rows x bn tokens per cluster of `split` CTAs, which
// share its K: each accumulates its part, sends every CTA of the cluster the
// columns that CTA finishes (over distributed shared memory), and finishes its
// own columns, adding the parts in rank order.
//
// The tensor core cuts its running sum at every step, so a long chain drifts:
// with fp32 outputs the sum moves to registers every `chain` K-steps (two
// tensor-memory buffers) and the pieces are added there, rounded to nearest;
// bf16 outputs take one chain, whose drift (2^-24 a step of 16) is far below
// the output's half step of 2^-9.
//
// NC: 16-column pieces per epilogue warp (bn <= 32 NC).
template <int NC>
__global__ void __launch_bounds__(kLtThreads, 1) linear_tile_kernel(const __grid_constant__ LinearTcParams a) {
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
    const LinearParams &p = a.p;
    const int nst = a.nst, bn = a.bn, S = a.split;
    const int SB = kLtA + bn * 128;
    uint64_t *full = reinterpret_cast<uint64_t *>(smem);
    uint64_t *empty = full + nst;
    uint64_t *afull = empty + nst;
    uint64_t *aempty = afull + 2;
    uint64_t *mdone = aempty + 2;
    uint32_t *tslot = reinterpret_cast<uint32_t *>(mdone + 1);
    volatile int *s_abort = reinterpret_cast<volatile int *>(tslot + 1);
    uint8_t *stages = smem + kLtHead;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (S > 1) umma::cluster_arrive();  // "this CTA has started": waited for before the first remote write
    if (threadIdx.x == 0) {
        for (int s = 0; s < nst; ++s) {
            mbar_init(&full[s], 1);
            mbar_init(&empty[s], 1);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(&afull[b], 1);
            mbar_init(&aempty[b], 8);
        }
        mbar_init(mdone, 1);
        fence_mbar_init();
        *s_abort = 0;
    }
    if (warp == 8 && lane == 0) {
        prefetch_tmap(a.tw);
        prefetch_tmap(a.tx);
    }
    if (warp == 0) umma::tmem_alloc(tslot, (uint32_t)a.tcols);
    umma::fence_before();
    __syncthreads();
    umma::fence_after();
    const uint32_t tbase = *tslot;
    const int rank = S > 1 ? (int)umma::cluster_rank() : 0;
    const int tile = blockIdx.x / S;
    const bool gated = p.wg != nullptr;
    const int nrow = gated ? 64 : 128;
    const int n0 = (tile % a.nrb) * nrow, t0 = (tile / a.nrb) * bn;
    const int nkt = ceil_div(p.K, kLtKStep);
    const int kt0 = (int)((long long)nkt * rank / S), nk = (int)((long long)nkt * (rank + 1) / S) - kt0;
    const int nch = ceil_div(nk, a.chain);
    auto wait = [&](uint64_t *bar, uint32_t parity) {
        if (*s_abort) return false;
        if (mbar_wait_bounded(bar, parity, a.hdr, a.wait_ns)) return true;
        *s_abort = 1;
        return false;
    };
    pdl_wait();
    pdl_trigger();

    const int half = warp >> 2, hcols = ((bn / 16 + 1) / 2) * 16;  // columns of the first of a quadrant's warps
    const int c0 = half * hcols, ncol = half ? bn - hcols : hcols;
    float acc[NC][16];
    if (warp == 8) {
        if (lane == 0) {
            int i = 0;
            for (; i < nk; ++i) {
                const int s = i % nst;
                if (i >= nst && !wait(&empty[s], (uint32_t)(((i / nst) + 1) & 1))) break;
                uint8_t *st = stages + s * SB;
                const int x = (kt0 + i) * kLtKStep;
                mbar_arrive_expect_tx(&full[s], (uint32_t)SB);
                umma::tma_load_2d(st, a.tw, x, n0, &full[s]);
                if (gated) umma::tma_load_2d(st + kLtA / 2, a.twg, x, n0, &full[s]);
                umma::tma_load_2d(st + kLtA, a.tx, x, t0, &full[s]);
            }
            if (*s_abort) {
                for (int s = 0; s < nst && s < i; ++s) {
                    const int last = s + ((i - 1 - s) / nst) * nst;
                    mbar_drain(&full[s], (uint32_t)((last / nst) & 1), a.wait_ns);
                }
            }
        }
    } else if (warp == 9) {
        if (lane == 0) {
            const uint64_t adesc = umma::smem_desc(smem_u32(stages), 16u, 1024u, umma::kLayoutSw128);
            const uint32_t idesc = umma::idesc_bf16(bn);
            bool ok = true;
            for (int c = 0; c < nch && ok; ++c) {
                const int buf = c & 1;
                if (c >= 2 && !wait(&aempty[buf], (uint32_t)(((c >> 1) + 1) & 1))) break;
                umma::fence_after();
                const uint32_t d = tbase + (uint32_t)(buf * bn);
                uint32_t go = 0u;
                const int i1 = min(nk, (c + 1) * a.chain);
                for (int i = c * a.chain; i < i1; ++i) {
                    const int s = i % nst;
                    if (!wait(&full[s], (uint32_t)((i / nst) & 1))) {
                        ok = false;
                        break;
                    }
                    umma::fence_after();
                    const uint64_t ad = adesc + ((uint32_t)(s * SB) >> 4), bd = ad + (kLtA >> 4);
                    const int steps = min(4, ceil_div(p.K - (kt0 + i) * kLtKStep, 16));  // past K: zeros from TMA
#pragma unroll
                    for (int sk = 0; sk < 4; ++sk) {
                        if (sk < steps) {
                            umma::mma_bf16(d, ad + 2 * sk, bd + 2 * sk, idesc, go);
                            go = 1u;
                        }
                    }
                    umma::commit(&empty[s]);
                }
                umma::commit(&afull[buf]);
            }
            umma::commit(mdone);
            mbar_drain(mdone, 0u, a.wait_ns);
        }
    } else {
        for (int c = 0; c < nch; ++c) {
            const int buf = c & 1;
            int got = 0;
            if (lane == 0) got = wait(&afull[buf], (uint32_t)((c >> 1) & 1));
            if (!__shfl_sync(0xffffffffu, got, 0)) break;
            umma::fence_after();
            const uint32_t src = tbase + umma::lane_base(warp) + (uint32_t)(buf * bn + c0);
#pragma unroll
            for (int j = 0; j < NC; ++j) {
                if (16 * j < ncol) {
                    uint32_t r[16];
                    umma::ld16(src + 16 * j, r);
                    umma::wait_ld();
#pragma unroll
                    for (int i = 0; i < 16; ++i)
                        acc[j][i] = c == 0 ? __uint_as_float(r[i]) : acc[j][i] + __uint_as_float(r[i]);
                }
            }
            umma::fence_before();
            __syncwarp();
            if (lane == 0)
                asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_u32(&aempty[buf])) : "memory");
        }
    }
    __syncwarp();

    const int row = 32 * (warp & 3) + lane;
    if (S == 1 && !gated) {
        const int n = n0 + row;
        if (warp < 8 && n < p.N) {
            const float b = p.bias ? __ldg(p.bias + n) : 0.f;
#pragma unroll
            for (int j = 0; j < NC; ++j) {
                if (16 * j < ncol) {
                    float r[16];
#pragma unroll
                    for (int i = 0; i < 16; ++i) {
                        const long long t = (long long)t0 + c0 + 16 * j + i;
                        r[i] = t < p.T ? linear_resid(p, t, n) : 0.f;
                    }
#pragma unroll
                    for (int i = 0; i < 16; ++i) {
                        const long long t = (long long)t0 + c0 + 16 * j + i;
                        if (t < p.T) linear_store(p, t, n, linear_value(p, acc[j][i], 0.f, b, 0.f, r[i]));
                    }
                }
            }
        }
    } else {
        // red[source][column][row] of the columns this CTA finishes
        const int cpo = ceil_div(bn, S);
        float *red = reinterpret_cast<float *>(smem + a.red);
        if (S > 1) umma::cluster_wait();
        if (warp < 8) {
            const uint32_t base = smem_u32(red) + (uint32_t)(rank * cpo * 128 + row) * 4u;
#pragma unroll
            for (int j = 0; j < NC; ++j) {
                if (16 * j < ncol) {
#pragma unroll
                    for (int i = 0; i < 16; ++i) {
                        const int col = c0 + 16 * j + i, o = col / cpo;
                        if (t0 + col < p.T) {
                            const uint32_t at = base + (uint32_t)(col - o * cpo) * 512u;
                            umma::st_cluster(S > 1 ? umma::mapa(at, (uint32_t)o) : at, acc[j][i]);
                        }
                    }
                }
            }
        }
        if (S > 1) {
            umma::cluster_arrive();
            umma::cluster_wait();
        } else {
            __syncthreads();
        }
        if (warp < 8) {
            const int nl = threadIdx.x & (nrow - 1), n = n0 + nl, step = 256 / nrow;
            const int jmax = min(cpo, min(bn, p.T - t0) - rank * cpo);
            const float b = p.bias && n < p.N ? __ldg(p.bias + n) : 0.f;
            const float bg = p.bias_g && n < p.N ? __ldg(p.bias_g + n) : 0.f;
            if (n < p.N) {
#pragma unroll 4
                for (int j = threadIdx.x / nrow; j < jmax; j += step) {
                    const long long t = (long long)t0 + rank * cpo + j;
                    const float res = linear_resid(p, t, n);
                    const float *r = red + j * 128 + nl;
                    float v = 0.f, g = 0.f;
                    for (int s = 0; s < S; ++s) {
                        v += r[s * cpo * 128];
                        if (gated) g += r[s * cpo * 128 + 64];
                    }
                    linear_store(p, t, n, linear_value(p, v, g, b, bg, res));
                }
            }
        }
    }
    umma::fence_before();
    __syncthreads();
    if (warp == 0) {
        umma::fence_after();
        umma::tmem_dealloc(tbase, (uint32_t)a.tcols);
    }
}

// Many tokens, bf16 output: persistent CTA pairs (cta_group::2), tiles of 256
// weight rows x bn tokens, each CTA of the pair loading its 128 weight rows
// and half of the tokens, so every operand byte a pair brings in feeds twice
// the MMA work of a single CTA's tile.  Two tensor-memory buffers: the
// epilogue of a tile runs under the next tile's MMAs.
constexpr int kLpExch = 4 * 32 * 32 * 4;  // gated: 32 x 32 fp32 for each of the four pairs of epilogue warps

__global__ void __launch_bounds__(kLtThreads, 1) linear_pair_kernel(const __grid_constant__ LinearTcParams a) {
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
    const LinearParams &p = a.p;
    const int nst = a.nst, bn = a.bn;
    const int SB = kLtA + bn * 64;
    uint64_t *full = reinterpret_cast<uint64_t *>(smem);
    uint64_t *empty = full + nst;
    uint64_t *afull = empty + nst;
    uint64_t *aempty = afull + 2;
    uint64_t *mdone = aempty + 2;
    uint32_t *tslot = reinterpret_cast<uint32_t *>(mdone + 1);
    volatile int *s_abort = reinterpret_cast<volatile int *>(tslot + 1);
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
            mbar_init(&aempty[b], 16);  // CTA 0's: the epilogue warps of both
        }
        mbar_init(mdone, 1);
        fence_mbar_init();
        *s_abort = 0;
    }
    if (warp == 8 && lane == 0) {
        prefetch_tmap(a.tw);
        prefetch_tmap(a.tx);
    }
    if (warp == 0) umma::tmem_alloc_pair(tslot, 512u);
    umma::fence_before();
    __syncthreads();
    umma::cluster_arrive();
    umma::cluster_wait();  // both CTAs' barriers are set up
    umma::fence_after();
    const uint32_t tbase = *tslot;
    const bool gated = p.wg != nullptr;
    const int nrow = gated ? 64 : 128;  // output columns of one CTA's rows
    const int nk = ceil_div(p.K, kLtKStep);
    const int pairs = gridDim.x >> 1, pair = blockIdx.x >> 1;
    const int items = a.nrb * a.ntt;
    // Tiles in bands of 8 token tiles, tokens innermost: the pairs at work at
    // one time share their weight rows and their tokens through L2.
    auto tile_at = [&](int it, int &n0, int &t0) {
        const int per = 8 * a.nrb, band = it / per, in = it - band * per;
        const int w = min(8, a.ntt - band * 8);
        n0 = ((in / w) * 2 + rank) * nrow;
        t0 = (band * 8 + in % w) * bn;
    };
    auto wait = [&](uint64_t *bar, uint32_t parity) {
        if (*s_abort) return false;
        if (mbar_wait_bounded(bar, parity, a.hdr, a.wait_ns)) return true;
        *s_abort = 1;
        return false;
    };
    pdl_wait();
    pdl_trigger();

    if (warp == 8) {
        if (lane == 0) {
            int i = 0;
            for (int it = pair; it < items && !*s_abort; it += pairs) {
                int n0, t0;
                tile_at(it, n0, t0);
                for (int kt = 0; kt < nk; ++kt, ++i) {
                    const int s = i % nst;
                    if (i >= nst && !wait(&empty[s], (uint32_t)(((i / nst) + 1) & 1))) break;
                    uint8_t *st = stages + s * SB;
                    const uint32_t bar = umma::mapa(smem_u32(&full[s]), 0u);
                    if (rank == 0) mbar_arrive_expect_tx(&full[s], (uint32_t)(2 * SB));
                    umma::tma_load_2d_pair(st, a.tw, kt * kLtKStep, n0, bar);
                    if (gated) umma::tma_load_2d_pair(st + kLtA / 2, a.twg, kt * kLtKStep, n0, bar);
                    umma::tma_load_2d_pair(st + kLtA, a.tx, kt * kLtKStep, t0 + rank * (bn / 2), bar);
                }
            }
            if (*s_abort && rank == 0) {
                for (int s = 0; s < nst && s < i; ++s) {
                    const int last = s + ((i - 1 - s) / nst) * nst;
                    mbar_drain(&full[s], (uint32_t)((last / nst) & 1), a.wait_ns);
                }
            }
        }
    } else if (warp == 9) {
        if (lane == 0 && rank == 0) {
            const uint64_t adesc = umma::smem_desc(smem_u32(stages), 16u, 1024u, umma::kLayoutSw128);
            const uint32_t idesc = umma::idesc_bf16_pair(bn);
            int i = 0, q = 0;
            bool ok = true;
            for (int it = pair; it < items && ok; it += pairs, ++q) {
                const int buf = q & 1;
                if (q >= 2 && !wait(&aempty[buf], (uint32_t)(((q >> 1) + 1) & 1))) break;
                umma::fence_after();
                const uint32_t d = tbase + (uint32_t)(buf * 256);
                uint32_t go = 0u;
                for (int kt = 0; kt < nk; ++kt, ++i) {
                    const int s = i % nst;
                    if (!wait(&full[s], (uint32_t)((i / nst) & 1))) {
                        ok = false;
                        break;
                    }
                    umma::fence_after();
                    const uint64_t ad = adesc + ((uint32_t)(s * SB) >> 4), bd = ad + (kLtA >> 4);
                    const int steps = min(4, ceil_div(p.K - kt * kLtKStep, 16));
#pragma unroll
                    for (int sk = 0; sk < 4; ++sk) {
                        if (sk < steps) {
                            umma::mma_bf16_pair(d, ad + 2 * sk, bd + 2 * sk, idesc, go);
                            go = 1u;
                        }
                    }
                    umma::commit_pair(&empty[s]);
                }
                umma::commit_pair(&afull[buf]);
            }
            umma::commit_pair(mdone);
        }
        if (lane == 0) mbar_drain(mdone, 0u, a.wait_ns);  // in both CTAs: the last arrival from the pair's MMAs
    } else {
        // Epilogue: warp w takes lane quadrant w % 4 and every second group of
        // 32 tokens.  Gated: quadrants 0, 1 hold w's rows and 2, 3 w_gate's;
        // the warps of quadrants u and u + 2 exchange halves, so that one
        // finishes 16 of the 32 tokens and the other the rest.
        const int quad = warp & 3, hv = warp >> 2;
        float *ex = reinterpret_cast<float *>(stages + nst * SB) + ((quad & 1) * 2 + hv) * (32 * 32);
        const int nl = gated ? 32 * (quad & 1) + lane : 32 * quad + lane;
        int q = 0;
        for (int it = pair; it < items; it += pairs, ++q) {
            int n0, t0;
            tile_at(it, n0, t0);
            const int n = n0 + nl, buf = q & 1;
            const bool nin = n < p.N;
            const float b = p.bias && nin ? __ldg(p.bias + n) : 0.f;
            const float bg = p.bias_g && nin ? __ldg(p.bias_g + n) : 0.f;
            const uint16_t *rp = reinterpret_cast<const uint16_t *>(p.resid);
            uint16_t *op = reinterpret_cast<uint16_t *>(p.out);
            int got = 0;
            if (lane == 0) got = wait(&afull[buf], (uint32_t)((q >> 1) & 1));
            got = __shfl_sync(0xffffffffu, got, 0);
            // the two warps that exchange go on together or not at all
            if (gated) got = umma::bar_red_and(1 + (quad & 1) * 2 + hv, 64, got != 0);
            if (!got) break;
            umma::fence_after();
            const uint32_t src = tbase + umma::lane_base(warp) + (uint32_t)(buf * 256);
            for (int c = hv * 32; c < bn; c += 64) {
                uint32_t v[32];
                umma::ld32(src + c, v);
                const int tc = t0 + c;
                if (!gated) {
                    uint32_t r[32];
#pragma unroll
                    for (int j = 0; j < 32; ++j)
                        r[j] = rp && nin && tc + j < p.T ? rp[(long long)(tc + j) * p.ldr + n] : 0u;
                    umma::wait_ld();
#pragma unroll
                    for (int j = 0; j < 32; ++j)
                        if (nin && tc + j < p.T)
                            op[(long long)(tc + j) * p.ldo + n] = __bfloat16_as_ushort(__float2bfloat16_rn(
                                linear_act(__uint_as_float(v[j]) + b, p.act) + bf16_lo(r[j])));
                } else {
                    umma::wait_ld();
                    const bool low = quad < 2;  // holds w's sums, finishes tokens 0-15
#pragma unroll
                    for (int j = 0; j < 16; ++j) {
                        ex[(low ? j + 16 : j) * 32 + lane] = __uint_as_float(low ? v[j + 16] : v[j]);
                    }
                    umma::bar_sync(1 + (quad & 1) * 2 + hv, 64);
#pragma unroll
                    for (int j = 0; j < 16; ++j) {
                        const float other = ex[(low ? j : j + 16) * 32 + lane];
                        const float mine = __uint_as_float(low ? v[j] : v[j + 16]);
                        const int t = tc + (low ? j : j + 16);
                        if (nin && t < p.T) {
                            const float res = rp ? bf16_lo(rp[(long long)t * p.ldr + n]) : 0.f;
                            const float o = linear_value(p, low ? mine : other, low ? other : mine, b, bg, res);
                            op[(long long)t * p.ldo + n] = __bfloat16_as_ushort(__float2bfloat16_rn(o));
                        }
                    }
                    umma::bar_sync(1 + (quad & 1) * 2 + hv, 64);
                }
            }
            umma::fence_before();
            __syncwarp();
            if (lane == 0) umma::arrive_cluster(umma::mapa(smem_u32(&aempty[buf]), 0u));
        }
    }
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
