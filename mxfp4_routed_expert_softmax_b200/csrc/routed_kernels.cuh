// The layer under a given routing (k3moe_layer_routed): what stands in the
// place of the router kernels.  Decode passes: one launch that checks the
// given picks, merges repeated ones, writes the dispatch and the tensor maps
// and quantises x; the gate/up and down kernels then run as after the router.
// Grouped passes: the picks and weights, checked and merged, into the pass's
// own tables, from which the sort by expert goes on.
#pragma once

#include "common.cuh"
#include "decode_kernels.cuh"
#include "layout.cuh"
#include "prefill_kernels.cuh"

namespace k3 {

// One token's given picks, by one warp (lane j < k holds pick j): a negative
// id, an id past the last expert (reported) and every repetition of an earlier
// pick become -1, and the weight of a pick is the sum of the weights given to
// its expert, in slot order.
__device__ __forceinline__ void merge_picks(int &e, float &w, int k, int E, WsHeader *hdr) {
    const int lane = threadIdx.x & 31;
    if (lane >= k) e = -1;
    if (e >= E) {
        set_status(hdr, kStDeviceCheck);
        e = -1;
    }
    if (e < 0) {
        e = -1;
        w = 0.f;
    }
    const uint32_t same = __match_any_sync(0xffffffffu, e);
    const int first = __ffs(same) - 1;
    float sum = 0.f;
    for (int j = 0; j < k; ++j) {
        const float wj = __shfl_sync(0xffffffffu, w, j);
        if ((same >> j) & 1u) sum += wj;
    }
    const bool keep = e >= 0 && lane == first;
    w = keep ? sum : 0.f;
    e = keep ? e : -1;
}

constexpr int kGivenThreads = 256;
constexpr int kGivenMaxE = 1024;

struct GivenParams {
    RouteParams r;         // shapes, blobs, tensor-map templates; x and Tc of this chunk
    const int32_t *idx;    // given [Tc][k]
    const float *weight;   // given [Tc][k]
};

// One decode pass (Tc <= kChunk).  CTA 0: warp t merges token t's picks; the
// distinct experts in ascending id get the slots 0, 1, ... as the router's
// dispatch orders them; the shared expert's and the selected experts' tensor
// maps are rewritten where their pointers changed; the dispatch is released
// for the down pass.  The other CTAs (all of them when there is one) quantise
// x.  A chunk without any expert gets one slot with no blob and no token,
// which the expert kernels take as an expert that adds nothing.
__global__ void __launch_bounds__(kGivenThreads) given_setup_kernel(const __grid_constant__ GivenParams p) {
    const RouteParams &r = p.r;
    const Layout &L = r.L;
    WsHeader *hdr = reinterpret_cast<WsHeader *>(r.ws + L.hdr);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int nwc = kGivenThreads / 32;
    // The gate/up pass, which may start now, waits for what it reads: x on
    // prep_done, the rest on this grid.  First this grid waits itself: the
    // counters of the previous call are then back at zero.
    pdl_wait();
    pdl_trigger();
    if (blockIdx.x > 0 || gridDim.x == 1) {
        const int b0 = gridDim.x == 1 ? 0 : 1;
        build_x_pieces(r.x, r.Tc, r.d, r.ws, L, (blockIdx.x - b0) * nwc + warp, (gridDim.x - b0) * nwc,
                       r.has_shared != 0);
    }
    if (blockIdx.x == 0 && threadIdx.x == 0) refresh_tmaps(r, r.E, 1);  // index E: the shared expert's maps
    __syncthreads();
    if (threadIdx.x == 0) red_add_release(&hdr->prep_done, 1u);  // this CTA's pieces (and the shared maps)
    if (blockIdx.x > 0) return;
    __shared__ uint32_t s_mask[kGivenMaxE];  // per expert: tokens that picked it
    __shared__ uint32_t s_bits[32], s_pref[32];
    for (int e = threadIdx.x; e < r.E; e += kGivenThreads) s_mask[e] = 0u;
    if (threadIdx.x < 32) s_bits[threadIdx.x] = 0u;
    __syncthreads();
    int e = -1;
    float w = 0.f;
    if (warp < r.Tc) {
        const bool in = lane < r.k;
        e = in ? p.idx[warp * r.k + lane] : -1;
        w = in && e >= 0 ? p.weight[warp * r.k + lane] : 0.f;
        merge_picks(e, w, r.k, r.E, hdr);
        if (in) {
            reinterpret_cast<int32_t *>(r.ws + L.idx)[warp * r.k + lane] = e;
            reinterpret_cast<float *>(r.ws + L.wt)[warp * r.k + lane] = w;
        }
        if (e >= 0) {
            atomicOr(&s_mask[e], 1u << warp);
            atomicOr(&s_bits[e >> 5], 1u << (e & 31));
        }
    }
    __syncthreads();
    if (warp == 0) {
        const uint32_t c = __popc(s_bits[lane]);
        uint32_t incl = c;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const uint32_t n = __shfl_up_sync(0xffffffffu, incl, o);
            if (lane >= o) incl += n;
        }
        s_pref[lane] = incl - c;
        if (lane == 31) hdr->n_unique = incl > 0u ? incl : 1u;
        if (lane == 31 && incl == 0u) {
            reinterpret_cast<const uint8_t **>(r.ws + L.uniq_blob)[0] = nullptr;
            reinterpret_cast<int32_t *>(r.ws + L.uniq_eid)[0] = 0;
            reinterpret_cast<uint32_t *>(r.ws + L.uniq_mask)[0] = 0u;
        }
    }
    __syncthreads();
    auto slot_of = [&](int x) { return (int)(s_pref[x >> 5] + __popc(s_bits[x >> 5] & ((1u << (x & 31)) - 1u))); };
    if (e >= 0)
        reinterpret_cast<int8_t *>(r.ws + L.uniq_slot)[(size_t)slot_of(e) * kChunk + warp] = (int8_t)lane;
    const uint8_t **tc = reinterpret_cast<const uint8_t **>(r.ws + L.tcache);
    for (int x = threadIdx.x; x < r.E; x += kGivenThreads) {
        if (s_mask[x] == 0u) continue;
        const int u = slot_of(x);
        const uint8_t *b = r.blobs[x];
        if (b == nullptr || (reinterpret_cast<uintptr_t>(b) & 15u) != 0u) {
            set_status(hdr, kStDeviceCheck);
            b = nullptr;
        }
        if (b != nullptr && tc[x] != b) {
            write_expert_tmaps(r.ws, L, x, b, r.tmpl, r.scale_mask);
            tc[x] = b;
        }
        reinterpret_cast<const uint8_t **>(r.ws + L.uniq_blob)[u] = b;
        reinterpret_cast<int32_t *>(r.ws + L.uniq_eid)[u] = x;
        reinterpret_cast<uint32_t *>(r.ws + L.uniq_mask)[u] = s_mask[x];
    }
    __syncthreads();
    if (threadIdx.x == 0) red_add_release(&hdr->disp_cnt, 1u);  // the dispatch is written
}

// A grouped pass: token by token (one warp each) the merged picks and weights
// into the pass's tables.
struct PfGivenParams {
    const int32_t *idx;
    const float *weight;
    int T, E, k;
    int32_t *idx_out;
    float *w_out;
    WsHeader *hdr;
};
__global__ void __launch_bounds__(kGivenThreads) pf_given_kernel(const __grid_constant__ PfGivenParams p) {
    pdl_wait();
    pdl_trigger();
    const int lane = threadIdx.x & 31;
    const int t = blockIdx.x * (kGivenThreads / 32) + (threadIdx.x >> 5);
    if (t >= p.T) return;
    const size_t i = (size_t)t * p.k + lane;
    const bool in = lane < p.k;
    int e = in ? p.idx[i] : -1;
    float w = in && e >= 0 ? p.weight[i] : 0.f;
    merge_picks(e, w, p.k, p.E, p.hdr);
    if (in) {
        p.idx_out[i] = e;
        p.w_out[i] = w;
    }
}

// The same for up to 64 tokens, with the sort by expert and the item lists, by
// one CTA: a token is a bit of its experts' masks, so a pair's rank among its
// expert's is a population count.  In the place of five launches (58 tokens,
// 22 experts of 1792 x 128: 53 us with them).
constexpr int kPfGivenSmallT = 64;
constexpr int kPfGivenSmallThreads = 1024;

struct PfGivenSmallParams {
    PfRouteParams r;
    const int32_t *idx;   // given [T][k]
    const float *weight;  // given [T][k]
};
__global__ void __launch_bounds__(kPfGivenSmallThreads) pf_given_small_kernel(const __grid_constant__ PfGivenSmallParams p) {
    const PfRouteParams &r = p.r;
    __shared__ unsigned long long s_mask[kGivenMaxE];  // per expert: its tokens
    __shared__ uint32_t s_pos[kGivenMaxE], s_g0[kGivenMaxE], s_tot[32], s_ng;
    __shared__ int4 s_grp[kPfGivenSmallT * 32 / kGroup + kGivenMaxE + kPfGivenSmallT / kGroup];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int E = r.r.E, k = r.r.k, T = r.T;
    uint8_t *ws = r.r.ws;
    WsHeader *hdr = reinterpret_cast<WsHeader *>(ws + r.r.L.hdr);
    pdl_wait();
    pdl_trigger();
    for (int e = threadIdx.x; e < E; e += blockDim.x) s_mask[e] = 0ull;
    __syncthreads();
    constexpr int R = kPfGivenSmallT / (kPfGivenSmallThreads / 32);  // tokens per warp
    int pe[R];
    float pw[R];
#pragma unroll
    for (int i = 0; i < R; ++i) {
        const int t = warp + 32 * i;
        pe[i] = -1;
        pw[i] = 0.f;
        if (t < T) {  // alike in the warp
            const size_t at = (size_t)t * k + lane;
            if (lane < k) pe[i] = p.idx[at];
            if (lane < k && pe[i] >= 0) pw[i] = p.weight[at];
            merge_picks(pe[i], pw[i], k, E, hdr);
            if (lane < k) {
                reinterpret_cast<int32_t *>(ws + r.P.idx)[at] = pe[i];
                reinterpret_cast<float *>(ws + r.P.wt)[at] = pw[i];
            }
            if (pe[i] >= 0) atomicOr(&s_mask[pe[i]], 1ull << t);
        }
    }
    refresh_tmaps(r.r, threadIdx.x, blockDim.x);
    __syncthreads();
    const int e = threadIdx.x;
    const uint32_t n = e < E ? (uint32_t)__popcll(s_mask[e]) : 0u, ng = (n + kGroup - 1) / kGroup;
    auto scan = [&](uint32_t v) {  // block-wide, exclusive
        uint32_t incl = v;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const uint32_t u = __shfl_up_sync(0xffffffffu, incl, o);
            if (lane >= o) incl += u;
        }
        __syncthreads();
        if (lane == 31) s_tot[warp] = incl;
        __syncthreads();
        uint32_t add = 0u;
        for (int w = 0; w < warp; ++w) add += s_tot[w];
        return add + incl - v;
    };
    const uint32_t pos = scan(n), g0 = scan(ng);
    if (e < E) {
        s_pos[e] = pos;
        s_g0[e] = g0;
        int ok = 1;
        if (n > 0u) {
            const uint8_t *b = r.r.blobs[e];
            if (b == nullptr || (reinterpret_cast<uintptr_t>(b) & 15u) != 0u) {
                set_status(hdr, kStDeviceCheck);
                ok = 0;
            }
        }
        for (uint32_t i = 0; i < ng; ++i)
            s_grp[g0 + i] = make_int4(e, (int)(pos + kGroup * i), (int)min((uint32_t)kGroup, n - kGroup * i), ok);
    }
    if (threadIdx.x == kPfGivenSmallThreads - 1) s_ng = g0 + ng;
    __syncthreads();
    const int NG = (int)s_ng;
    if (threadIdx.x < r.ngs)
        s_grp[NG + threadIdx.x] = make_int4(-1, kGroup * threadIdx.x, min(kGroup, T - kGroup * (int)threadIdx.x), 1);
    if (threadIdx.x == 0) hdr->n_unique = (uint32_t)NG;
    int32_t *ploc = reinterpret_cast<int32_t *>(ws + r.P.ploc), *perm = reinterpret_cast<int32_t *>(ws + r.P.perm);
    float *pwo = reinterpret_cast<float *>(ws + r.P.pw);
#pragma unroll
    for (int i = 0; i < R; ++i) {
        const int t = warp + 32 * i;
        if (t < T && lane < k) {
            const int pid = t * k + lane;
            if (pe[i] < 0) {
                ploc[pid] = -1;
            } else {
                const uint32_t rel = (uint32_t)__popcll(s_mask[pe[i]] & ((1ull << t) - 1ull));
                perm[s_pos[pe[i]] + rel] = pid;
                pwo[s_pos[pe[i]] + rel] = pw[i];
                ploc[pid] = (int)((s_g0[pe[i]] + rel / kGroup) * kGroup + rel % kGroup);
            }
        }
    }
    __syncthreads();
    pf_write_items(r, s_grp, NG, threadIdx.x, blockDim.x);
}

}  // namespace k3
