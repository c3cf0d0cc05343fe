// route_topk.cu -- top-k routing: the experts and gate weights of every token from
// its router logits, and the (token, slot) pairs grouped by expert.
//
// Per token t with logits l [E]: the top_k largest logits, in descending order, equal
// ones in ascending expert order; with s_e = softmax(l)_e or sigmoid(l_e) the gate
// weights are scale * s_e, or scale * s_e / sum of the chosen s when renormalised.
// The routed layer's pages take ids and weights as given; this is the usual router.
// A logit of -inf closes an expert to a token; a slot that finds no open expert gets
// id -1 and weight 0.  A row with a NaN or +inf logit gets -1 and 0 in every slot and
// sets BITSMOE_ST_NONFINITE.
// Groups: pairs p = t top_k + slot sorted by expert, ascending p inside an expert
// (a stable counting sort, so the order does not depend on timing), -1 behind them.
//
// A warp owns a token: logits in registers as order-preserving integers, one pick =
// a lane-local maximum, one warp-wide integer maximum and, among the lanes that
// hold it, one warp-wide minimum of the expert index (two `redux` instructions).
// The sort counts with warp matches instead of atomics.  Up to kRouteOneTokens tokens
// one CTA does both (one launch); beyond, the picks and each CTA's expert counts are
// one launch and the placement -- every CTA sums the counts of the CTAs before it --
// a second.  Both are latency-bound: the bytes (T E logits, T top_k x 12 out) are
// a microsecond of HBM at 16,384 tokens.
#include <algorithm>

#include "elem.cuh"

namespace bitsmoe {

constexpr int kRtThreads = 1024;
constexpr int kRtWarps = kRtThreads / 32;
constexpr int kRouteOneTokens = 128;  // tokens one CTA routes and groups
constexpr int kRouteMaxBlocks = 296;  // CTAs of the two-launch path: two per SM
constexpr int kRouteMaxE = 8192;
constexpr int kRouteMaxK = 1024;
constexpr int kRouteHistInts = 11264;  // ints of shared memory for the per-warp expert counts (44 KB)

struct RouteParams {
    const void* logits;
    int64_t ld;
    int type, T, E, K;
    int sigmoid, renorm;
    float scale;
    int32_t* ids;      // [T][K]
    float* gw;         // [T][K]
    int32_t* offsets;  // [E+1] or NULL
    int32_t* order;    // [T*K] or NULL
    int32_t* hist;     // [nb][E] expert counts of each CTA's tokens (two-launch path)
    int32_t* status;
    int tpb;  // tokens per CTA
    int nw;   // warps that count in the placement (their counts fit shared memory)
};

// Order-preserving integer of a finite logit or -inf (-0 and +0 are equal).
__device__ __forceinline__ uint32_t logit_key(float v) {
    const uint32_t b = __float_as_uint(v + 0.0f);
    return b ^ ((b >> 31) ? 0xffffffffu : 0x80000000u);
}
__device__ __forceinline__ float key_logit(uint32_t k) {
    return __uint_as_float(k ^ ((k >> 31) ? 0x80000000u : 0xffffffffu));
}
constexpr uint32_t kKeyClosed = 0x007fffffu;  // -inf

// The score of a logit up to a factor common to the row (m: the row's largest logit):
// e^(l - m) for softmax; for sigmoid 1 / (e^a + e^(a - l)) with a = 0, or, when the
// weights are renormalised, a = min(m, 0), which keeps a row of very negative logits
// from underflowing to 0 / 0.
__device__ __forceinline__ float score_of(const RouteParams& P, float l, float m) {
    if (!P.sigmoid) return expf(l - m);
    const float a = P.renorm ? fminf(m, 0.0f) : 0.0f;
    return 1.0f / (expf(a) + expf(a - l));
}

__device__ __forceinline__ float load_logit(const RouteParams& P, int64_t row, int e) {
    float v[1];
    load_elems<1>(P.logits, P.type, row + e, v);
    return v[0];
}

// One token by one warp.  NV > 0: E <= 32 NV, the keys stay in registers; NV = 0: any
// E, the logits are read again for every pick (the next pick is the largest key that
// comes after the last one in the order of descending key, ascending expert).
template <int NV>
__device__ void route_token(const RouteParams& P, int t, int lane) {
    const int64_t row = (int64_t)t * P.ld;
    int32_t* ids = P.ids + (int64_t)t * P.K;
    float* gw = P.gw + (int64_t)t * P.K;
    uint32_t key[NV > 0 ? NV : 1];
    bool bad = false;
    float m = -INFINITY;
    if constexpr (NV > 0) {
#pragma unroll
        for (int j = 0; j < NV; j++) {
            const int e = lane + 32 * j;
            const float v = e < P.E ? load_logit(P, row, e) : -INFINITY;
            bad |= !(v < INFINITY);
            key[j] = e < P.E ? logit_key(v) : 0u;
        }
    } else {
        for (int e = lane; e < P.E; e += 32) bad |= !(load_logit(P, row, e) < INFINITY);
    }
    if (__any_sync(0xffffffffu, bad)) {
        for (int k = lane; k < P.K; k += 32) {
            ids[k] = -1;
            gw[k] = 0.0f;
        }
        if (lane == 0 && P.status) atomicOr(P.status, BITSMOE_ST_NONFINITE);
        return;
    }
    // picks: lane k mod 32 keeps pick k while there are at most 32, else they go through memory
    int my_id = -1;
    float my_l = -INFINITY, chosen = 0.0f;
    uint32_t last = 0xffffffffu;
    int last_e = -1;
    for (int k = 0; k < P.K; k++) {
        uint32_t best = 0u;
        int be = 0x7fffffff;
        if constexpr (NV > 0) {
#pragma unroll
            for (int j = 0; j < NV; j++)
                if (key[j] > best) {
                    best = key[j];
                    be = lane + 32 * j;
                }
        } else {
            for (int e = lane; e < P.E; e += 32) {
                const uint32_t q = logit_key(load_logit(P, row, e));
                if ((q < last || (q == last && e > last_e)) && q > best) {
                    best = q;
                    be = e;
                }
            }
        }
        const uint32_t top = __reduce_max_sync(0xffffffffu, best);
        int e = -1;
        float l = -INFINITY;
        if (top > kKeyClosed) {
            e = (int)__reduce_min_sync(0xffffffffu, best == top ? (uint32_t)be : 0x7fffffffu);
            l = key_logit(top);
            if (k == 0) m = l;
            last = top;
            last_e = e;
            if constexpr (NV > 0) {
#pragma unroll
                for (int j = 0; j < NV; j++)
                    if (e == lane + 32 * j) key[j] = 0u;
            }
        }
        if (P.K <= 32) {
            if (lane == k) {
                my_id = e;
                my_l = l;
            }
        } else if (lane == 0) {
            const float s = e >= 0 ? score_of(P, l, m) : 0.0f;
            ids[k] = e;
            gw[k] = s;
            chosen += s;
        }
        if (e < 0 && P.K > 32) {  // no open expert is left: the other slots are empty too
            for (int q = k + 1 + lane; q < P.K; q += 32) {
                ids[q] = -1;
                gw[q] = 0.0f;
            }
            break;
        }
    }
    float total = 1.0f;
    if (!P.renorm && !P.sigmoid) {
        // softmax over every expert: the picked ones are added from their logits
        float sum = 0.0f;
        if constexpr (NV > 0) {
#pragma unroll
            for (int j = 0; j < NV; j++)
                if (key[j] > kKeyClosed) sum += expf(key_logit(key[j]) - m);
            if (P.K <= 32 && my_id >= 0) sum += expf(my_l - m);
        } else {
            for (int e = lane; e < P.E; e += 32) {
                const float v = load_logit(P, row, e);
                if (v > -INFINITY) sum += expf(v - m);
            }
        }
        total = warp_sum(sum);
        if (NV > 0 && P.K > 32) total += __shfl_sync(0xffffffffu, chosen, 0);
    }
    if (P.K <= 32) {
        const float s = my_id >= 0 ? score_of(P, my_l, m) : 0.0f;
        if (P.renorm) total = warp_sum(s);
        if (lane < P.K) {
            ids[lane] = my_id;
            gw[lane] = my_id >= 0 ? P.scale * (s / total) : 0.0f;
        }
    } else {
        if (P.renorm) total = __shfl_sync(0xffffffffu, chosen, 0);
        __syncwarp();
        for (int k = lane; k < P.K; k += 32) gw[k] = ids[k] >= 0 ? P.scale * (gw[k] / total) : 0.0f;
    }
}

__device__ __forceinline__ int pair_expert(const RouteParams& P, int p, int p1) { return p < p1 ? P.ids[p] : -1; }

// Counts (or places) the pairs [p0, p1) of one warp's share in ascending order; cnt
// [E]: the warp's counts, or the position of its next pair of each expert.
template <bool PLACE>
__device__ void walk_pairs(const RouteParams& P, int p0, int p1, int32_t* cnt, int lane) {
    for (int q = p0; q < p1; q += 32) {
        const int e = pair_expert(P, q + lane, p1);
        const unsigned same = __match_any_sync(0xffffffffu, e);
        const int before = __popc(same & ((1u << lane) - 1u));
        if (e >= 0) {
            const int base = cnt[e];
            if (PLACE) P.order[base + before] = q + lane;
        }
        __syncwarp();
        if (e >= 0 && before == 0) cnt[e] += __popc(same);
        __syncwarp();
    }
}

// Groups the pairs of the CTA's tokens [t0, t1).  nb > 1: the counts of the other
// CTAs' tokens are in P.hist.  s_cnt [nw][E].
__device__ void group_pairs(const RouteParams& P, int t0, int t1, int b, int nb, int32_t* s_cnt, int* s_warp) {
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int p0 = t0 * P.K, n = (t1 - t0) * P.K;
    const int share = (int)roundup((uint64_t)((n + P.nw - 1) / P.nw), 32);
    const int w0 = min(n, warp * share), w1 = min(n, (warp + 1) * share);
    for (int i = tid; i < P.nw * P.E; i += kRtThreads) s_cnt[i] = 0;
    __syncthreads();
    if (warp < P.nw && P.order) walk_pairs<false>(P, p0 + w0, p0 + w1, s_cnt + warp * P.E, lane);
    if (!P.order && warp == 0) walk_pairs<false>(P, p0, p0 + n, s_cnt, lane);  // offsets alone
    __syncthreads();
    // per expert: the pairs of the CTAs before this one, of all CTAs, and of the warps before each
    int carry = 0;
    for (int e0 = 0; e0 < P.E; e0 += kRtThreads) {
        const int e = e0 + tid;
        int before = 0, total = 0, mine = 0;
        if (e < P.E) {
            for (int w = 0; w < P.nw; w++) mine += s_cnt[w * P.E + e];
            total = mine;
            if (nb > 1) {
                total = 0;
                for (int q = 0; q < nb; q++) {
                    const int c = P.hist[(int64_t)q * P.E + e];
                    total += c;
                    if (q < b) before += c;
                }
            }
        }
        const int end = carry + cta_scan<kRtThreads>(total, s_warp);
        if (e < P.E) {
            int run = end - total + before;
            for (int w = 0; w < P.nw; w++) {
                const int c = s_cnt[w * P.E + e];
                s_cnt[w * P.E + e] = run;
                run += c;
            }
            if (b == 0 && P.offsets) {
                P.offsets[e + 1] = end;
                if (e == 0) P.offsets[0] = 0;
            }
        }
        if (tid == kRtThreads - 1) s_warp[0] = end;
        __syncthreads();
        carry = s_warp[0];
        __syncthreads();
    }
    if (!P.order) return;
    if (warp < P.nw) walk_pairs<true>(P, p0 + w0, p0 + w1, s_cnt + warp * P.E, lane);
    if (b == nb - 1)  // the places behind the last pair
        for (int p = carry + tid; p < P.T * P.K; p += kRtThreads) P.order[p] = -1;
}

// Routes the CTA's tokens and, with one CTA, groups their pairs; with more, leaves
// each expert's count in P.hist.
template <int NV>
__global__ void __launch_bounds__(kRtThreads) k_topk_route(const RouteParams P) {
    extern __shared__ int32_t s_cnt[];
    __shared__ int s_warp[32];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int t0 = (int)blockIdx.x * P.tpb, t1 = min(P.T, t0 + P.tpb);
    pdl_wait();
    pdl_trigger();
    for (int t = t0 + warp; t < t1; t += kRtWarps) route_token<NV>(P, t, lane);
    if (!P.offsets && !P.order) return;
    __syncthreads();  // the CTA's ids are written
    if (gridDim.x == 1) {
        group_pairs(P, t0, t1, 0, 1, s_cnt, s_warp);
        return;
    }
    for (int e = threadIdx.x; e < P.E; e += kRtThreads) s_cnt[e] = 0;
    __syncthreads();
    for (int p = t0 * P.K + threadIdx.x; p < t1 * P.K; p += kRtThreads) {
        const int e = P.ids[p];
        if (e >= 0) atomicAdd(&s_cnt[e], 1);  // counts: the order of the additions does not matter
    }
    __syncthreads();
    for (int e = threadIdx.x; e < P.E; e += kRtThreads) P.hist[(int64_t)blockIdx.x * P.E + e] = s_cnt[e];
}

__global__ void __launch_bounds__(kRtThreads) k_group_pairs(const RouteParams P) {
    extern __shared__ int32_t s_cnt[];
    __shared__ int s_warp[32];
    const int t0 = (int)blockIdx.x * P.tpb, t1 = min(P.T, t0 + P.tpb);
    pdl_wait();
    pdl_trigger();
    group_pairs(P, t0, t1, (int)blockIdx.x, (int)gridDim.x, s_cnt, s_warp);
}

static int route_blocks(int T) {
    if (T <= kRouteOneTokens) return 1;
    return std::min(kRouteMaxBlocks, (T + kRtWarps - 1) / kRtWarps);
}

template <int NV>
static int launch_route_kernel(const RouteParams& P, unsigned grid, size_t smem, cudaStream_t s) {
    return launch_pdl(k_topk_route<NV>, dim3(grid), dim3(kRtThreads), smem, s, P);
}

}  // namespace bitsmoe

using namespace bitsmoe;

BITSMOE_API uint64_t bitsmoe_topk_route_workspace_bytes(int32_t T, int32_t n_experts, int32_t top_k) {
    if (T < 1 || n_experts < 1 || n_experts > kRouteMaxE || top_k < 1) return 0;
    const int nb = route_blocks(T);
    return nb == 1 ? 0 : 4ull * nb * n_experts;
}

BITSMOE_API int bitsmoe_topk_route(const bitsmoe_route_args* args, void* stream) {
    if (!args) return BITSMOE_EINVAL;
    const bitsmoe_route_args& a = *args;
    const int T = a.tokens, n_experts = a.n_experts, top_k = a.top_k;
    if (T < 0 || n_experts < 1 || n_experts > kRouteMaxE || top_k < 1 || top_k > n_experts || top_k > kRouteMaxK ||
        !elem_ok(a.logits_type) || (a.scoring != BITSMOE_SCORE_SOFTMAX && a.scoring != BITSMOE_SCORE_SIGMOID) ||
        (int64_t)T * top_k > 0x7fffffff || a.reserved)
        return BITSMOE_EINVAL;
    if (T == 0 && !a.offsets) return BITSMOE_OK;
    if (T > 0 && (!a.logits || !a.topk_ids || !a.gate_w || a.logits_stride < 0)) return BITSMOE_EINVAL;
    if ((uintptr_t)a.logits % elem_bytes(a.logits_type) || (uintptr_t)a.topk_ids % 4 || (uintptr_t)a.gate_w % 4 ||
        (uintptr_t)a.offsets % 4 || (uintptr_t)a.order % 4)
        return BITSMOE_EINVAL;
    const int nb = T == 0 ? 1 : route_blocks(T);
    const bool groups = a.offsets || a.order;
    if (groups && nb > 1) {
        if (!a.workspace || (uintptr_t)a.workspace % 256) return BITSMOE_EINVAL;
        if (a.workspace_bytes < bitsmoe_topk_route_workspace_bytes(T, n_experts, top_k)) return BITSMOE_ESIZE;
    }
    cudaStream_t s = (cudaStream_t)stream;
    RouteParams P{};
    P.logits = a.logits;
    P.ld = a.logits_stride;
    P.type = a.logits_type;
    P.T = T;
    P.E = n_experts;
    P.K = top_k;
    P.sigmoid = a.scoring == BITSMOE_SCORE_SIGMOID;
    P.renorm = a.renormalise != 0;
    P.scale = a.scale;
    P.ids = a.topk_ids;
    P.gw = a.gate_w;
    P.offsets = a.offsets;
    P.order = a.order;
    P.hist = groups && nb > 1 ? (int32_t*)a.workspace : nullptr;
    P.status = a.status;
    P.tpb = (T + nb - 1) / nb;
    P.nw = std::max(1, std::min(kRtWarps, kRouteHistInts / n_experts));
    const unsigned grid = T == 0 ? 1u : (unsigned)((T + P.tpb - 1) / P.tpb);
    // expert counts: of every counting warp where this CTA places pairs, else one set
    const size_t smem_group = 4ull * P.nw * n_experts;
    const size_t smem = !groups ? 0 : grid == 1 ? smem_group : 4ull * n_experts;
    int rc;
    if (n_experts <= 32)
        rc = launch_route_kernel<1>(P, grid, smem, s);
    else if (n_experts <= 64)
        rc = launch_route_kernel<2>(P, grid, smem, s);
    else if (n_experts <= 128)
        rc = launch_route_kernel<4>(P, grid, smem, s);
    else if (n_experts <= 256)
        rc = launch_route_kernel<8>(P, grid, smem, s);
    else if (n_experts <= 512)
        rc = launch_route_kernel<16>(P, grid, smem, s);
    else
        rc = launch_route_kernel<0>(P, grid, smem, s);
    if (rc || !groups || grid == 1) return rc;
    return launch_pdl(k_group_pairs, dim3(grid), dim3(kRtThreads), smem_group, s, P);
}
