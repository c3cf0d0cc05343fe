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
// A warp owns a token: logits in registers as order-preserving integers.  Up to 128
// experts a lane sorts its four first, a pick is one warp-wide integer maximum of the
// lanes' heads and a vote for who holds it, and two tokens go through a warp together,
// so that one's instructions run in the other's latencies; with more experts a pick is a
// lane-local maximum, a warp-wide one and, among the lanes that hold it, a warp-wide
// minimum of the expert index.
// The sort: a token's experts differ, so a pair's place inside its group is the number of
// earlier tokens that picked the same expert: a bit per token and expert in shared memory,
// and population counts.  Up to kRouteOneTokens tokens one CTA does both (one launch);
// beyond, the picks and each CTA's expert counts are one launch and the placement -- every
// CTA sums the counts of the CTAs before it -- a second.  Both are latency-bound: the bytes
// (T E logits, T top_k x 12 out) are a microsecond of HBM at 16,384 tokens, which take
// 17 us: 11 of picks, in which 67% of the issue slots are used, and 6 of placement.  One
// token: 4.4 us.
#include <algorithm>

#include "elem.cuh"

namespace bitsmoe {

constexpr int kRtThreads = 1024;
constexpr int kRtWarps = kRtThreads / 32;
// Tokens one CTA routes and groups.  (One launch and two, us: 128 experts, 64 tokens 8.1 and 7.1, 128 tokens
// 13.2 and 7.2; 16 experts, 64 tokens 5.2 and 5.5, 128 tokens 7.1 and 5.5; 512 experts, 64 tokens 23.6 and 16.8.)
constexpr int kRouteOneTokens = 32;
constexpr int kRouteMaxBlocks = 148;  // CTAs of the two-launch path: one per SM (each sums the others' counts)
constexpr int kRouteMaxE = 8192;
constexpr int kRouteMaxK = 1024;
constexpr int kRouteMaxPairs = 1 << 30;  // T K: pairs are walked by ints in steps of kRtThreads
constexpr int kRouteBitInts = 8192;   // ints of shared memory for the bits (32 KB), if 32 tokens' fit them

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
    int32_t* hist;     // [E][nb] expert counts of each CTA's tokens (two-launch path)
    int32_t* status;
    int tpb;  // tokens per CTA
    int words;  // 32-token words of bits per expert
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

// R tokens by one warp: at most 32 NV <= 128 experts and 32 picks.  A row that is not
// finite is routed as if every expert were closed.  t[r] < 0: no token.
template <int NV, int R>
__device__ __forceinline__ void route_tokens(const RouteParams& P, const int (&t)[R], int lane) {
    uint32_t key[R][NV];
    int from[R][NV];  // the keys' experts, / 32
    float m[R], my_l[R];
    int my_id[R];
#pragma unroll
    for (int r = 0; r < R; r++)
#pragma unroll
        for (int j = 0; j < NV; j++) {
            const int e = lane + 32 * j;
            key[r][j] = __float_as_uint(t[r] >= 0 && e < P.E ? load_logit(P, (int64_t)t[r] * P.ld, e) : -INFINITY);
        }
#pragma unroll
    for (int r = 0; r < R; r++) {
        bool bad = false;
#pragma unroll
        for (int j = 0; j < NV; j++) {
            const float v = __uint_as_float(key[r][j]);
            bad |= !(v < INFINITY);
            key[r][j] = lane + 32 * j < P.E ? logit_key(v) : 0u;
            from[r][j] = j;
        }
        bad = __any_sync(0xffffffffu, bad);
        if (bad && lane == 0 && P.status) atomicOr(P.status, BITSMOE_ST_NONFINITE);
#pragma unroll
        for (int j = 0; j < NV; j++)
            if (bad) key[r][j] = 0u;
        // descending; equal keys stay in ascending order of their experts
#pragma unroll
        for (int i = 0; i + 1 < NV; i++)
#pragma unroll
            for (int j = NV - 2; j >= i; j--) {
                const bool swap = key[r][j + 1] > key[r][j];
                const uint32_t hi = swap ? key[r][j + 1] : key[r][j], lo = swap ? key[r][j] : key[r][j + 1];
                const int fh = swap ? from[r][j + 1] : from[r][j], fl = swap ? from[r][j] : from[r][j + 1];
                key[r][j] = hi;
                key[r][j + 1] = lo;
                from[r][j] = fh;
                from[r][j + 1] = fl;
            }
        my_id[r] = -1;
        my_l[r] = m[r] = -INFINITY;
    }
    for (int k = 0; k < P.K; k++) {
        uint32_t top[R];
        unsigned who[R];
#pragma unroll
        for (int r = 0; r < R; r++) top[r] = __reduce_max_sync(0xffffffffu, key[r][0]);
#pragma unroll
        for (int r = 0; r < R; r++) who[r] = __ballot_sync(0xffffffffu, key[r][0] == top[r]);
#pragma unroll
        for (int r = 0; r < R; r++) {
            const int be = lane + 32 * from[r][0];
            int e;
            if (who[r] & (who[r] - 1u))  // equal logits: the lowest expert
                e = (int)__reduce_min_sync(0xffffffffu, key[r][0] == top[r] ? (uint32_t)be : 0x7fffffffu);
            else
                e = __shfl_sync(0xffffffffu, be, __ffs(who[r]) - 1);
            const bool open = top[r] > kKeyClosed;
            const float l = open ? key_logit(top[r]) : -INFINITY;
            if (k == 0) m[r] = l;
            if (lane == k) {
                my_id[r] = open ? e : -1;
                my_l[r] = l;
            }
            if (open && be == e) {
#pragma unroll
                for (int j = 0; j + 1 < NV; j++) {
                    key[r][j] = key[r][j + 1];
                    from[r][j] = from[r][j + 1];
                }
                key[r][NV - 1] = 0u;
            }
        }
    }
#pragma unroll
    for (int r = 0; r < R; r++) {
        const float s = my_id[r] >= 0 ? score_of(P, my_l[r], m[r]) : 0.0f;
        float total = 1.0f;
        if (P.renorm) {
            total = warp_sum(s);
        } else if (!P.sigmoid) {  // softmax over every expert: the picked ones, and what is left
            float sum = s;
#pragma unroll
            for (int j = 0; j < NV; j++)
                if (key[r][j] > kKeyClosed) sum += expf(key_logit(key[r][j]) - m[r]);
            total = warp_sum(sum);
        }
        if (t[r] >= 0 && lane < P.K) {
            P.ids[(int64_t)t[r] * P.K + lane] = my_id[r];
            P.gw[(int64_t)t[r] * P.K + lane] = my_id[r] >= 0 ? P.scale * (s / total) : 0.0f;
        }
    }
}

// Groups the pairs of the CTA's tokens [t0, t1).  nb > 1: the counts of every CTA's tokens
// are in P.hist.  s_base [E], s_bits [E][words].
__device__ void group_pairs(const RouteParams& P, int t0, int t1, int b, int nb, int32_t* s_base, uint32_t* s_bits,
                            int* s_warp) {
    __shared__ int s_total[kRtThreads], s_before[kRtThreads];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    if (nb == 1) {
        for (int e = tid; e < P.E; e += kRtThreads) s_base[e] = 0;
        __syncthreads();
        for (int p = t0 * P.K + tid; p < t1 * P.K; p += kRtThreads) {
            const int e = P.ids[p];
            if (e >= 0) atomicAdd(&s_base[e], 1);  // counts: the order of the additions does not matter
        }
        __syncthreads();
    }
    // per expert: the pairs of all CTAs, and of the CTAs before this one; then where its first pair goes
    int carry = 0;
    for (int e0 = 0; e0 < P.E; e0 += kRtThreads) {
        const int e = e0 + tid;
        if (nb > 1) {  // a warp sums four experts' counts at a time, lanes over the CTAs
            const int ne = min(kRtThreads, P.E - e0);
            for (int i = warp; i < ne; i += 4 * kRtWarps) {
                int total[4] = {}, before[4] = {};
#pragma unroll 2
                for (int q = lane; q < nb; q += 32)
#pragma unroll
                    for (int x = 0; x < 4; x++) {
                        const int c = i + x * kRtWarps < ne ? P.hist[(int64_t)(e0 + i + x * kRtWarps) * nb + q] : 0;
                        total[x] += c;
                        if (q < b) before[x] += c;
                    }
#pragma unroll
                for (int x = 0; x < 4; x++) {
                    const int t = __reduce_add_sync(0xffffffffu, total[x]), f = __reduce_add_sync(0xffffffffu, before[x]);
                    if (lane == 0 && i + x * kRtWarps < ne) {
                        s_total[i + x * kRtWarps] = t;
                        s_before[i + x * kRtWarps] = f;
                    }
                }
            }
            __syncthreads();
        }
        const int total = e >= P.E ? 0 : nb > 1 ? s_total[tid] : s_base[e];
        const int end = carry + cta_scan<kRtThreads>(total, s_warp);
        if (e < P.E) {
            s_base[e] = end - total + (nb > 1 ? s_before[tid] : 0);
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
    const int span = 32 * P.words;  // tokens whose bits fit
    for (int c0 = t0; c0 < t1; c0 += span) {
        const int p0 = c0 * P.K, p1 = min(t1, c0 + span) * P.K;
        for (int i = tid; i < P.E * P.words; i += kRtThreads) s_bits[i] = 0u;
        __syncthreads();
        for (int p = p0 + tid; p < p1; p += kRtThreads) {
            const int e = P.ids[p], t = p / P.K - c0;
            if (e >= 0) atomicOr(&s_bits[e * P.words + (t >> 5)], 1u << (t & 31));
        }
        __syncthreads();
        for (int p = p0 + tid; p < p1; p += kRtThreads) {
            const int e = P.ids[p], t = p / P.K - c0;
            if (e < 0) continue;
            const uint32_t* w = s_bits + e * P.words;
            int at = s_base[e] + __popc(w[t >> 5] & ((1u << (t & 31)) - 1u));
            for (int i = 0; i < t >> 5; i++) at += __popc(w[i]);
            P.order[at] = p;
        }
        if (c0 + span >= t1) break;
        __syncthreads();
        for (int e = tid; e < P.E; e += kRtThreads)
            for (int i = 0; i < P.words; i++) s_base[e] += __popc(s_bits[e * P.words + i]);
        __syncthreads();
    }
    if (b == nb - 1)  // the places behind the last pair
        for (int p = carry + tid; p < P.T * P.K; p += kRtThreads) P.order[p] = -1;
}

// Routes the CTA's tokens and, with one CTA, groups their pairs; with more, leaves
// each expert's count in P.hist.
template <int NV>
__global__ void __launch_bounds__(kRtThreads) k_topk_route(const RouteParams P) {
    extern __shared__ int32_t s_base[];
    __shared__ int s_warp[32];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int t0 = (int)blockIdx.x * P.tpb, t1 = min(P.T, t0 + P.tpb);
    pdl_wait();
    pdl_trigger();
    if (NV >= 1 && NV <= 4 && P.K <= 32) {
        constexpr int N = NV < 1 ? 1 : NV > 4 ? 4 : NV;
        int t = t0 + warp;
        for (; t + kRtWarps < t1; t += 2 * kRtWarps) {
            const int two[2] = {t, t + kRtWarps};
            route_tokens<N, 2>(P, two, lane);
        }
        if (t < t1) {
            const int one[1] = {t};
            route_tokens<N, 1>(P, one, lane);
        }
    } else {
        for (int t = t0 + warp; t < t1; t += kRtWarps) route_token<NV>(P, t, lane);
    }
    if (!P.offsets && !P.order) return;
    __syncthreads();  // the CTA's ids are written
    if (gridDim.x == 1) {
        group_pairs(P, t0, t1, 0, 1, s_base, reinterpret_cast<uint32_t*>(s_base + P.E), s_warp);
        return;
    }
    for (int e = threadIdx.x; e < P.E; e += kRtThreads) s_base[e] = 0;
    __syncthreads();
    for (int p = t0 * P.K + threadIdx.x; p < t1 * P.K; p += kRtThreads) {
        const int e = P.ids[p];
        if (e >= 0) atomicAdd(&s_base[e], 1);
    }
    __syncthreads();
    for (int e = threadIdx.x; e < P.E; e += kRtThreads) P.hist[(int64_t)e * gridDim.x + blockIdx.x] = s_base[e];
}

__global__ void __launch_bounds__(kRtThreads) k_group_pairs(const RouteParams P) {
    extern __shared__ int32_t s_base[];
    __shared__ int s_warp[32];
    const int t0 = (int)blockIdx.x * P.tpb, t1 = min(P.T, t0 + P.tpb);
    pdl_wait();
    pdl_trigger();
    group_pairs(P, t0, t1, (int)blockIdx.x, (int)gridDim.x, s_base, reinterpret_cast<uint32_t*>(s_base + P.E), s_warp);
}

static int route_blocks(int T) {
    if (T <= kRouteOneTokens) return 1;
    return std::min(kRouteMaxBlocks, (T + kRtWarps - 1) / kRtWarps);
}

constexpr int kRouteSmem = 80 * 1024;  // dynamic shared memory at most (8192 experts)

template <typename K>
static int grant_route_smem(K kernel, size_t smem) {
    if (smem <= 36 * 1024) return BITSMOE_OK;
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kRouteSmem);
    return e == cudaSuccess ? BITSMOE_OK : set_cuda_error(e);
}

template <int NV>
static int launch_route_kernel(const RouteParams& P, unsigned grid, size_t smem, cudaStream_t s) {
    const int rc = grant_route_smem(k_topk_route<NV>, smem);
    if (rc) return rc;
    return launch_pdl(k_topk_route<NV>, dim3(grid), dim3(kRtThreads), smem, s, P);
}

}  // namespace bitsmoe

using namespace bitsmoe;

BITSMOE_API uint64_t bitsmoe_topk_route_workspace_bytes(int32_t T, int32_t n_experts, int32_t top_k) {
    if (T < 1 || n_experts < 1 || n_experts > kRouteMaxE || top_k < 1 || (int64_t)T * top_k > kRouteMaxPairs) return 0;
    const int nb = route_blocks(T);
    return nb == 1 ? 0 : 4ull * nb * n_experts;
}

BITSMOE_API int bitsmoe_topk_route(const bitsmoe_route_args* args, void* stream) {
    if (!args) return BITSMOE_EINVAL;
    const bitsmoe_route_args& a = *args;
    const int T = a.tokens, n_experts = a.n_experts, top_k = a.top_k;
    if (T < 0 || n_experts < 1 || n_experts > kRouteMaxE || top_k < 1 || top_k > n_experts || top_k > kRouteMaxK ||
        !elem_ok(a.logits_type) || (a.scoring != BITSMOE_SCORE_SOFTMAX && a.scoring != BITSMOE_SCORE_SIGMOID) ||
        (int64_t)T * top_k > kRouteMaxPairs || a.reserved)
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
    P.words = std::max(1, std::min((P.tpb + 31) / 32, kRouteBitInts / n_experts));
    const unsigned grid = T == 0 ? 1u : (unsigned)((T + P.tpb - 1) / P.tpb);
    // the experts' places and, where this CTA places pairs, the bits
    const size_t smem_group = 4ull * n_experts * (1 + P.words);
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
    rc = grant_route_smem(k_group_pairs, smem_group);
    if (rc) return rc;
    return launch_pdl(k_group_pairs, dim3(grid), dim3(kRtThreads), smem_group, s, P);
}
