// norm.cu -- the norms before and after a block, fused with its gate and residual.
//
// Per token (row) of width d, with h the residual stream and y a block's output:
//   u  = y                                        (w_post NULL)
//   u  = y rsqrt(mean(y^2) + eps) w_post          (a norm on the block's output)
//   h' = h + alpha gate u                         (gate: one factor per token, per channel, or both)
//   x  = h' rsqrt(mean(h'^2) + eps) w_pre         (the next block's input)
// The spectral layer's pages do not state a block's surroundings; this is the usual
// pre-norm block, with the optional second norm.  x is formed from the fp32 h', not
// from the stored one: one rounding fewer where h is held in 16 bits.
//
// One pass over memory: a row stays in registers between its loads and its stores,
// so the step is bound by HBM (h and y read once, h' and x written once).  A row
// belongs to a CTA (to one warp when that holds it in a chunk per lane: no CTA
// barrier); the two sums are reduced in a fixed order, so results do not depend on
// timing.  Rows too wide for registers are read once more per sum.
//
// 8,192 x 4,096, bf16 h and x, fp32 y, both norms and a gate per channel: 70 us, 4.8 TB/s
// (the floor is 52).  The rest is each row's chain -- loads, two sums over the CTA, three
// vectors from L1 -- at 94% of the SM's threads.  Slower were: two rows a CTA (83 us), 256
// threads a row (72), loads through a ring in shared memory by persistent CTAs (73 to 124,
// by its depth), the channel vectors held in registers (86 and more): all hold fewer rows
// or leave L1 too small for the vectors.
#include <algorithm>

#include "elem.cuh"

namespace bitsmoe {

constexpr int kNormThreads = 512;  // threads per row, at most, while it stays in registers

struct NormParams {
    const void* h;
    const void* y;        // or NULL
    const float* w_post;  // or NULL
    const float* gate;    // or NULL
    const float* w_pre;   // or NULL when x is NULL
    void* h_out;          // or NULL
    void* x;              // or NULL
    int64_t h_ld, y_ld, ho_ld, x_ld, gate_t, gate_i;
    int64_t T;
    int d, h_type, y_type, x_type;
    float alpha, eps;
};

// Sum over the row's threads, the same in every one of them (fixed order).
template <bool WARP>
__device__ __forceinline__ float row_sum(float v, float* s_part) {
    v = warp_sum(v);
    if (WARP) return v;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, nw = (int)blockDim.x >> 5;
    if (lane == 0) s_part[warp] = v;
    __syncthreads();
    v = lane < nw ? s_part[lane] : 0.0f;
    return warp_sum(v);
}

// NC chunks of V elements per thread; NC = 0: the row is read again for every sum.
template <int V, int NC, bool WARP>
__global__ void __launch_bounds__(WARP ? 256 : NC > 0 ? kNormThreads : 1024) k_norm_residual(const NormParams P) {
    __shared__ float s_part[2][32];
    const int lane_in_row = WARP ? (int)threadIdx.x & 31 : (int)threadIdx.x;
    const int nthr = WARP ? 32 : (int)blockDim.x;
    const int64_t t = WARP ? (int64_t)blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5) : (int64_t)blockIdx.x;
    const int nch = P.d / V;
    const float inv_d = 1.0f / (float)P.d;
    pdl_wait();
    pdl_trigger();
    if (t >= P.T) return;  // whole warps (WARP) only
    const int64_t h0 = t * P.h_ld, y0 = t * P.y_ld, ho0 = t * P.ho_ld, x0 = t * P.x_ld, g0 = t * P.gate_t;

    if constexpr (NC > 0) {
        float hv[NC][V], yv[NC][V];
#pragma unroll
        for (int j = 0; j < NC; j++) {
            const int c = lane_in_row + j * nthr;
            if (c < nch) {
                load_elems<V>(P.h, P.h_type, h0 + (int64_t)c * V, hv[j]);
                if (P.y) load_elems<V>(P.y, P.y_type, y0 + (int64_t)c * V, yv[j]);
            } else {
#pragma unroll
                for (int i = 0; i < V; i++) hv[j][i] = yv[j][i] = 0.0f;
            }
        }
        if (P.y) {
            float r = P.alpha;
            if (P.w_post) {
                float ss = 0.0f;
#pragma unroll
                for (int j = 0; j < NC; j++)
#pragma unroll
                    for (int i = 0; i < V; i++) ss = fmaf(yv[j][i], yv[j][i], ss);
                const float ry = rsqrtf(fmaf(row_sum<WARP>(ss, s_part[0]), inv_d, P.eps));
#pragma unroll
                for (int j = 0; j < NC; j++) {
                    const int c = lane_in_row + j * nthr;
                    if (c < nch) {
                        float w[V];
                        load_elems<V>(P.w_post, BITSMOE_F32, (int64_t)c * V, w);
#pragma unroll
                        for (int i = 0; i < V; i++) yv[j][i] *= ry * w[i];
                    }
                }
            }
            if (P.gate && P.gate_i == 0) r *= P.gate[g0];
#pragma unroll
            for (int j = 0; j < NC; j++) {
                const int c = lane_in_row + j * nthr;
                if (c < nch) {
                    if (P.gate && P.gate_i) {
                        float g[V];
                        load_elems<V>(P.gate, BITSMOE_F32, g0 + (int64_t)c * V, g);
#pragma unroll
                        for (int i = 0; i < V; i++) yv[j][i] *= g[i];
                    }
#pragma unroll
                    for (int i = 0; i < V; i++) hv[j][i] = fmaf(r, yv[j][i], hv[j][i]);
                }
            }
        }
        if (P.h_out) {
#pragma unroll
            for (int j = 0; j < NC; j++) {
                const int c = lane_in_row + j * nthr;
                if (c < nch) store_elems<V>(P.h_out, P.h_type, ho0 + (int64_t)c * V, hv[j]);
            }
        }
        if (!P.x) return;
        float ss = 0.0f;
#pragma unroll
        for (int j = 0; j < NC; j++)
#pragma unroll
            for (int i = 0; i < V; i++) ss = fmaf(hv[j][i], hv[j][i], ss);
        const float rx = rsqrtf(fmaf(row_sum<WARP>(ss, s_part[1]), inv_d, P.eps));
#pragma unroll
        for (int j = 0; j < NC; j++) {
            const int c = lane_in_row + j * nthr;
            if (c < nch) {
                float w[V];
                load_elems<V>(P.w_pre, BITSMOE_F32, (int64_t)c * V, w);
#pragma unroll
                for (int i = 0; i < V; i++) hv[j][i] *= rx * w[i];
                store_elems<V>(P.x, P.x_type, x0 + (int64_t)c * V, hv[j]);
            }
        }
    } else {
        float ry = 1.0f;
        if (P.y && P.w_post) {
            float ss = 0.0f;
            for (int c = lane_in_row; c < nch; c += nthr) {
                float v[V];
                load_elems<V>(P.y, P.y_type, y0 + (int64_t)c * V, v);
#pragma unroll
                for (int i = 0; i < V; i++) ss = fmaf(v[i], v[i], ss);
            }
            ry = rsqrtf(fmaf(row_sum<WARP>(ss, s_part[0]), inv_d, P.eps));
        }
        float r = P.alpha;
        if (P.gate && P.gate_i == 0) r *= P.gate[g0];
        auto chunk = [&](int c, float(&hv)[V]) {
            load_elems<V>(P.h, P.h_type, h0 + (int64_t)c * V, hv);
            if (!P.y) return;
            float v[V], w[V];
            load_elems<V>(P.y, P.y_type, y0 + (int64_t)c * V, v);
            if (P.w_post) {
                load_elems<V>(P.w_post, BITSMOE_F32, (int64_t)c * V, w);
#pragma unroll
                for (int i = 0; i < V; i++) v[i] *= ry * w[i];
            }
            if (P.gate && P.gate_i) {
                load_elems<V>(P.gate, BITSMOE_F32, g0 + (int64_t)c * V, w);
#pragma unroll
                for (int i = 0; i < V; i++) v[i] *= w[i];
            }
#pragma unroll
            for (int i = 0; i < V; i++) hv[i] = fmaf(r, v[i], hv[i]);
        };
        float rx = 1.0f;
        if (P.x) {
            float ss = 0.0f;
            for (int c = lane_in_row; c < nch; c += nthr) {
                float v[V];
                chunk(c, v);
#pragma unroll
                for (int i = 0; i < V; i++) ss = fmaf(v[i], v[i], ss);
            }
            rx = rsqrtf(fmaf(row_sum<WARP>(ss, s_part[1]), inv_d, P.eps));
        }
        // h_out may be h: a thread reads a chunk before it overwrites it, and no other thread reads it
        for (int c = lane_in_row; c < nch; c += nthr) {
            float v[V];
            chunk(c, v);
            if (P.h_out) store_elems<V>(P.h_out, P.h_type, ho0 + (int64_t)c * V, v);
            if (P.x) {
                float w[V];
                load_elems<V>(P.w_pre, BITSMOE_F32, (int64_t)c * V, w);
#pragma unroll
                for (int i = 0; i < V; i++) v[i] *= rx * w[i];
                store_elems<V>(P.x, P.x_type, x0 + (int64_t)c * V, v);
            }
        }
    }
}

constexpr int kNormWarpRows = 8;  // rows (warps) per CTA when a row belongs to a warp

template <int V>
static int launch_norm(const NormParams& P, cudaStream_t s) {
    const int nch = P.d / V;
    // A row in one warp while it is one chunk a lane; longer ones are a chain of too many instructions (8,192 rows of
    // 256: 4.1 us against 8.9 with a CTA each; of 512: 8.7 and 9.0, but 16 rows 2.6 and 1.9; of 1024: 27 and 14).
    if (nch <= 32 && P.T > 1) {
        const dim3 grid((unsigned)((P.T + kNormWarpRows - 1) / kNormWarpRows)), block(32 * kNormWarpRows);
        return launch_pdl(k_norm_residual<V, 1, true>, grid, block, 0, s, P);
    }
    const dim3 grid((unsigned)P.T);
    auto threads = [&](int nc) { return (unsigned)std::max<int64_t>(32, roundup((nch + nc - 1) / nc, 32)); };
    constexpr int N0 = V == 8 ? 1 : 4;  // chunks per thread: N0, 2 N0 or 4 N0
    if (nch <= N0 * kNormThreads) return launch_pdl(k_norm_residual<V, N0, false>, grid, threads(N0), 0, s, P);
    if (nch <= 2 * N0 * kNormThreads) return launch_pdl(k_norm_residual<V, 2 * N0, false>, grid, threads(2 * N0), 0, s, P);
    if (nch <= 4 * N0 * kNormThreads) return launch_pdl(k_norm_residual<V, 4 * N0, false>, grid, threads(4 * N0), 0, s, P);
    return launch_pdl(k_norm_residual<V, 0, false>, grid, 1024, 0, s, P);
}

}  // namespace bitsmoe

using namespace bitsmoe;

BITSMOE_API int bitsmoe_norm_residual(const bitsmoe_norm_args* args, void* stream) {
    if (!args) return BITSMOE_EINVAL;
    const bitsmoe_norm_args& a = *args;
    if (a.rows < 0 || a.d < 1 || !elem_ok(a.h_type) || (a.y && !elem_ok(a.y_type)) || (a.x && !elem_ok(a.x_type)))
        return BITSMOE_EINVAL;
    if (a.rows == 0) return BITSMOE_OK;
    if (!a.h || (!a.h_out && !a.x) || (a.x && !a.w_pre) || (!a.y && (a.w_post || a.gate))) return BITSMOE_EINVAL;
    if (a.h_stride < 0 || (a.y && a.y_stride < 0) || a.gate_stride < 0 || !(a.eps >= 0.0f)) return BITSMOE_EINVAL;
    // rows that are written must not overlap, and a row of h is read before its place is written
    if (a.rows > 1 && ((a.h_out && a.h_out_stride < a.d) || (a.x && a.x_stride < a.d) ||
                       (a.h_out == a.h && a.h_out_stride != a.h_stride)))
        return BITSMOE_EINVAL;
    const int hb = elem_bytes(a.h_type);
    if ((uintptr_t)a.h % hb || (uintptr_t)a.h_out % hb || (a.y && (uintptr_t)a.y % elem_bytes(a.y_type)) ||
        (a.x && (uintptr_t)a.x % elem_bytes(a.x_type)) || (uintptr_t)a.w_post % 4 || (uintptr_t)a.gate % 4 ||
        (uintptr_t)a.w_pre % 4)
        return BITSMOE_EINVAL;
    NormParams P{};
    P.h = a.h;
    P.y = a.y;
    P.w_post = a.w_post;
    P.gate = a.gate;
    P.w_pre = a.w_pre;
    P.h_out = a.h_out;
    P.x = a.x;
    P.h_ld = a.h_stride;
    P.y_ld = a.y_stride;
    P.ho_ld = a.h_out_stride;
    P.x_ld = a.x_stride;
    P.gate_t = a.gate_stride;
    P.gate_i = a.gate_per_channel ? 1 : 0;
    P.T = a.rows;
    P.d = a.d;
    P.h_type = a.h_type;
    P.y_type = a.y_type;
    P.x_type = a.x_type;
    P.alpha = a.alpha;
    P.eps = a.eps;
    // 16-byte accesses where every row of every buffer starts on a 16-byte boundary
    auto vec = [](const void* p, int type, int64_t ld) {
        return !p || ((uintptr_t)p % 16 == 0 && (ld * elem_bytes(type)) % 16 == 0);
    };
    const bool v8 = a.d % 8 == 0 && vec(a.h, a.h_type, a.h_stride) && vec(a.y, a.y_type, a.y_stride) &&
                    vec(a.h_out, a.h_type, a.h_out_stride) && vec(a.x, a.x_type, a.x_stride) &&
                    vec(a.w_post, BITSMOE_F32, 0) && vec(a.w_pre, BITSMOE_F32, 0) &&
                    (!a.gate_per_channel || vec(a.gate, BITSMOE_F32, a.gate_stride));
    return v8 ? launch_norm<8>(P, (cudaStream_t)stream) : launch_norm<1>(P, (cudaStream_t)stream);
}
