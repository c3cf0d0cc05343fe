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
// One pass over memory: a row stays in registers between its loads and its stores, so
// the step is bound by HBM (h and y read once, h' and x written once).  A row belongs to
// a CTA (up to 512 columns to a warp: no CTA barrier); the two sums are reduced in a
// fixed order, so results do not depend on timing.  Rows too wide for registers are read
// once more per sum.
//
// What decides the time is how many rows an SM has under way, and how long each takes
// from its loads to its stores.  So: every load of a phase in straight-line code, with the
// conversions behind them (under a branch per chunk 8,192 rows of 4,096 took 66 us
// instead of 61.5, 4,096 rows of 8,192 107 instead of 53); h kept in 16 bits until it is
// needed, which leaves registers for a fifth row; element widths fixed when the kernel is
// built.  8,192 x 4,096, bf16 h and x, fp32 y, both norms and a gate per channel: 57.5 us in a
// single launch (5.8 TB/s, 90% of a plain copy's rate), 62 (84%) in a loop, where the board's
// power limit holds the SMs near 1.69 GHz.  Slower were two rows a CTA (83 us), loads through
// a ring in shared memory by persistent CTAs (73 to 124, by its depth) and the channel
// vectors held in registers (86 and more): they hold fewer rows, or leave the L1 cache
// too small for the vectors.
#include <algorithm>
#include <type_traits>

#include "elem.cuh"

namespace bitsmoe {

// Threads per row, at most, while it stays in registers, and the CTAs that an SM is to hold then.
constexpr int norm_threads(int v, int nc) { return v == 4 && nc > 2 ? 256 : 512; }
constexpr int norm_ctas(int v, int nc, bool h32) { return v != 4 || nc > 8 ? 1 : nc <= 2 ? 4 : nc == 4 ? 5 : h32 ? 2 : 3; }

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

// Loads and stores of V elements: 4, of a type whose width the kernel is built for, or 1 of any type.
template <int V, bool F32>
__device__ __forceinline__ void norm_load(const void* p, int type, int64_t i, float (&v)[V]) {
    if constexpr (V == 4)
        load4<F32>(p, type, i, v);
    else
        load_elems<V>(p, type, i, v);
}
template <int V, bool F32>
__device__ __forceinline__ void norm_store(void* p, int type, int64_t i, const float (&v)[V]) {
    if constexpr (V == 4)
        store4<F32>(p, type, i, v);
    else
        store_elems<V>(p, type, i, v);
}

// V elements as they are in memory: h waits so for the sum over y.
template <int V, bool F32>
struct NormRaw {
    float v[V];
    __device__ __forceinline__ void load(const void* p, int type, int64_t i) { norm_load<V, F32>(p, type, i, v); }
    __device__ __forceinline__ void get(int, float (&o)[V]) const {
#pragma unroll
        for (int j = 0; j < V; j++) o[j] = v[j];
    }
};
template <>
struct NormRaw<4, false> {
    uint2 w;
    __device__ __forceinline__ void load(const void* p, int, int64_t i) {
        w = *reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(p) + i);
    }
    __device__ __forceinline__ void get(int type, float (&o)[4]) const { unpack4(w, type, o); }
};

// v[j] times the channel vector w's chunk at at[j].
template <int V, int NC>
__device__ __forceinline__ void norm_scale(float (&v)[NC][V], const float* w, const int64_t (&at)[NC]) {
    float f[NC][V];
#pragma unroll
    for (int j = 0; j < NC; j++) norm_load<V, true>(w, BITSMOE_F32, at[j], f[j]);
#pragma unroll
    for (int j = 0; j < NC; j++)
#pragma unroll
        for (int i = 0; i < V; i++) v[j][i] *= f[j][i];
}

// NC chunks of V elements per thread; NC = 0: the row is read again for every sum.  H32, Y32, X32 (V = 4): h, y and x
// are fp32.
template <int V, int NC, bool WARP, bool H32, bool Y32, bool X32>
__global__ void __launch_bounds__(WARP ? 256 : NC > 0 ? norm_threads(V, NC) : 1024, WARP || NC == 0 ? 1 : norm_ctas(V, NC, H32))
    k_norm_residual(const NormParams P) {
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
        // Every load of a phase stands in straight-line code, conversions after them, so that they are in flight
        // together: threads past the row's end read its last chunk and count nothing.
        int64_t at[NC];
        bool in[NC];
#pragma unroll
        for (int j = 0; j < NC; j++) {
            const int c = lane_in_row + j * nthr;
            in[j] = c < nch;
            at[j] = (int64_t)min(c, nch - 1) * V;
        }
        NormRaw<V, H32> h[NC];
        NormRaw<V, Y32> y[NC];
        float hv[NC][V];  // y, then h'
#pragma unroll
        for (int j = 0; j < NC; j++) h[j].load(P.h, P.h_type, h0 + at[j]);
        if (P.y) {
#pragma unroll
            for (int j = 0; j < NC; j++) y[j].load(P.y, P.y_type, y0 + at[j]);
#pragma unroll
            for (int j = 0; j < NC; j++) y[j].get(P.y_type, hv[j]);
            float r = P.alpha;
            if (P.gate && P.gate_i == 0) r *= P.gate[g0];
            if (P.w_post) {
                float ss = 0.0f;
#pragma unroll
                for (int j = 0; j < NC; j++)
#pragma unroll
                    for (int i = 0; i < V; i++) ss = in[j] ? fmaf(hv[j][i], hv[j][i], ss) : ss;
                r *= rsqrtf(fmaf(row_sum<WARP>(ss, s_part[0]), inv_d, P.eps));
                norm_scale<V, NC>(hv, P.w_post, at);
            }
            if (P.gate && P.gate_i) norm_scale<V, NC>(hv, P.gate + g0, at);
#pragma unroll
            for (int j = 0; j < NC; j++) {
                float v[V];
                h[j].get(P.h_type, v);
#pragma unroll
                for (int i = 0; i < V; i++) hv[j][i] = fmaf(r, hv[j][i], v[i]);
            }
        } else {
#pragma unroll
            for (int j = 0; j < NC; j++) h[j].get(P.h_type, hv[j]);
        }
        if (P.h_out) {
#pragma unroll
            for (int j = 0; j < NC; j++)
                if (in[j]) norm_store<V, H32>(P.h_out, P.h_type, ho0 + at[j], hv[j]);
        }
        if (!P.x) return;
        float ss = 0.0f;
#pragma unroll
        for (int j = 0; j < NC; j++)
#pragma unroll
            for (int i = 0; i < V; i++) ss = in[j] ? fmaf(hv[j][i], hv[j][i], ss) : ss;
        const float rx = rsqrtf(fmaf(row_sum<WARP>(ss, s_part[1]), inv_d, P.eps));
        norm_scale<V, NC>(hv, P.w_pre, at);
#pragma unroll
        for (int j = 0; j < NC; j++) {
#pragma unroll
            for (int i = 0; i < V; i++) hv[j][i] *= rx;
            if (in[j]) norm_store<V, X32>(P.x, P.x_type, x0 + at[j], hv[j]);
        }
    } else {
        float ry = 1.0f;
        if (P.y && P.w_post) {
            float ss = 0.0f;
            for (int c = lane_in_row; c < nch; c += nthr) {
                float v[V];
                norm_load<V, Y32>(P.y, P.y_type, y0 + (int64_t)c * V, v);
#pragma unroll
                for (int i = 0; i < V; i++) ss = fmaf(v[i], v[i], ss);
            }
            ry = rsqrtf(fmaf(row_sum<WARP>(ss, s_part[0]), inv_d, P.eps));
        }
        float r = P.alpha;
        if (P.gate && P.gate_i == 0) r *= P.gate[g0];
        auto chunk = [&](int c, float(&hv)[V]) {
            norm_load<V, H32>(P.h, P.h_type, h0 + (int64_t)c * V, hv);
            if (!P.y) return;
            float v[V], w[V];
            norm_load<V, Y32>(P.y, P.y_type, y0 + (int64_t)c * V, v);
            if (P.w_post) {
                norm_load<V, true>(P.w_post, BITSMOE_F32, (int64_t)c * V, w);
#pragma unroll
                for (int i = 0; i < V; i++) v[i] *= ry * w[i];
            }
            if (P.gate && P.gate_i) {
                norm_load<V, true>(P.gate, BITSMOE_F32, g0 + (int64_t)c * V, w);
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
            if (P.h_out) norm_store<V, H32>(P.h_out, P.h_type, ho0 + (int64_t)c * V, v);
            if (P.x) {
                float w[V];
                norm_load<V, true>(P.w_pre, BITSMOE_F32, (int64_t)c * V, w);
#pragma unroll
                for (int i = 0; i < V; i++) v[i] *= rx * w[i];
                norm_store<V, X32>(P.x, P.x_type, x0 + (int64_t)c * V, v);
            }
        }
    }
}

// Rows that start anywhere: groups of 4 elements on their natural boundary all the same, the first of which may begin
// q = 1 to 3 elements before the row and the last end behind it; those two go element by element, and nothing outside
// the row is read or written.  A CTA per row.  Bound by L1 (72% busy): the channel vectors, which start on no boundary
// of these groups, come as single floats.
// (Against one element per load, us: 4,000 rows x 1,999 in bf16 22.4 and 46.5, 868 x 3,251 11.9 and 18.5, 583 x 1,281 4.2
// and 5.1; but 1,000 x 300 3.7 and 3.5, 1 x 3,251 3.7 and 3.5, 8,192 x 20 12.2 and 2.5.)
constexpr int kShiftChunks = 4, kShiftThreads = 256, kShiftMinCols = 1024, kShiftMinRows = 128;

template <bool H32, bool Y32, bool X32>
__global__ void __launch_bounds__(kShiftThreads, 4) k_norm_shift(const NormParams P) {
    constexpr int NC = kShiftChunks;
    __shared__ float s_part[2][32];
    const int64_t t = blockIdx.x;
    const int d = P.d, q = (int)((t * P.h_ld) & 3);  // the same for every operand: their strides agree modulo 4
    const float inv_d = 1.0f / (float)d;
    const int64_t h0 = t * P.h_ld, y0 = t * P.y_ld, ho0 = t * P.ho_ld, x0 = t * P.x_ld, g0 = t * P.gate_t;
    int s[NC], at[NC];  // first element of each group; where it is loaded from: a whole group in any case
    bool full[NC];
#pragma unroll
    for (int j = 0; j < NC; j++) {
        s[j] = 4 * ((int)threadIdx.x + j * (int)blockDim.x) - q;
        full[j] = s[j] >= 0 && s[j] + 4 <= d;
        at[j] = full[j] ? s[j] : (4 - q) & 3;
    }
    pdl_wait();
    pdl_trigger();
    auto inside = [&](int j, int i) { return s[j] + i >= 0 && s[j] + i < d; };
    NormRaw<4, H32> h[NC];
    NormRaw<4, Y32> y[NC];
    float hv[NC][4];
#pragma unroll
    for (int j = 0; j < NC; j++) h[j].load(P.h, P.h_type, h0 + at[j]);
    if (P.y) {
#pragma unroll
        for (int j = 0; j < NC; j++) y[j].load(P.y, P.y_type, y0 + at[j]);
    }
    // the elements of partial groups, and zeros outside the row
    auto take = [&](const void* p, int type, int64_t row, int j, float(&v)[4]) {
        if (full[j]) return;
#pragma unroll
        for (int i = 0; i < 4; i++) {
            float one[1] = {0.0f};
            if (inside(j, i)) load_elems<1>(p, type, row + s[j] + i, one);
            v[i] = one[0];
        }
    };
    auto scale = [&](const float* w) {
        float f[NC][4];
#pragma unroll
        for (int j = 0; j < NC; j++)
#pragma unroll
            for (int i = 0; i < 4; i++) f[j][i] = w[min(max(s[j] + i, 0), d - 1)];
#pragma unroll
        for (int j = 0; j < NC; j++)
#pragma unroll
            for (int i = 0; i < 4; i++) hv[j][i] *= f[j][i];
    };
    if (P.y) {
#pragma unroll
        for (int j = 0; j < NC; j++) {
            y[j].get(P.y_type, hv[j]);
            take(P.y, P.y_type, y0, j, hv[j]);
        }
        float r = P.alpha;
        if (P.gate && P.gate_i == 0) r *= P.gate[g0];
        if (P.w_post) {
            float ss = 0.0f;
#pragma unroll
            for (int j = 0; j < NC; j++)
#pragma unroll
                for (int i = 0; i < 4; i++) ss = fmaf(hv[j][i], hv[j][i], ss);
            r *= rsqrtf(fmaf(row_sum<false>(ss, s_part[0]), inv_d, P.eps));
            scale(P.w_post);
        }
        if (P.gate && P.gate_i) scale(P.gate + g0);
#pragma unroll
        for (int j = 0; j < NC; j++) {
            float v[4];
            h[j].get(P.h_type, v);
            take(P.h, P.h_type, h0, j, v);
#pragma unroll
            for (int i = 0; i < 4; i++) hv[j][i] = full[j] || inside(j, i) ? fmaf(r, hv[j][i], v[i]) : 0.0f;
        }
    } else {
#pragma unroll
        for (int j = 0; j < NC; j++) {
            h[j].get(P.h_type, hv[j]);
            take(P.h, P.h_type, h0, j, hv[j]);
        }
    }
    if (P.h_out) {
#pragma unroll
        for (int j = 0; j < NC; j++) {
            if (full[j]) {
                store4<H32>(P.h_out, P.h_type, ho0 + s[j], hv[j]);
            } else {
#pragma unroll
                for (int i = 0; i < 4; i++) {
                    const float one[1] = {hv[j][i]};
                    if (inside(j, i)) store_elems<1>(P.h_out, P.h_type, ho0 + s[j] + i, one);
                }
            }
        }
    }
    if (!P.x) return;
    float ss = 0.0f;
#pragma unroll
    for (int j = 0; j < NC; j++)
#pragma unroll
        for (int i = 0; i < 4; i++) ss = fmaf(hv[j][i], hv[j][i], ss);
    const float rx = rsqrtf(fmaf(row_sum<false>(ss, s_part[1]), inv_d, P.eps));
    scale(P.w_pre);
#pragma unroll
    for (int j = 0; j < NC; j++) {
#pragma unroll
        for (int i = 0; i < 4; i++) hv[j][i] *= rx;
        if (full[j]) {
            store4<X32>(P.x, P.x_type, x0 + s[j], hv[j]);
        } else {
#pragma unroll
            for (int i = 0; i < 4; i++) {
                const float one[1] = {hv[j][i]};
                if (inside(j, i)) store_elems<1>(P.x, P.x_type, x0 + s[j] + i, one);
            }
        }
    }
}

constexpr int kNormMaxCols = 1 << 30;  // a column's index and a step of 1024 threads behind it are ints
constexpr int kNormWarpRows = 8;  // rows (warps) per CTA when a row belongs to a warp

template <int V, bool H32, bool Y32, bool X32>
static int launch_norm(const NormParams& P, cudaStream_t s) {
    const int nch = P.d / V;
    // A row in one warp up to 512 columns (8,192 rows, one warp each and a CTA each, us: 256 columns 4.1 and 8.9,
    // 512 columns 8.9 and 9.7; of 768 and more a CTA is as fast).
    if (nch <= 32 * (V == 4 ? 4 : 1)) {
        const dim3 rows((unsigned)((P.T + kNormWarpRows - 1) / kNormWarpRows)), block(32 * kNormWarpRows);
        if constexpr (V == 1) return launch_pdl(k_norm_residual<V, 1, true, H32, Y32, X32>, rows, block, 0, s, P);
        if constexpr (V == 4) {
            if (nch <= 64) return launch_pdl(k_norm_residual<V, 2, true, H32, Y32, X32>, rows, block, 0, s, P);
            return launch_pdl(k_norm_residual<V, 4, true, H32, Y32, X32>, rows, block, 0, s, P);
        }
    }
    const dim3 grid((unsigned)P.T);
    auto threads = [&](int nc) { return (unsigned)std::max<int64_t>(32, roundup((nch + nc - 1) / nc, 32)); };
    if constexpr (V == 4) {
        // 512 threads of 8 elements, or 256 of 16 with an SM's 5 rows in place of 4: with h in 16 bits the second is
        // faster for many rows (8,192 x 4,096: 57.5 against 61.5 us; 1,024 rows 10.1 and 10.1; 1 row 2.8 and 2.6).
        if constexpr (!H32)
            if (P.T >= 2048 && P.d >= 1536 && nch <= 4 * norm_threads(V, 4))
                return launch_pdl(k_norm_residual<V, 4, false, H32, Y32, X32>, grid, threads(4), 0, s, P);
        if (nch <= 2 * norm_threads(V, 2))
            return launch_pdl(k_norm_residual<V, 2, false, H32, Y32, X32>, grid, threads(2), 0, s, P);
    } else if (nch <= 4 * norm_threads(V, 4)) {
        return launch_pdl(k_norm_residual<V, 4, false, H32, Y32, X32>, grid, threads(4), 0, s, P);
    }
    if (nch <= 8 * norm_threads(V, 8))
        return launch_pdl(k_norm_residual<V, 8, false, H32, Y32, X32>, grid, threads(8), 0, s, P);
    if (nch <= 16 * norm_threads(V, 16))
        return launch_pdl(k_norm_residual<V, 16, false, H32, Y32, X32>, grid, threads(16), 0, s, P);
    return launch_pdl(k_norm_residual<V, 0, false, H32, Y32, X32>, grid, 1024, 0, s, P);
}

template <bool H32, bool Y32, bool X32>
static int launch_norm_shift(const NormParams& P, cudaStream_t s) {
    const int groups = (P.d + 6) / 4;  // with the partial ones
    const unsigned threads = (unsigned)roundup((groups + kShiftChunks - 1) / kShiftChunks, 32);
    return launch_pdl(k_norm_shift<H32, Y32, X32>, dim3((unsigned)P.T), dim3(threads), 0, s, P);
}

// One of the kernels built for each set of element widths.
template <bool SHIFT>
static int launch_norm4(const NormParams& P, cudaStream_t s) {
    const bool h32 = P.h_type == BITSMOE_F32, y32 = P.y_type == BITSMOE_F32, x32 = P.x_type == BITSMOE_F32;
    auto run = [&](auto h, auto y, auto x) {
        constexpr bool H = decltype(h)::value, Y = decltype(y)::value, X = decltype(x)::value;
        if constexpr (SHIFT) return launch_norm_shift<H, Y, X>(P, s);
        else return launch_norm<4, H, Y, X>(P, s);
    };
    const std::true_type f32;
    const std::false_type f16;
    if (h32) {
        if (y32) return x32 ? run(f32, f32, f32) : run(f32, f32, f16);
        return x32 ? run(f32, f16, f32) : run(f32, f16, f16);
    }
    if (y32) return x32 ? run(f16, f32, f32) : run(f16, f32, f16);
    return x32 ? run(f16, f16, f32) : run(f16, f16, f16);
}

}  // namespace bitsmoe

using namespace bitsmoe;

BITSMOE_API int bitsmoe_norm_residual(const bitsmoe_norm_args* args, void* stream) {
    if (!args) return BITSMOE_EINVAL;
    const bitsmoe_norm_args& a = *args;
    if (a.rows < 0 || a.d < 1 || a.d > kNormMaxCols || !elem_ok(a.h_type) || (a.y && !elem_ok(a.y_type)) || (a.x && !elem_ok(a.x_type)))
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
    const bool vec4 = a.d % 8 == 0 && vec(a.h, a.h_type, a.h_stride) && vec(a.y, a.y_type, a.y_stride) &&
                    vec(a.h_out, a.h_type, a.h_out_stride) && vec(a.x, a.x_type, a.x_stride) &&
                    vec(a.w_post, BITSMOE_F32, 0) && vec(a.w_pre, BITSMOE_F32, 0) &&
                    (!a.gate_per_channel || vec(a.gate, BITSMOE_F32, a.gate_stride));
    if (vec4) return launch_norm4<false>(P, (cudaStream_t)stream);
    auto same = [&](const void* p, int64_t ld) { return !p || ((uintptr_t)p % 16 == 0 && ((ld - a.h_stride) & 3) == 0); };
    const bool shift = a.rows >= kShiftMinRows && a.d >= kShiftMinCols && a.d <= 4 * kShiftChunks * kShiftThreads - 6 &&
                       same(a.h, a.h_stride) && same(a.y, a.y_stride) && same(a.h_out, a.h_out_stride) &&
                       same(a.x, a.x_stride);
    return shift ? launch_norm4<true>(P, (cudaStream_t)stream) : launch_norm<1, false, false, false>(P, (cudaStream_t)stream);
}
