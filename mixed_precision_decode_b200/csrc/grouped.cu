// grouped.cu -- matrix products grouped by expert, with ragged group sizes.
//
// Sorted row i of expert e (offsets[e] <= i < offsets[e+1]) with input row a_i:
//   out_i[n] = sum_k W[e][n][k] a_i[k]
//   out_i[n] = SiLU(sum_k W[e][n][k] a_i[k]) (sum_k W_up[e][n][k] a_i[k])     (gated)
// a_i is row i of A, or row rows[i] / rows_per_a (the token of a routed pair); the
// result goes to row i of out, or to row rows[i].  16-bit operands, fp32 sums, one
// rounding to the output's type.
#include <algorithm>

#include "elem.cuh"

namespace bitsmoe {

struct GmmParams {
    const uint16_t* a;
    const uint16_t* w;
    const uint16_t* w_up;    // or NULL
    const int32_t* offsets;  // [E+1]
    const int32_t* rows;     // [P] or NULL
    void* out;               // [P][N]
    int32_t* status;
    int64_t lda;             // elements between rows of A
    int P, N, D, E, n_a, div, type, out_type, scatter;
};

// The group of expert e, inside [0, P] whatever the offsets hold.
__device__ __forceinline__ void group_range(const GmmParams& P, int e, int& i0, int& i1) {
    const int a = P.offsets[e], b = P.offsets[e + 1];
    i0 = min(max(a, 0), P.P);
    i1 = min(max(b, i0), P.P);
    if ((i0 != a || i1 != b) && P.status) atomicOr(P.status, BITSMOE_ST_BADGROUP);
}

// Input and output row of sorted row i; false (and the status bit) for a bad index.
__device__ __forceinline__ bool row_pair(const GmmParams& P, int i, int64_t& src, int64_t& dst) {
    if (!P.rows) {
        src = dst = i;
        return true;
    }
    const int r = P.rows[i];
    if (r < 0 || r / P.div >= P.n_a || (P.scatter && r >= P.P)) {
        if (P.status) atomicOr(P.status, BITSMOE_ST_BADGROUP);
        return false;
    }
    src = r / P.div;
    dst = P.scatter ? r : i;
    return true;
}

__device__ __forceinline__ float silu_f(float v) { return v / (1.0f + expf(-v)); }

// ---------------------------------------------------------------------------
// few rows per expert
// ---------------------------------------------------------------------------
// Bound by the weights' bytes.  A CTA owns 16 rows of one expert's matrix (of both,
// when gated) and up to 8 NTL of its input rows; its 8 warps take an eighth of K
// each, so that every SM has enough loads in flight when only a few experts are
// touched, and add their fp32 partial tiles in warp order.  The products are
// mma.sync m16n8k16 on operands that go from global memory to registers: a lane
// loads 16 contiguous bytes of weight row g (and g + 8), eight k's that the two MMAs
// of a 32-wide step take as k = 2c, 2c+1, 2c+8, 2c+9; the input rows are loaded with
// the same order of k, so the sum over k is the same and no operand is rearranged.
constexpr int kMvWarps = 8;
constexpr int kMvThreads = 32 * kMvWarps;
constexpr int kMvRows = 16;
constexpr int kMvUnroll = 4;  // 32-wide k steps in flight per warp

__device__ __forceinline__ uint4 ld_stream(const uint16_t* p) {
    uint4 v;
    asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "l"(p));
    return v;
}

template <bool BF16>
__device__ __forceinline__ void mma16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
    if constexpr (BF16)
        asm volatile(
            "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
            : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
            : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
    else
        asm volatile(
            "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
            : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
            : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Expert and first sorted row of work slot `slot`: the experts' groups cut into pieces
// of `tok` rows, in expert order.  Every warp of the CTA calls it; false past the end.
__device__ __forceinline__ bool find_slot(const GmmParams& P, int slot, int tok, int& e_out, int& i0_out, int& n_out) {
    const int lane = threadIdx.x & 31;
    int base = 0;
    for (int e0 = 0; e0 < P.E; e0 += 32) {
        const int e = e0 + lane;
        int i0 = 0, i1 = 0;
        if (e < P.E) group_range(P, e, i0, i1);
        const int n = (i1 - i0 + tok - 1) / tok;
        int inc = n;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int u = __shfl_up_sync(0xffffffffu, inc, o);
            if (lane >= o) inc += u;
        }
        const bool mine = slot >= base + inc - n && slot < base + inc;
        const unsigned who = __ballot_sync(0xffffffffu, mine);
        if (who) {
            const int l = __ffs(who) - 1;
            const int first = i0 + (slot - (base + inc - n)) * tok;
            e_out = e0 + l;
            i0_out = __shfl_sync(0xffffffffu, first, l);
            n_out = min(tok, __shfl_sync(0xffffffffu, i1, l) - i0_out);
            return true;
        }
        base += __shfl_sync(0xffffffffu, inc, 31);
    }
    return false;
}

template <bool BF16, bool GATED, int NTL>
__global__ void __launch_bounds__(kMvThreads) k_gmm_mv(const GmmParams P) {
    constexpr int NW = GATED ? 2 : 1;
    __shared__ float s_part[kMvWarps][NW][kMvRows][8 * NTL + 1];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, c = lane & 3;
    pdl_wait();
    pdl_trigger();
    int e, i0, nt;
    if (!find_slot(P, (int)blockIdx.y, 8 * NTL, e, i0, nt)) return;
    const int n0 = (int)blockIdx.x * kMvRows;

    // this lane's input rows (row g of each group of 8) and weight rows
    const uint16_t* brow[NTL];
#pragma unroll
    for (int j = 0; j < NTL; j++) {
        const int i = 8 * j + g;
        int64_t src = 0, dst;
        const bool ok = i < nt && row_pair(P, i0 + i, src, dst);
        brow[j] = ok ? P.a + src * P.lda : nullptr;
    }
    const uint16_t* wrow[NW][2];
#pragma unroll
    for (int m = 0; m < NW; m++)
#pragma unroll
        for (int r = 0; r < 2; r++) {
            const int n = n0 + g + 8 * r;
            wrow[m][r] = n < P.N ? (m ? P.w_up : P.w) + ((int64_t)e * P.N + n) * P.D : nullptr;
        }
    float acc[NW][NTL][4];
#pragma unroll
    for (int m = 0; m < NW; m++)
#pragma unroll
        for (int j = 0; j < NTL; j++)
#pragma unroll
            for (int q = 0; q < 4; q++) acc[m][j][q] = 0.0f;

    const int steps = (P.D + 31) / 32, per = (steps + kMvWarps - 1) / kMvWarps;
    const int s0 = min(steps, warp * per), s1 = min(steps, s0 + per);
    constexpr int U = NW * NTL > 4 ? 2 : kMvUnroll;
    for (int s = s0; s < s1; s += U) {
        uint4 wv[U][NW][2], bv[U][NTL];
#pragma unroll
        for (int u = 0; u < U; u++) {
            const int k = (s + u) * 32 + 8 * c;  // D is a multiple of 8: a lane's 8 k's are inside or outside together
            const bool in = s + u < s1 && k < P.D;
#pragma unroll
            for (int m = 0; m < NW; m++)
#pragma unroll
                for (int r = 0; r < 2; r++)
                    wv[u][m][r] = in && wrow[m][r] ? ld_stream(wrow[m][r] + k) : make_uint4(0, 0, 0, 0);
#pragma unroll
            for (int j = 0; j < NTL; j++)
                bv[u][j] = in && brow[j] ? *reinterpret_cast<const uint4*>(brow[j] + k) : make_uint4(0, 0, 0, 0);
        }
#pragma unroll
        for (int u = 0; u < U; u++)
#pragma unroll
            for (int m = 0; m < NW; m++)
#pragma unroll
                for (int j = 0; j < NTL; j++) {
                    mma16816<BF16>(acc[m][j], wv[u][m][0].x, wv[u][m][1].x, wv[u][m][0].y, wv[u][m][1].y, bv[u][j].x,
                                   bv[u][j].y);
                    mma16816<BF16>(acc[m][j], wv[u][m][0].z, wv[u][m][1].z, wv[u][m][0].w, wv[u][m][1].w, bv[u][j].z,
                                   bv[u][j].w);
                }
    }
#pragma unroll
    for (int m = 0; m < NW; m++)
#pragma unroll
        for (int j = 0; j < NTL; j++)
#pragma unroll
            for (int q = 0; q < 4; q++)
                s_part[warp][m][g + 8 * (q >> 1)][8 * j + 2 * c + (q & 1)] = acc[m][j][q];
    __syncthreads();
    for (int v = threadIdx.x; v < nt * kMvRows; v += kMvThreads) {
        const int i = v / kMvRows, r = v % kMvRows;
        int64_t src, dst;
        if (n0 + r >= P.N || !row_pair(P, i0 + i, src, dst)) continue;
        float y[NW];
#pragma unroll
        for (int m = 0; m < NW; m++) {
            float sum = 0.0f;
#pragma unroll
            for (int w = 0; w < kMvWarps; w++) sum += s_part[w][m][r][i];
            y[m] = sum;
        }
        const float o[1] = {GATED ? silu_f(y[0]) * y[NW - 1] : y[0]};
        store_elems<1>(P.out, P.out_type, dst * P.N + n0 + r, o);
    }
}

template <bool BF16, bool GATED>
static int launch_gmm_mv(const GmmParams& P, cudaStream_t s) {
    const int avg = P.P / P.E;
    const int ntl = avg <= 6 ? 1 : avg <= 12 ? 2 : 4;  // input rows a CTA takes: 8, 16 or 32
    const int64_t slots = std::min<int64_t>(P.P, P.E) + P.P / (8 * ntl);  // at least the pieces of every group
    const unsigned tiles = (unsigned)((P.N + kMvRows - 1) / kMvRows);
    if (slots > 65535) return BITSMOE_EINVAL;
    const dim3 grid(tiles, (unsigned)slots), block(kMvThreads);
    if (ntl == 1) return launch_pdl(k_gmm_mv<BF16, GATED, 1>, grid, block, 0, s, P);
    if (ntl == 2) return launch_pdl(k_gmm_mv<BF16, GATED, 2>, grid, block, 0, s, P);
    return launch_pdl(k_gmm_mv<BF16, GATED, 4>, grid, block, 0, s, P);
}

}  // namespace bitsmoe

using namespace bitsmoe;

BITSMOE_API int bitsmoe_grouped_matmul(const bitsmoe_gmm_dims* dims, const void* A, int64_t a_stride, const void* W,
                                       const void* W_up, const int32_t* offsets, const int32_t* rows,
                                       int32_t rows_per_a, int32_t scatter, void* out, int32_t* status, void* stream) {
    if (!dims) return BITSMOE_EINVAL;
    const bitsmoe_gmm_dims& d = *dims;
    if (d.n_rows < 0 || d.n_a_rows < 0 || d.n_out < 1 || d.n_in < 8 || d.n_in % 8 || d.n_experts < 1 ||
        d.n_experts > BITSMOE_GMM_MAX_EXPERTS || (d.in_type != BITSMOE_F16 && d.in_type != BITSMOE_BF16) ||
        (d.out_type != BITSMOE_F32 && d.out_type != d.in_type) || rows_per_a < 1 ||
        (int64_t)d.n_experts * d.n_out > 0x7fffffff)
        return BITSMOE_EINVAL;
    if (!rows && (scatter || rows_per_a != 1 || d.n_a_rows < d.n_rows)) return BITSMOE_EINVAL;
    if (d.n_rows == 0) return BITSMOE_OK;
    if (!A || !W || !offsets || !out || a_stride < d.n_in || a_stride % 8) return BITSMOE_EINVAL;
    if ((uintptr_t)A % 16 || (uintptr_t)W % 16 || (uintptr_t)W_up % 16 || (uintptr_t)offsets % 4 || (uintptr_t)rows % 4 ||
        (uintptr_t)out % 4)
        return BITSMOE_EINVAL;
    GmmParams P{};
    P.a = (const uint16_t*)A;
    P.w = (const uint16_t*)W;
    P.w_up = (const uint16_t*)W_up;
    P.offsets = offsets;
    P.rows = rows;
    P.out = out;
    P.status = status;
    P.lda = a_stride;
    P.P = d.n_rows;
    P.N = d.n_out;
    P.D = d.n_in;
    P.E = d.n_experts;
    P.n_a = d.n_a_rows;
    P.div = rows_per_a;
    P.type = d.in_type;
    P.out_type = d.out_type;
    P.scatter = scatter != 0;
    cudaStream_t s = (cudaStream_t)stream;
    if (d.in_type == BITSMOE_BF16) return W_up ? launch_gmm_mv<true, true>(P, s) : launch_gmm_mv<true, false>(P, s);
    return W_up ? launch_gmm_mv<false, true>(P, s) : launch_gmm_mv<false, false>(P, s);
}
