// q4.cu -- down projections held in 4 bits with group scales: packing and the routed
// matrix-vector products.
//
// The spectral layer leaves an expert's down matrix dense; at one token its fp16 rows
// are half of the FFN's bytes.  Here each group of G columns of a row (G = 32, 64 or
// 128) has the library's mid-rise quantiser at 4 bits:
//   s = fp16(2 max|w| / 15),  q = clamp(floor(w / s + 8), 0, 15),  w ~ s (q - 7.5),
// and the step computes
//   h[t][j] = SiLU(Yg[t][j]) * Yu[t][j]            (or h = Yg when Yu is NULL)
//   out[t][i] = sum_j g[t][j] sum_m w_e[i][m] h[t][j][m],      e = ids[t][j].
//
// Packed layout (bitsmoe.h has it in full): per expert and block of 16 rows, 512-byte
// tiles of 16 x 64 codes in the order in which the lanes of mma.sync m16n8k16 hold
// its A operand, so a lane's 32 codes of a tile are one 16-byte load and no code
// moves between lanes; then the group scales.
//
// Arithmetic: q - 8 is exact in fp16, two codes by one mask and one addition (from the
// bit pattern 0x6400 | q = 1024 + q) or fused multiply-add (0x6400 | 16 q = 1024 + 16 q).
// h is split into an fp16 high part and the fp16 rest after a power-of-two scaling into
// fp16's range; the two are two columns of the B operand, so a product keeps fp32's
// precision.  A group's fp32 sum starts from half the sum of its h, which makes its
// codes q - 7.5, and is multiplied by its scale in fp32.
#include <algorithm>

#include "elem.cuh"

namespace bitsmoe {

constexpr int kQ4Cols = 64;        // columns of a tile
constexpr int kQ4Rows = 16;        // rows of a tile
constexpr int kQ4TileBytes = 512;  // 16 x 64 codes

__host__ __device__ inline int q4_cols_padded(int cols, int group) {
    const int m = group > kQ4Cols ? group : kQ4Cols;
    return (cols + m - 1) / m * m;
}
// Bytes of one block of 16 rows: codes, then scales.
__host__ __device__ inline int64_t q4_block_bytes(int cols_p, int group) {
    return (int64_t)cols_p * 8 + (int64_t)(cols_p / group) * 32;
}
static bool q4_group_ok(int g) { return g == 32 || g == 64 || g == 128; }

// ---------------------------------------------------------------------------
// packing
// ---------------------------------------------------------------------------
struct Q4PackParams {
    const void* w;
    uint8_t* blob;
    int32_t* status;
    int type, rows, cols, cols_p, nblk;
    int64_t supers;  // super-tiles (16 rows x max(64, G) columns) in all
};

// A warp per 16 rows x max(64, G) columns: lane 4a + b holds rows a and a + 8 at
// columns 16t + 2b + {0, 1, 8, 9}, as the packed tile does, so a group's maximum is a
// reduction over four lanes and the codes are written where they were computed.
template <int G>
__global__ void __launch_bounds__(256) k_q4_pack(const Q4PackParams P) {
    constexpr int NT = G > kQ4Cols ? G / kQ4Cols : 1;  // tiles of a super-tile
    constexpr int NG = G < kQ4Cols ? kQ4Cols / G : 1;  // groups of a super-tile
    const int lane = threadIdx.x & 31, a = lane >> 2, b = lane & 3;
    const int64_t st = (int64_t)blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5);
    if (st >= P.supers) return;
    const int per_block = P.cols_p / (NT * kQ4Cols);
    const int64_t blk = st / per_block;  // expert * nblk + block
    const int sc = (int)(st % per_block);
    const int64_t e = blk / P.nblk;
    const int r0 = (int)(blk % P.nblk) * kQ4Rows;
    uint8_t* out = P.blob + blk * q4_block_bytes(P.cols_p, G);
    float v[NT][4][2][2][2];  // [tile][t][u][row half][p]
    int st_bits = 0;
    float amax[NG][2];
    bool fin[NG][2];
#pragma unroll
    for (int g = 0; g < NG; g++) amax[g][0] = amax[g][1] = 0.0f, fin[g][0] = fin[g][1] = true;
#pragma unroll
    for (int n = 0; n < NT; n++)
#pragma unroll
        for (int t = 0; t < 4; t++)
#pragma unroll
            for (int u = 0; u < 2; u++)
#pragma unroll
                for (int h = 0; h < 2; h++)
#pragma unroll
                    for (int p = 0; p < 2; p++) {
                        const int row = r0 + a + 8 * h, col = (sc * NT + n) * kQ4Cols + 16 * t + 8 * u + 2 * b + p;
                        float x[1] = {0.0f};
                        if (row < P.rows && col < P.cols) load_elems<1>(P.w, P.type, (e * P.rows + row) * P.cols + col, x);
                        v[n][t][u][h][p] = x[0];
                        const int g = NG > 1 ? t / (4 / NG) : 0;
                        amax[g][h] = fmaxf(amax[g][h], fabsf(x[0]));
                        fin[g][h] = fin[g][h] && isfinite(x[0]);
                    }
    float s[NG][2];
    uint16_t sh[NG][2];
#pragma unroll
    for (int g = 0; g < NG; g++)
#pragma unroll
        for (int h = 0; h < 2; h++) {
            float m = amax[g][h];
            m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 1));
            m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 2));
            const unsigned bad = __ballot_sync(0xffffffffu, !fin[g][h]);
            __half sc16 = __float2half_rn(__fdiv_rn(2.0f * m, 15.0f));
            if ((bad >> (lane & ~3)) & 0xfu) {  // a non-finite element: the group is stored as zeros
                st_bits |= BITSMOE_ST_NONFINITE;
                sc16 = __ushort_as_half(0);
            } else if (!isfinite(__half2float(sc16))) {
                st_bits |= BITSMOE_ST_BADSCALE;
                sc16 = __ushort_as_half(0);
            }
            sh[g][h] = __half_as_ushort(sc16);
            s[g][h] = __half2float(sc16);
        }
#pragma unroll
    for (int n = 0; n < NT; n++) {
        uint32_t word[4];
#pragma unroll
        for (int t = 0; t < 4; t++) {
            word[t] = 0;
#pragma unroll
            for (int u = 0; u < 2; u++)
#pragma unroll
                for (int h = 0; h < 2; h++)
#pragma unroll
                    for (int p = 0; p < 2; p++) {
                        const int g = NG > 1 ? t / (4 / NG) : 0;
                        const int row = r0 + a + 8 * h, col = (sc * NT + n) * kQ4Cols + 16 * t + 8 * u + 2 * b + p;
                        uint32_t q = 0;
                        if (s[g][h] > 0.0f && row < P.rows && col < P.cols)
                            q = (uint32_t)fminf(
                                fmaxf(floorf(__fadd_rn(__fdiv_rn(v[n][t][u][h][p], s[g][h]), 8.0f)), 0.0f), 15.0f);
                        word[t] |= q << (4 * (4 * p + 2 * u + h));
                    }
        }
        *reinterpret_cast<uint4*>(out + (int64_t)(sc * NT + n) * kQ4TileBytes + 16 * lane) =
            make_uint4(word[0], word[1], word[2], word[3]);
    }
    uint16_t* scales = reinterpret_cast<uint16_t*>(out + (int64_t)P.cols_p * 8);
    if (b < 2) {
#pragma unroll
        for (int g = 0; g < NG; g++) scales[(sc * NG + g) * kQ4Rows + a + 8 * b] = b ? sh[g][1] : sh[g][0];
    }
    if (st_bits && P.status) atomicOr(P.status, st_bits);
}

struct Q4Matrix {
    const uint8_t* blob;
    int rows, cols, cols_p, group, nblk;
};

// fp32 values of the packed matrices (a thread per element).
__global__ void k_q4_unpack(const Q4Matrix M, int64_t n, float* __restrict__ out) {
    for (int64_t x = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; x < n; x += (int64_t)gridDim.x * blockDim.x) {
        const int64_t er = x / M.cols;
        const int col = (int)(x % M.cols), row = (int)(er % M.rows);
        const int64_t blk = er / M.rows * M.nblk + row / kQ4Rows;
        const uint8_t* b = M.blob + blk * q4_block_bytes(M.cols_p, M.group);
        const int lane = row % 8 * 4 + col % 8 / 2;
        const uint32_t word = *reinterpret_cast<const uint32_t*>(b + (int64_t)(col / kQ4Cols) * kQ4TileBytes + 16 * lane +
                                                                 4 * (col % kQ4Cols / 16));
        const int nib = 4 * (col & 1) + 2 * (col % 16 / 8) + row % kQ4Rows / 8;
        const uint16_t s = reinterpret_cast<const uint16_t*>(b + (int64_t)M.cols_p * 8)[col / M.group * kQ4Rows +
                                                                                         row % kQ4Rows];
        out[x] = __half2float(__ushort_as_half(s)) * ((float)((word >> (4 * nib)) & 15u) - 7.5f);
    }
}

// ---------------------------------------------------------------------------
// products
// ---------------------------------------------------------------------------
// Two registers of the A operand of a k step: q - 8 in fp16, exact, of the nibbles at
// bits 0 and 16 and at bits 4 and 20.
__device__ __forceinline__ void q4_pairs(uint32_t w, uint32_t& a0, uint32_t& a1) {
    const uint32_t l = (w & 0x000f000fu) | 0x64006400u, h = (w & 0x00f000f0u) | 0x64006400u;
    const __half2 m1032 = __half2half2(__ushort_as_half(0xe408)), sixteenth = __half2half2(__ushort_as_half(0x2c00)),
                  m72 = __half2half2(__ushort_as_half(0xd480));
    const __half2 lo = __hadd2(*reinterpret_cast<const __half2*>(&l), m1032);
    const __half2 hi = __hfma2(*reinterpret_cast<const __half2*>(&h), sixteenth, m72);
    a0 = *reinterpret_cast<const uint32_t*>(&lo);
    a1 = *reinterpret_cast<const uint32_t*>(&hi);
}

__device__ __forceinline__ void q4_mma(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// The same from c = (start, 0, start, 0).
__device__ __forceinline__ void q4_mma_start(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1, float start) {
    asm(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%11,%10,%11};"
        : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(start), "f"(0.0f));
}

// SiLU(yg) * yu of 8 values (yu NULL: yg itself).
__device__ __forceinline__ void q4_h8(const float* yg, const float* yu, int64_t i, float (&h)[8]) {
    load_elems<8>(yg, BITSMOE_F32, i, h);
    if (!yu) return;
    float u[8];
    load_elems<8>(yu, BITSMOE_F32, i, u);
#pragma unroll
    for (int j = 0; j < 8; j++) h[j] = silu_f(h[j]) * u[j];
}

// Power of two that brings values of magnitude up to m into [2^14, 2^15) (1 for 0 or
// a non-finite m), kept where its reciprocal is finite.
__device__ __forceinline__ float q4_h_scale(float m) {
    return m > 0.0f && m <= 3.0e38f ? ldexpf(1.0f, max(ilogbf(m) - 14, -100)) : 1.0f;
}

// hi + lo = v, both fp16, for two neighbouring values.
__device__ __forceinline__ void q4_split(float v0, float v1, uint32_t& hi, uint32_t& lo) {
    const __half a0 = __float2half_rn(v0), a1 = __float2half_rn(v1);
    const __half b0 = __float2half_rn(v0 - __half2float(a0)), b1 = __float2half_rn(v1 - __half2float(a1));
    hi = (uint32_t)__half_as_ushort(a0) | ((uint32_t)__half_as_ushort(a1) << 16);
    lo = (uint32_t)__half_as_ushort(b0) | ((uint32_t)__half_as_ushort(b1) << 16);
}

// The B operand of a 64-column tile for one column (the high or the low part of a
// row of h): lane column c reads words [c][t][u] (u = 0: k = 16t + 2c + {0, 1}, u = 1:
// 8 more), 32 bytes.  Word of the pair of columns (k, k + 1), k even, inside the tile:
__host__ __device__ constexpr int q4_b_word(int k) { return (k % 8) / 2 * 8 + k / 16 * 2 + k % 16 / 8; }

struct Q4Params {
    Q4Matrix M;
    const float* yg;     // [pairs][cols]
    const float* yu;     // or NULL
    const int32_t* ids;  // [pairs]
    const float* gw;     // [pairs]
    float* out;          // [T][rows]
    int32_t* status;
    int32_t* order;      // [pairs] grouped by expert
    int4* pieces;        // [slots] expert (-1: none), first place in order, pairs
    uint32_t* hb;        // [pairs][cols_p / 64][2][32] B operands (high part, low part)
    float* hsum;         // [pairs][cols_p / G] half the sums of h / hscale over the groups
    float* hscale;       // [pairs]
    float* y;            // [pairs][rows]
    int E, K, T, pairs, slots;
    int tok;             // pairs per piece
    int ksplit;          // warps that share row blocks along the columns
};

// 16 weight bytes of a lane, read once.
__device__ __forceinline__ uint4 q4_ld(const uint8_t* p) {
    uint4 v;
    asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "l"(p));
    return v;
}

// U consecutive tiles of RB row blocks in one lane's registers: codes, and the scales of
// rows g and g + 8 (of both groups of a tile when G = 32).  codes[r]: this lane's 16
// bytes of the first tile of row block r; scales[r]: its rows' scales of that tile's group.
template <int G, int RB, int U>
struct Q4Tiles {
    static constexpr int NS = G < kQ4Cols ? kQ4Cols / G : 1;
    uint4 w[U][RB];
    uint16_t s[U][RB][NS][2];

    __device__ __forceinline__ void load(const uint8_t* const (&codes)[RB], const uint16_t* const (&scales)[RB]) {
#pragma unroll
        for (int u = 0; u < U; u++)
#pragma unroll
            for (int r = 0; r < RB; r++) {
                w[u][r] = q4_ld(codes[r] + u * kQ4TileBytes);
#pragma unroll
                for (int n = 0; n < NS; n++) {
                    const uint16_t* sc = scales[r] + (G > kQ4Cols ? u / (G / kQ4Cols) : u * NS + n) * kQ4Rows;
                    s[u][r][n][0] = __ldg(sc);
                    s[u][r][n][1] = __ldg(sc + 8);
                }
            }
    }
};
// Moves tile pointers on by n tiles (a multiple of 2 when a group is two tiles).
template <int G, int RB>
__device__ __forceinline__ void q4_advance(const uint8_t* (&codes)[RB], const uint16_t* (&scales)[RB], int n) {
#pragma unroll
    for (int r = 0; r < RB; r++) {
        codes[r] += n * kQ4TileBytes;
        scales[r] += n * kQ4Cols / G * kQ4Rows;
    }
}

// One tile times its B operands (NB of the NL column groups that acc has), added to the
// row block's sums.  start: half the sum of h over each group that begins here, for the
// pair of this lane's accumulator columns.  With G = 128 a group is two tiles: `part`
// carries its sum from the first (half = 0) to the second, where its scale is applied.
template <int G, int NB, int NL>
__device__ __forceinline__ void q4_tile(const uint4 w, const uint16_t (*s)[2], const uint32_t (&bw)[NL][8],
                                        const float (*start)[NL], int half, float (&part)[NL][4], float (&acc)[NL][4]) {
    const uint32_t word[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int t = 0; t < 4; t++) {
        uint32_t a[4];
        q4_pairs(word[t], a[0], a[1]);
        q4_pairs(word[t] >> 8, a[2], a[3]);
        const bool begins = G <= 32 ? (t & 1) == 0 : t == 0;
#pragma unroll
        for (int j = 0; j < NB; j++) {
            if (begins && (G <= kQ4Cols || half == 0))
                q4_mma_start(part[j], a, bw[j][2 * t], bw[j][2 * t + 1], start[G <= 32 ? t >> 1 : 0][j]);
            else
                q4_mma(part[j], a, bw[j][2 * t], bw[j][2 * t + 1]);
        }
        const bool ends = G <= 32 ? (t & 1) : t == 3;
        if (ends && (G <= kQ4Cols || half == 1)) {
            const int n = G <= 32 ? t >> 1 : 0;
            const float s0 = __half2float(__ushort_as_half(s[n][0])), s1 = __half2float(__ushort_as_half(s[n][1]));
#pragma unroll
            for (int j = 0; j < NB; j++) {
                acc[j][0] = fmaf(s0, part[j][0], acc[j][0]);
                acc[j][1] = fmaf(s0, part[j][1], acc[j][1]);
                acc[j][2] = fmaf(s1, part[j][2], acc[j][2]);
                acc[j][3] = fmaf(s1, part[j][3], acc[j][3]);
            }
        }
    }
}

// Half the sum of a group's h from the group's chunks of 8 columns, one per lane, in
// neighbouring lanes: returned in every one of them.
template <int G>
__device__ __forceinline__ float q4_group_half(const uint32_t (&hi)[4], const uint32_t (&lo)[4]) {
    float v = 0.0f;
#pragma unroll
    for (int j = 0; j < 4; j++) {
        const float2 a = __half22float2(*reinterpret_cast<const __half2*>(&hi[j]));
        const float2 b = __half22float2(*reinterpret_cast<const __half2*>(&lo[j]));
        v += (a.x + b.x) + (a.y + b.y);
    }
#pragma unroll
    for (int o = 1; o < G / 8; o <<= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return 0.5f * v;
}

// ---------------------------------------------------------------------------
// one token
// ---------------------------------------------------------------------------
// One launch.  A CTA owns blocks of 16 output rows for every slot, so the sum over the
// slots, in order, stays inside it; its 16 warps are the slots x ranges of columns.
// Each warp forms the B operands of its own range of its slot's h in shared memory --
// scaled by the range's own power of two -- while its first weights are on their way.
// Before the programmatic-launch wait the CTA asks L2 for its rows of the experts that
// the ids name at that moment (a prefetch alone: nothing read there is used, and the
// loads after the wait go by the ids as they are then).
constexpr int kQ4T1Warps = 16;
constexpr size_t kQ4T1Smem = 200 * 1024;

// U tiles of one row block times h; sums: of the first tile's group.
template <int G, int U>
__device__ __forceinline__ void q4_t1_batch(const Q4Tiles<G, 1, U>& tiles, const uint32_t* hb, const float* sums, int g,
                                            int c, float (&part)[1][4], float (&acc)[1][4]) {
#pragma unroll
    for (int u = 0; u < U; u++) {
        uint32_t bw[1][8] = {};
        if (g < 2) {  // column 0: the high part, column 1: the rest; the others are zero
            const uint4* src = reinterpret_cast<const uint4*>(hb + u * 64 + 32 * g + 8 * c);
            const uint4 lo = src[0], hi = src[1];
            bw[0][0] = lo.x; bw[0][1] = lo.y; bw[0][2] = lo.z; bw[0][3] = lo.w;
            bw[0][4] = hi.x; bw[0][5] = hi.y; bw[0][6] = hi.z; bw[0][7] = hi.w;
        }
        constexpr int NS = Q4Tiles<G, 1, U>::NS;
        float start[NS][1];
#pragma unroll
        for (int n = 0; n < NS; n++) start[n][0] = c == 0 ? sums[u * kQ4Cols / G + n] : 0.0f;
        q4_tile<G, 1, 1>(tiles.w[u][0], tiles.s[u][0], bw, start, u & 1, part, acc);
    }
}

template <int G>
__global__ void __launch_bounds__(32 * kQ4T1Warps) k_q4_t1(const Q4Params P) {
    constexpr int U = 6, V = G > kQ4Cols ? 2 : 1;  // tiles per batch, and per step of what is left
    extern __shared__ __align__(16) uint32_t s_h[];  // [K][tiles][2][32], then [K][groups], [row blocks][unit][16], ids, weights
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, c = lane & 3;
    const int ntiles = P.M.cols_p / kQ4Cols, nblk = P.M.nblk;
    const int nrb = (nblk - (int)blockIdx.x + (int)gridDim.x - 1) / (int)gridDim.x;  // row blocks blockIdx + i gridDim
    const int ngroups = P.M.cols_p / G;
    float* s_sum = reinterpret_cast<float*>(s_h + (size_t)P.K * P.M.cols_p);
    float* s_part = s_sum + P.K * ngroups;
    int* s_e = reinterpret_cast<int*>(s_part + (size_t)nrb * P.K * P.ksplit * kQ4Rows);
    float* s_g = reinterpret_cast<float*>(s_e + P.K);
    const int64_t bb = q4_block_bytes(P.M.cols_p, G), scale_off = (int64_t)P.M.cols_p * 8;
    for (int v = threadIdx.x; v < P.K * nrb; v += 32 * kQ4T1Warps) {
        const int e = P.ids[v % P.K];
        if (e >= 0 && e < P.E)
            asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(
                             P.M.blob + ((int64_t)e * nblk + blockIdx.x + (int64_t)(v / P.K) * gridDim.x) * bb),
                         "r"((uint32_t)bb)
                         : "memory");
    }
    pdl_wait();
    pdl_trigger();
    if (threadIdx.x < P.K) {
        const int e = P.ids[threadIdx.x];
        const bool ok = e >= 0 && e < P.E;
        s_e[threadIdx.x] = ok ? e : -1;
        s_g[threadIdx.x] = P.gw[threadIdx.x];
        if (!ok && blockIdx.x == 0 && P.status) atomicOr(P.status, BITSMOE_ST_BADEXPERT);
    }
    __syncthreads();
    // units: (slot, range of whole groups)
    constexpr int TG = G > kQ4Cols ? G / kQ4Cols : 1;
    const int per = ((ntiles / TG + P.ksplit - 1) / P.ksplit) * TG;
    for (int unit = warp; unit < P.K * P.ksplit; unit += kQ4T1Warps) {
        const int j = unit / P.ksplit, t0 = min(ntiles, unit % P.ksplit * per), t1 = min(ntiles, t0 + per);
        const int e = s_e[j];
        uint32_t* hb = s_h + ((size_t)j * ntiles) * 64;
        const float* sums = s_sum + j * ngroups;
        float scale = 1.0f;
        Q4Tiles<G, 1, U> tiles;
        const bool batches = t1 - t0 >= U;
        if (e >= 0 && t0 < t1) {
            const uint8_t* base = P.M.blob + ((int64_t)e * nblk + blockIdx.x) * bb;
            const uint8_t* codes[1] = {base + 16 * lane};
            const uint16_t* scales[1] = {reinterpret_cast<const uint16_t*>(base + scale_off) + g};
            q4_advance<G>(codes, scales, t0);
            if (batches) tiles.load(codes, scales);
            const int64_t hrow = (int64_t)j * P.M.cols;
            const int c1 = min(8 * t1, P.M.cols / 8);
            constexpr int KEEP = 2;  // chunks of 8 columns a lane keeps between the two passes
            float kept[KEEP][8];
            float m = 0.0f;
            auto h_of = [&](int ch, float(&h)[8]) {
#pragma unroll
                for (int i = 0; i < 8; i++) h[i] = 0.0f;
                if (ch < c1) q4_h8(P.yg, P.yu, hrow + 8 * ch, h);
            };
#pragma unroll
            for (int k = 0; k < KEEP; k++) h_of(8 * t0 + lane + 32 * k, kept[k]);
#pragma unroll
            for (int k = 0; k < KEEP; k++)
#pragma unroll
                for (int i = 0; i < 8; i++) m = fmaxf(m, fabsf(kept[k][i]));
            for (int ch = 8 * t0 + lane + 32 * KEEP; ch < c1; ch += 32) {
                float h[8];
                h_of(ch, h);
#pragma unroll
                for (int i = 0; i < 8; i++) m = fmaxf(m, fabsf(h[i]));
            }
            scale = q4_h_scale(__uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(m))));
            const float inv = 1.0f / scale;
            // whole warps: a group's chunks sit in neighbouring lanes
            auto put = [&](int ch, const float(&h)[8]) {
                uint32_t hi[4], lo[4];
#pragma unroll
                for (int i = 0; i < 4; i++) q4_split(h[2 * i] * inv, h[2 * i + 1] * inv, hi[i], lo[i]);
                const float sum = q4_group_half<G>(hi, lo);
                if (ch < 8 * t1) {
#pragma unroll
                    for (int i = 0; i < 4; i++) {
                        const int w = q4_b_word(ch % 8 * 8 + 2 * i);
                        hb[(ch / 8) * 64 + w] = hi[i];
                        hb[(ch / 8) * 64 + 32 + w] = lo[i];
                    }
                    if (ch % (G / 8) == 0) s_sum[j * ngroups + ch / (G / 8)] = sum;
                }
            };
#pragma unroll
            for (int k = 0; k < KEEP; k++)
                if (8 * t0 + 32 * k < 8 * t1) put(8 * t0 + lane + 32 * k, kept[k]);
            for (int c0 = 8 * t0 + 32 * KEEP; c0 < 8 * t1; c0 += 32) {
                float h[8];
                h_of(c0 + lane, h);
                put(c0 + lane, h);
            }
            __syncwarp();
        }
        for (int i = 0; i < nrb; i++) {
            float acc[1][4] = {}, part[1][4] = {};
            if (e >= 0 && t0 < t1) {
                const uint8_t* base = P.M.blob + ((int64_t)e * nblk + blockIdx.x + (int64_t)i * gridDim.x) * bb;
                const uint8_t* codes[1] = {base + 16 * lane};
                const uint16_t* scales[1] = {reinterpret_cast<const uint16_t*>(base + scale_off) + g};
                q4_advance<G>(codes, scales, t0);
                int tb = t0;
                for (; tb + U <= t1; tb += U) {
                    if (i > 0 || tb > t0) tiles.load(codes, scales);
                    q4_t1_batch<G, U>(tiles, hb + tb * 64, sums + tb * kQ4Cols / G, g, c, part, acc);
                    q4_advance<G>(codes, scales, U);
                }
                for (; tb < t1; tb += V) {
                    Q4Tiles<G, 1, V> one;
                    one.load(codes, scales);
                    q4_t1_batch<G, V>(one, hb + tb * 64, sums + tb * kQ4Cols / G, g, c, part, acc);
                    q4_advance<G>(codes, scales, V);
                }
            }
            if (c == 0) {
                float* o = s_part + ((size_t)i * P.K * P.ksplit + unit) * kQ4Rows;
                o[g] = (acc[0][0] + acc[0][1]) * scale;
                o[g + 8] = (acc[0][2] + acc[0][3]) * scale;
            }
        }
    }
    __syncthreads();
    for (int v = threadIdx.x; v < nrb * kQ4Rows; v += 32 * kQ4T1Warps) {
        const int i = v / kQ4Rows, r = v % kQ4Rows;
        const int row = ((int)blockIdx.x + i * (int)gridDim.x) * kQ4Rows + r;
        if (row >= P.M.rows) continue;
        float y = 0.0f;
        for (int j = 0; j < P.K; j++) {
            if (s_e[j] < 0) continue;
            float d = 0.0f;
            for (int k = 0; k < P.ksplit; k++) d += s_part[((size_t)i * P.K * P.ksplit + j * P.ksplit + k) * kQ4Rows + r];
            y = fmaf(s_g[j], d, y);
        }
        P.out[row] = y;
    }
}

// ---------------------------------------------------------------------------
// several tokens
// ---------------------------------------------------------------------------
// First launch: the first CTA groups the pairs by expert and cuts the groups into
// pieces of `tok` pairs; every other CTA forms h, its scale and its B operands for one
// pair (independent of the grouping).
constexpr int kQ4PrepThreads = 512;

__device__ void q4_group(const Q4Params& P, int32_t* s_cnt) {
    __shared__ int s_warp[32];
    __shared__ int s_carry[2];
    const int tid = threadIdx.x;
    for (int e = tid; e < P.E; e += kQ4PrepThreads) s_cnt[e] = 0;
    if (tid < 2) s_carry[tid] = 0;
    __syncthreads();
    bool bad = false;
    for (int p = tid; p < P.pairs; p += kQ4PrepThreads) {
        const int e = P.ids[p];
        if (e >= 0 && e < P.E)
            atomicAdd(&s_cnt[e], 1);
        else
            bad = true;
    }
    if (bad && P.status) atomicOr(P.status, BITSMOE_ST_BADEXPERT);
    __syncthreads();
    for (int e0 = 0; e0 < P.E; e0 += kQ4PrepThreads) {
        const int e = e0 + tid, n = e < P.E ? s_cnt[e] : 0, np = (n + P.tok - 1) / P.tok;
        const int end = cta_scan<kQ4PrepThreads>(n, s_warp) + s_carry[0];
        const int pend = cta_scan<kQ4PrepThreads>(np, s_warp) + s_carry[1];
        if (e < P.E) s_cnt[e] = end - n;  // becomes the place of the expert's next pair
        for (int i = 0; i < np; i++)
            P.pieces[pend - np + i] = make_int4(e, end - n + i * P.tok, min(P.tok, n - i * P.tok), 0);
        __syncthreads();
        if (tid == kQ4PrepThreads - 1) {
            s_carry[0] = end;
            s_carry[1] = pend;
        }
        __syncthreads();
    }
    for (int i = s_carry[1] + tid; i < P.slots; i += kQ4PrepThreads) P.pieces[i] = make_int4(-1, 0, 0, 0);
    // a pair's place inside its group may vary; its result does not depend on it
    for (int p = tid; p < P.pairs; p += kQ4PrepThreads) {
        const int e = P.ids[p];
        if (e >= 0 && e < P.E) P.order[atomicAdd(&s_cnt[e], 1)] = p;
    }
}

template <int G>
__global__ void __launch_bounds__(kQ4PrepThreads) k_q4_prep(const Q4Params P) {
    extern __shared__ int32_t s_cnt[];
    __shared__ unsigned s_max;
    const int tid = threadIdx.x;
    pdl_wait();
    pdl_trigger();
    if (blockIdx.x == 0) {
        q4_group(P, s_cnt);
        return;
    }
    const int pair = (int)blockIdx.x - 1, e = P.ids[pair];
    if (e < 0 || e >= P.E) return;  // in no group
    if (tid == 0) s_max = 0u;
    __syncthreads();
    const int64_t base = (int64_t)pair * P.M.cols;
    const int nch = P.M.cols / 8;
    constexpr int KEEP = 2;  // chunks of 8 a thread keeps between the two passes
    float h[KEEP][8];
    float m = 0.0f;
#pragma unroll
    for (int i = 0; i < KEEP; i++) {
        const int c = tid + i * kQ4PrepThreads;
#pragma unroll
        for (int j = 0; j < 8; j++) h[i][j] = 0.0f;
        if (c < nch) q4_h8(P.yg, P.yu, base + 8 * c, h[i]);
#pragma unroll
        for (int j = 0; j < 8; j++) m = fmaxf(m, fabsf(h[i][j]));
    }
    for (int c = tid + KEEP * kQ4PrepThreads; c < nch; c += kQ4PrepThreads) {
        float v[8];
        q4_h8(P.yg, P.yu, base + 8 * c, v);
#pragma unroll
        for (int j = 0; j < 8; j++) m = fmaxf(m, fabsf(v[j]));
    }
    const unsigned wm = __reduce_max_sync(0xffffffffu, __float_as_uint(m));  // non-negative: ordered like their bits
    if ((tid & 31) == 0) atomicMax(&s_max, wm);
    __syncthreads();
    const float scale = q4_h_scale(__uint_as_float(s_max)), inv = 1.0f / scale;
    if (tid == 0) P.hscale[pair] = scale;
    uint32_t* hb = P.hb + (int64_t)pair * P.M.cols_p;
    // whole warps: a group's chunks sit in neighbouring lanes
    auto put = [&](int c, const float(&v)[8]) {
        uint32_t hi[4], lo[4];
#pragma unroll
        for (int j = 0; j < 4; j++) q4_split(v[2 * j] * inv, v[2 * j + 1] * inv, hi[j], lo[j]);
        const float sum = q4_group_half<G>(hi, lo);
        if (c >= P.M.cols_p / 8) return;
        uint32_t* tile = hb + (int64_t)(c / 8) * 64;
#pragma unroll
        for (int j = 0; j < 4; j++) {
            const int w = q4_b_word(c % 8 * 8 + 2 * j);
            tile[w] = hi[j];
            tile[32 + w] = lo[j];
        }
        if (c % (G / 8) == 0) P.hsum[(int64_t)pair * (P.M.cols_p / G) + c / (G / 8)] = sum;
    };
#pragma unroll
    for (int i = 0; i < KEEP; i++)
        if (i * kQ4PrepThreads < P.M.cols_p / 8) put(tid + i * kQ4PrepThreads, h[i]);
    for (int c0 = KEEP * kQ4PrepThreads; c0 < P.M.cols_p / 8; c0 += kQ4PrepThreads) {
        const int c = c0 + tid;
        float v[8] = {};
        if (c < nch) q4_h8(P.yg, P.yu, base + 8 * c, v);
        put(c, v);
    }
}

// Second launch: CTA = (a piece of up to 4 NTL pairs of one expert, (8 / ksplit) RB
// blocks of 16 rows); its 8 warps are row groups x ranges of columns.  A warp's next U
// tiles are loaded while it multiplies the last ones; the B operands come through L1.
// Bound by instructions as much as by HBM: a tile of 512 bytes takes 44 to turn its
// codes into fp16, 4 MMAs per column group and about 12 for loads and scales.
constexpr int kQ4Warps = 8;
constexpr int kQ4Threads = 32 * kQ4Warps;

// U tiles of a warp's row blocks times the first NB of NTL column groups; hb: B operands
// of the first tile, sums: half sums of its group.
template <int G, int NB, int NTL, int RB, int U>
__device__ __forceinline__ void q4_batch(const Q4Tiles<G, RB, U>& tiles, const uint32_t* const (&hb)[NTL],
                                         const float* const (&sums)[NTL], float (&part)[RB][NTL][4],
                                         float (&acc)[RB][NTL][4]) {
    constexpr int NS = Q4Tiles<G, RB, U>::NS;
#pragma unroll
    for (int u = 0; u < U; u++) {
        uint32_t bw[NTL][8];
        float start[NS][NTL];
#pragma unroll
        for (int j = 0; j < NB; j++) {
            const uint4* src = reinterpret_cast<const uint4*>(hb[j] + u * 64);
            const uint4 lo = src[0], hi = src[1];
            bw[j][0] = lo.x; bw[j][1] = lo.y; bw[j][2] = lo.z; bw[j][3] = lo.w;
            bw[j][4] = hi.x; bw[j][5] = hi.y; bw[j][6] = hi.z; bw[j][7] = hi.w;
#pragma unroll
            for (int n = 0; n < NS; n++) start[n][j] = sums[j][u * kQ4Cols / G + n];
        }
#pragma unroll
        for (int r = 0; r < RB; r++)
            q4_tile<G, NB, NTL>(tiles.w[u][r], tiles.s[u][r], bw, start, u & 1, part[r], acc[r]);
    }
}

// n tiles of a warp's row blocks; while one batch of U is multiplied the next is loaded.
template <int G, int NB, int NTL, int RB, int U>
__device__ __forceinline__ void q4_range(const uint8_t* (&codes)[RB], const uint16_t* (&scales)[RB],
                                         const uint32_t* (&hb)[NTL], const float* (&sums)[NTL], int n,
                                         float (&acc)[RB][NTL][4]) {
    constexpr int V = G > kQ4Cols ? 2 : 1;
    float part[RB][NTL][4];
    Q4Tiles<G, RB, U> one, two;
    int left = n / U;
    auto next = [&](Q4Tiles<G, RB, U>& t) {
        t.load(codes, scales);
        q4_advance<G>(codes, scales, U);
    };
    auto use = [&](const Q4Tiles<G, RB, U>& t) {
        q4_batch<G, NB, NTL, RB, U>(t, hb, sums, part, acc);
#pragma unroll
        for (int j = 0; j < NB; j++) {
            hb[j] += U * 64;
            sums[j] += U * kQ4Cols / G;
        }
        left--;
    };
    if (left > 0) next(one);
    while (left > 0) {
        if (left > 1) next(two);
        use(one);
        if (left == 0) break;
        if (left > 1) next(one);
        use(two);
    }
    for (int k = n % U; k > 0; k -= V) {
        Q4Tiles<G, RB, V> t;
        t.load(codes, scales);
        q4_advance<G>(codes, scales, V);
        q4_batch<G, NB, NTL, RB, V>(t, hb, sums, part, acc);
#pragma unroll
        for (int j = 0; j < NB; j++) {
            hb[j] += V * 64;
            sums[j] += V * kQ4Cols / G;
        }
    }
}

template <int G, int NTL, int RB, int U>
__global__ void __launch_bounds__(kQ4Threads, 2) k_q4_mt(const Q4Params P) {
    __shared__ float s_part[kQ4Warps][RB * kQ4Rows][4 * NTL + 1];
    __shared__ int s_pair[4 * NTL];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, c = lane & 3;
    pdl_wait();
    pdl_trigger();
    const int4 piece = P.pieces[blockIdx.y];
    const int e = piece.x, np = piece.z;
    if (e < 0) return;
    const int ntiles = P.M.cols_p / kQ4Cols;
    const int wk = warp % P.ksplit, wr = warp / P.ksplit, nwr = kQ4Warps / P.ksplit;
    constexpr int TG = G > kQ4Cols ? G / kQ4Cols : 1;  // ranges of whole groups
    const int per = ((ntiles / TG + P.ksplit - 1) / P.ksplit) * TG;
    const int t0 = min(ntiles, wk * per), t1 = min(ntiles, t0 + per);
    const int64_t bb = q4_block_bytes(P.M.cols_p, G);
    const int blk0 = (int)blockIdx.x * nwr * RB;
    const uint8_t* codes[RB];
    const uint16_t* scales[RB];
#pragma unroll
    for (int r = 0; r < RB; r++) {
        const uint8_t* base = P.M.blob + ((int64_t)e * P.M.nblk + min(blk0 + wr * RB + r, P.M.nblk - 1)) * bb;
        codes[r] = base + 16 * lane;
        scales[r] = reinterpret_cast<const uint16_t*>(base + (int64_t)P.M.cols_p * 8) + g;
    }
    // this lane's column g of each 8-column B operand: pair g / 2, high part for even g; columns past the last pair
    // repeat it and are not stored
    const uint32_t* hb[NTL];
    const float* sums[NTL];  // of the pair of its accumulator columns 2c (high part) and 2c + 1
#pragma unroll
    for (int j = 0; j < NTL; j++) {
        const int i = min(4 * j + g / 2, np - 1), k = min(4 * j + c, np - 1);
        hb[j] = P.hb + (int64_t)P.order[piece.y + i] * P.M.cols_p + 32 * (g & 1) + 8 * c + t0 * 64;
        sums[j] = P.hsum + (int64_t)P.order[piece.y + k] * (P.M.cols_p / G) + t0 * kQ4Cols / G;
    }
    if (threadIdx.x < np) s_pair[threadIdx.x] = P.order[piece.y + threadIdx.x];
    float acc[RB][NTL][4];
#pragma unroll
    for (int r = 0; r < RB; r++)
#pragma unroll
        for (int j = 0; j < NTL; j++)
#pragma unroll
            for (int q = 0; q < 4; q++) acc[r][j][q] = 0.0f;
    q4_advance<G>(codes, scales, t0);
    if (NTL > 2 && np > 8)
        q4_range<G, NTL, NTL, RB, U>(codes, scales, hb, sums, t1 - t0, acc);
    else if (NTL > 1 && np > 4)
        q4_range<G, NTL < 2 ? 1 : 2, NTL, RB, U>(codes, scales, hb, sums, t1 - t0, acc);
    else
        q4_range<G, 1, NTL, RB, U>(codes, scales, hb, sums, t1 - t0, acc);
    // columns 2c and 2c + 1 of a fragment are the high and the low part of pair c
#pragma unroll
    for (int r = 0; r < RB; r++)
#pragma unroll
        for (int j = 0; j < NTL; j++) {
            s_part[warp][r * kQ4Rows + g][4 * j + c] = acc[r][j][0] + acc[r][j][1];
            s_part[warp][r * kQ4Rows + g + 8][4 * j + c] = acc[r][j][2] + acc[r][j][3];
        }
    __syncthreads();
    const int rows_cta = nwr * RB * kQ4Rows;
    for (int v = threadIdx.x; v < rows_cta * np; v += kQ4Threads) {
        const int r = v % rows_cta, i = v / rows_cta;
        const int row = blk0 * kQ4Rows + r;
        if (row >= P.M.rows) continue;
        float sum = 0.0f;
        for (int k = 0; k < P.ksplit; k++) sum += s_part[r / (RB * kQ4Rows) * P.ksplit + k][r % (RB * kQ4Rows)][i];
        const int pair = s_pair[i];
        P.y[(int64_t)pair * P.M.rows + row] = sum * P.hscale[pair];
    }
}

// Third launch: each token's sum over its slots, in order.
__global__ void __launch_bounds__(256) k_q4_sum(const Q4Params P) {
    pdl_wait();
    pdl_trigger();
    const int64_t n = (int64_t)P.T * P.M.rows;
    for (int64_t x = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; x < n; x += (int64_t)gridDim.x * blockDim.x) {
        const int64_t t = x / P.M.rows;
        const int row = (int)(x % P.M.rows);
        float acc = 0.0f;
        for (int j = 0; j < P.K; j++) {
            const int64_t pair = t * P.K + j;
            const int e = P.ids[pair];
            if (e >= 0 && e < P.E) acc = fmaf(P.gw[pair], P.y[pair * P.M.rows + row], acc);
        }
        P.out[x] = acc;
    }
}

// ---------------------------------------------------------------------------
// host side
// ---------------------------------------------------------------------------
constexpr int kQ4MaxE = 8192;  // the grouping counts them in shared memory (32 KB)

// Pairs per piece: 4, 8 or 16, by the expected group size.
static int q4_tok(int pairs, int E) {
    const int avg = pairs / E;
    return avg <= 3 ? 4 : avg <= 6 ? 8 : 16;
}
static int q4_slots(int pairs, int E) { return std::min(pairs, E) + pairs / q4_tok(pairs, E); }

// The single-token kernel: h and the partial sums of a CTA's row blocks fit its shared memory.
static size_t q4_t1_smem(const bitsmoe_ffn_dims* d, int group, int sms) {
    const int nblk = (d->d_model + kQ4Rows - 1) / kQ4Rows, grid = std::min(nblk, sms), nrb = (nblk + grid - 1) / grid;
    const size_t units = (size_t)d->top_k * std::max(1, kQ4T1Warps / d->top_k);
    const size_t cols_p = q4_cols_padded(d->d_ff, group);
    return 4ull * d->top_k * (cols_p + cols_p / group) + 4ull * nrb * units * kQ4Rows + 8ull * d->top_k;
}
constexpr int kQ4Sms = 148;  // CTAs of the single-token kernel: one per SM
static bool q4_single(const bitsmoe_ffn_dims* d, int group, int T) {
    return T == 1 && d->top_k <= 64 && q4_t1_smem(d, group, kQ4Sms) <= kQ4T1Smem;
}

struct Q4WS {
    int32_t* order;
    int4* pieces;
    uint32_t* hb;
    float* hsum;
    float* hscale;
    float* y;
    uint64_t used;
};

static Q4WS q4_ws(const bitsmoe_ffn_dims* d, int group, int T, uint8_t* base) {
    Q4WS w{};
    uint64_t used = 0;
    auto take = [&](uint64_t bytes) -> void* {
        const uint64_t off = roundup(used, 256);
        used = off + bytes;
        return base ? base + off : nullptr;
    };
    const uint64_t pairs = (uint64_t)T * d->top_k, dp = q4_cols_padded(d->d_ff, group);
    w.order = (int32_t*)take(4 * pairs);
    w.pieces = (int4*)take(16ull * q4_slots((int)pairs, d->n_experts));
    w.hb = (uint32_t*)take(4 * pairs * dp);
    w.hsum = (float*)take(4 * pairs * (dp / group));
    w.hscale = (float*)take(4 * pairs);
    w.y = (float*)take(4 * pairs * d->d_model);
    w.used = used;
    return w;
}

static bool q4_dims_ok(const bitsmoe_ffn_dims* d, int group, int T) {
    return d && d->d_model >= 1 && d->d_ff >= 8 && d->d_ff % 8 == 0 && d->n_experts >= 1 && d->n_experts <= kQ4MaxE &&
           d->top_k >= 1 && q4_group_ok(group) && T >= 0 && (int64_t)T * d->top_k <= 0x3fffffff &&
           d->d_ff <= (1 << 30) && d->d_model <= (1 << 30);
}

template <int G>
static int launch_q4_mt(Q4Params& P, cudaStream_t s) {
    // warps along the columns: enough of them to fill the SMs when few row blocks are touched
    const int rb = P.tok == 16 ? 1 : 2;
    const int64_t tasks = (int64_t)std::min(P.pairs, P.E) * ((P.M.nblk + rb - 1) / rb);
    const int64_t want = 148 * 24;
    P.ksplit = tasks >= want ? 1 : 2 * tasks >= want ? 2 : 4 * tasks >= want ? 4 : 8;
    const int per_cta = kQ4Warps / P.ksplit * rb;
    if (P.slots > 65535) return BITSMOE_EINVAL;
    const dim3 grid((unsigned)((P.M.nblk + per_cta - 1) / per_cta), (unsigned)P.slots), block(kQ4Threads);
    if (P.tok == 4) return launch_pdl(k_q4_mt<G, 1, 2, 2>, grid, block, 0, s, P);
    if (P.tok == 8) return launch_pdl(k_q4_mt<G, 2, 2, 2>, grid, block, 0, s, P);
    return launch_pdl(k_q4_mt<G, 4, 1, 4>, grid, block, 0, s, P);
}

template <int G>
static int launch_q4_t1(Q4Params& P, size_t smem, cudaStream_t s) {
    P.ksplit = std::max(1, kQ4T1Warps / P.K);
    const cudaError_t e = cudaFuncSetAttribute(k_q4_t1<G>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kQ4T1Smem);
    if (e != cudaSuccess) return set_cuda_error(e);
    return launch_pdl(k_q4_t1<G>, dim3((unsigned)std::min(P.M.nblk, kQ4Sms)), dim3(32 * kQ4T1Warps), smem, s, P);
}

}  // namespace bitsmoe

using namespace bitsmoe;

static bool q4_shape_ok(int32_t E, int32_t rows, int32_t cols, int32_t group) {
    return E >= 1 && rows >= 1 && cols >= 1 && rows <= (1 << 30) && cols <= (1 << 30) && q4_group_ok(group);
}

BITSMOE_API uint64_t bitsmoe_q4_bytes(int32_t n_experts, int32_t rows, int32_t cols, int32_t group) {
    if (!q4_shape_ok(n_experts, rows, cols, group)) return 0;
    return (uint64_t)n_experts * ((rows + kQ4Rows - 1) / kQ4Rows) * q4_block_bytes(q4_cols_padded(cols, group), group);
}

BITSMOE_API int bitsmoe_q4_pack(const void* W, int32_t w_type, int32_t n_experts, int32_t rows, int32_t cols,
                                int32_t group, void* blob, int32_t* status, void* stream) {
    if (!q4_shape_ok(n_experts, rows, cols, group) || !elem_ok(w_type) || !W || !blob) return BITSMOE_EINVAL;
    if ((uintptr_t)W % elem_bytes(w_type) || (uintptr_t)blob % 16) return BITSMOE_EINVAL;
    Q4PackParams P{};
    P.w = W;
    P.blob = (uint8_t*)blob;
    P.status = status;
    P.type = w_type;
    P.rows = rows;
    P.cols = cols;
    P.cols_p = q4_cols_padded(cols, group);
    P.nblk = (rows + kQ4Rows - 1) / kQ4Rows;
    P.supers = (int64_t)n_experts * P.nblk * (P.cols_p / std::max(group, kQ4Cols));
    const int64_t blocks = (P.supers + 7) / 8;
    if (blocks > 0x7fffffff) return BITSMOE_EINVAL;
    cudaStream_t s = (cudaStream_t)stream;
    if (group == 32)
        k_q4_pack<32><<<(unsigned)blocks, 256, 0, s>>>(P);
    else if (group == 64)
        k_q4_pack<64><<<(unsigned)blocks, 256, 0, s>>>(P);
    else
        k_q4_pack<128><<<(unsigned)blocks, 256, 0, s>>>(P);
    return check_launch();
}

static Q4Matrix q4_matrix(const void* blob, int rows, int cols, int group) {
    Q4Matrix M{};
    M.blob = (const uint8_t*)blob;
    M.rows = rows;
    M.cols = cols;
    M.cols_p = q4_cols_padded(cols, group);
    M.group = group;
    M.nblk = (rows + kQ4Rows - 1) / kQ4Rows;
    return M;
}

BITSMOE_API int bitsmoe_q4_unpack(const void* blob, int32_t n_experts, int32_t rows, int32_t cols, int32_t group,
                                  float* W, void* stream) {
    if (!q4_shape_ok(n_experts, rows, cols, group) || !blob || !W) return BITSMOE_EINVAL;
    if ((uintptr_t)W % 4 || (uintptr_t)blob % 16) return BITSMOE_EINVAL;
    const int64_t n = (int64_t)n_experts * rows * cols;
    const unsigned blocks = (unsigned)std::min<int64_t>((n + 255) / 256, 148 * 16);
    k_q4_unpack<<<blocks, 256, 0, (cudaStream_t)stream>>>(q4_matrix(blob, rows, cols, group), n, W);
    return check_launch();
}

BITSMOE_API uint64_t bitsmoe_ffn_down_q4_workspace_bytes(const bitsmoe_ffn_dims* dims, int32_t group, int32_t T) {
    if (!q4_dims_ok(dims, group, T) || T == 0 || q4_single(dims, group, T)) return 0;
    return q4_ws(dims, group, T, nullptr).used;
}

BITSMOE_API int bitsmoe_ffn_down_q4_launches(const bitsmoe_ffn_dims* dims, int32_t group, int32_t T) {
    if (!q4_dims_ok(dims, group, T)) return BITSMOE_EINVAL;
    return T == 0 ? 0 : q4_single(dims, group, T) ? 1 : 3;
}

BITSMOE_API int bitsmoe_ffn_down_q4(const bitsmoe_q4_args* args, void* stream) {
    if (!args) return BITSMOE_EINVAL;
    const bitsmoe_q4_args& a = *args;
    const bitsmoe_ffn_dims* dims = &a.dims;
    const int group = a.group, T = a.tokens;
    if (!q4_dims_ok(dims, group, T)) return BITSMOE_EINVAL;
    if (T == 0) return BITSMOE_OK;
    if (!a.blob || !a.Y_gate || !a.topk_ids || !a.gate_w || !a.out) return BITSMOE_EINVAL;
    if ((uintptr_t)a.blob % 16 || (uintptr_t)a.Y_gate % 16 || (uintptr_t)a.Y_up % 16 || (uintptr_t)a.out % 4 ||
        (uintptr_t)a.topk_ids % 4 || (uintptr_t)a.gate_w % 4)
        return BITSMOE_EINVAL;
    const uint64_t need = bitsmoe_ffn_down_q4_workspace_bytes(dims, group, T);
    if (need > 0 && (!a.workspace || (uintptr_t)a.workspace % 256)) return BITSMOE_EINVAL;
    if (a.workspace_bytes < need) return BITSMOE_ESIZE;
    cudaStream_t s = (cudaStream_t)stream;
    Q4Params P{};
    P.M = q4_matrix(a.blob, dims->d_model, dims->d_ff, group);
    P.yg = a.Y_gate;
    P.yu = a.Y_up;
    P.ids = a.topk_ids;
    P.gw = a.gate_w;
    P.out = a.out;
    P.status = a.status;
    P.E = dims->n_experts;
    P.K = dims->top_k;
    P.T = T;
    P.pairs = T * dims->top_k;
    if (q4_single(dims, group, T)) {
        const size_t smem = q4_t1_smem(dims, group, kQ4Sms);
        return group == 32 ? launch_q4_t1<32>(P, smem, s) : group == 64 ? launch_q4_t1<64>(P, smem, s) : launch_q4_t1<128>(P, smem, s);
    }
    const Q4WS w = q4_ws(dims, group, T, (uint8_t*)a.workspace);
    P.order = w.order;
    P.pieces = w.pieces;
    P.hb = w.hb;
    P.hsum = w.hsum;
    P.hscale = w.hscale;
    P.y = w.y;
    P.tok = q4_tok(P.pairs, P.E);
    P.slots = q4_slots(P.pairs, P.E);
    const dim3 pgrid((unsigned)P.pairs + 1), pblock(kQ4PrepThreads);
    int rc = group == 32   ? launch_pdl(k_q4_prep<32>, pgrid, pblock, 4ull * P.E, s, P)
             : group == 64 ? launch_pdl(k_q4_prep<64>, pgrid, pblock, 4ull * P.E, s, P)
                           : launch_pdl(k_q4_prep<128>, pgrid, pblock, 4ull * P.E, s, P);
    if (rc) return rc;
    rc = group == 32 ? launch_q4_mt<32>(P, s) : group == 64 ? launch_q4_mt<64>(P, s) : launch_q4_mt<128>(P, s);
    if (rc) return rc;
    const int64_t n = (int64_t)T * dims->d_model;
    return launch_pdl(k_q4_sum, dim3((unsigned)std::min<int64_t>((n + 255) / 256, 148 * 16)), dim3(256), 0, s, P);
}
