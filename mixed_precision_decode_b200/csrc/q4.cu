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
// Arithmetic: integer products, exact.  h is taken as a 32-bit fixed-point number relative
// to a power of two above the row's largest |h| (an error of 2^-32 of that) and cut into
// four signed digits of 8 bits, which are four columns of the B operand of mma.sync
// m16n8k32 (u8 x s8, 32-bit sums); the codes are its u8 operand after one mask, or a
// shift and a mask, per four of them.  Two digits' sums over a group are one integer,
// which becomes fp32, takes its share of -7.5 sum h, and is multiplied by the group's
// scale.  With fp16 operands (two columns a row of h) the conversion of the codes alone
// took 36 instructions a tile, most of them at half rate, and the step 1.6 times as long.
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
__device__ __forceinline__ void q4_mma(int (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k32.row.col.s32.u8.s8.s32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+r"(c[0]), "+r"(c[1]), "+r"(c[2]), "+r"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void q4_mma_zero(int (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k32.row.col.s32.u8.s8.s32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
        : "=r"(c[0]), "=r"(c[1]), "=r"(c[2]), "=r"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "r"(0));
}

// SiLU(yg) * yu of 8 values, 16-byte aligned (yu NULL: yg itself).
__device__ __forceinline__ void q4_h8(const float* yg, const float* yu, int64_t i, float (&h)[8]) {
    float lo[4], hi[4];
    load4<true>(yg, BITSMOE_F32, i, lo);
    load4<true>(yg, BITSMOE_F32, i + 4, hi);
#pragma unroll
    for (int j = 0; j < 4; j++) {
        h[j] = lo[j];
        h[4 + j] = hi[j];
    }
    if (!yu) return;
    load4<true>(yu, BITSMOE_F32, i, lo);
    load4<true>(yu, BITSMOE_F32, i + 4, hi);
#pragma unroll
    for (int j = 0; j < 8; j++) h[j] = silu_f(h[j]) * (j < 4 ? lo[j] : hi[j - 4]);
}

// The exponent e of a power of two above a row's largest |h| (m): |h| 2^(30 - e) < 2^30.
// (A row below 2^-95 keeps fewer bits: its unit is 2^-125.)
// m holds the bits of the largest |h|, so a NaN counts as larger than all.
__device__ __forceinline__ int q4_exponent(float m) {
    const int e = (int)(__float_as_uint(m) >> 23) - 126;
    return e > 128 ? 0 : max(e, -95);
}
__device__ __forceinline__ float q4_pow2(int e) { return __uint_as_float((uint32_t)(e + 127) << 23); }

// The value of the fixed-point unit 2^(e - 30); a row with a NaN or an infinity gets NaN,
// and so do its results.
__device__ __forceinline__ float q4_unit(float m, int e) { return m <= 3.4028235e38f ? q4_pow2(e - 30) : NAN; }

// 16 neighbouring columns of h as digits: out[d][c] is word c of digit d (0: the most
// significant) of the half step they are, bytes in the order of the codes' bytes -- columns
// 2c, 2c + 8, 2c + 1, 2c + 9; hi, lo: the sums of digits 0 and 1 and of digits 2 and 3 as
// numbers of 16 bits.  v = round(h 2^(30 - e)) = 2^16 hi + lo per column, digits signed: adding
// 128 to a byte and flipping its top bit subtracts it again.
__device__ __forceinline__ void q4_digits(const float (&h)[16], float to_fixed, uint32_t (&out)[4][4], int& hi, int& lo) {
    uint32_t w[16];
    hi = lo = 0;
#pragma unroll
    for (int i = 0; i < 16; i++) {
        const int v = __float2int_rn(h[i] * to_fixed);
        const int top = (v + 0x8080) >> 16;
        hi += top;
        lo += v - (top << 16);
        w[i] = ((uint32_t)v + 0x00808080u) ^ 0x00808080u;
    }
#pragma unroll
    for (int c = 0; c < 4; c++) {  // 4 x 4 bytes transposed
        const uint32_t a = w[2 * c], b = w[2 * c + 8], e = w[2 * c + 1], f = w[2 * c + 9];
        const uint32_t ab0 = __byte_perm(a, b, 0x5140), ab1 = __byte_perm(a, b, 0x7362);
        const uint32_t ef0 = __byte_perm(e, f, 0x5140), ef1 = __byte_perm(e, f, 0x7362);
        out[3][c] = __byte_perm(ab0, ef0, 0x5410);
        out[2][c] = __byte_perm(ab0, ef0, 0x7632);
        out[1][c] = __byte_perm(ab1, ef1, 0x5410);
        out[0][c] = __byte_perm(ab1, ef1, 0x7632);
    }
}
// The sums of hi and lo over a group of G columns, from its chunks of 16 in neighbouring lanes.
template <int G>
__device__ __forceinline__ void q4_group_sums(int& hi, int& lo) {
#pragma unroll
    for (int o = 1; o < G / 16; o <<= 1) {
        hi += __shfl_xor_sync(0xffffffffu, hi, o);
        lo += __shfl_xor_sync(0xffffffffu, lo, o);
    }
}
// The B operand of a tile for one column (a digit of a row of h): word [c][t] at 4 c + t is
// the half step t (16 columns) of lane column c.  A row of h has [tile][digit][16] words.
constexpr int kQ4BTile = 64;  // words of a row per tile
// Where chunk ch (16 columns) of a row puts digit d of lane column c.
__device__ __forceinline__ int q4_b_at(int ch, int d, int c) { return ch / 4 * kQ4BTile + 16 * d + 4 * c + ch % 4; }

struct Q4Params {
    Q4Matrix M;
    const float* yg;     // [pairs][cols]
    const float* yu;     // or NULL
    const int32_t* ids;  // [pairs]
    const float* gw;     // [pairs]
    float* out;          // [T][rows]
    int32_t* status;
    int32_t* runs;       // [grid + 1] first unit of each CTA of the second launch
    int grid;            // its CTAs
    int32_t* pieces;     // [1 + slots][kQ4Rec]: after an unused record, expert, pairs, pair indexes
    uint32_t* hb;        // [pairs][cols_p / 64][4][16] B operands
    float* hsum;         // [pairs][cols_p / G][2]: -7.5 times the groups' sums of hi and of lo
    float* hscale;       // [pairs] value of the fixed-point unit
    float* y;            // [ranges of columns][pairs][rows]
    int E, K, T, pairs, slots;
    int tok;             // pairs per piece
    int ksplit;          // ranges of columns (one token: per slot)
    int kper;            // tiles of a range
};
constexpr int kQ4Rec = 12;   // ints of a piece's record: expert, pairs in it, 2 unused, 8 pair indexes
constexpr int kQ4Slot0 = 4;
// Cost of a unit of a piece with np pairs: unpacking the codes, and 1, 2 or 4 blocks of 2 pairs each.  (As 5 : 7 : 11
// 128 tokens of 128 experts took 65.1 us instead of 64.5, 32 tokens of 8 experts 4096 x 14336 138 instead of 134.)
__host__ __device__ constexpr int q4_cost(int np) { return np <= 2 ? 3 : np <= 4 ? 4 : 7; }

// 16 weight bytes of a lane, read once.
__device__ __forceinline__ uint4 q4_ld(const uint8_t* p) {
    uint4 v;
    asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "l"(p));
    return v;
}

// U consecutive tiles in one lane's registers: codes, and the scales of rows g and g + 8 (of
// both groups of a tile when G = 32).  codes: this lane's 16 bytes of the first tile; scales:
// its rows' scales of that tile's group.
template <int G, int U>
struct Q4Tiles {
    static constexpr int NS = G < kQ4Cols ? kQ4Cols / G : 1;
    uint4 w[U];
    uint16_t s[U][NS][2];

    __device__ __forceinline__ void load(const uint8_t* codes, const uint16_t* scales) {
#pragma unroll
        for (int u = 0; u < U; u++) {
            w[u] = q4_ld(codes + u * kQ4TileBytes);
#pragma unroll
            for (int n = 0; n < NS; n++) {
                const uint16_t* sc = scales + (G > kQ4Cols ? u / (G / kQ4Cols) : u * NS + n) * kQ4Rows;
                s[u][n][0] = __ldg(sc);
                s[u][n][1] = __ldg(sc + 8);
            }
        }
    }
};
// Moves tile pointers on by n tiles (a multiple of 2 when a group is two tiles).
template <int G>
__device__ __forceinline__ void q4_advance(const uint8_t*& codes, const uint16_t*& scales, int n) {
    codes += n * kQ4TileBytes;
    scales += n * kQ4Cols / G * kQ4Rows;
}

// One tile times the B operands of NB blocks of 8 columns (2 rows of h), added to the row
// block's sums acc (rows g and g + 8 of this lane's two digits).  start: the lane's share of
// -7.5 sum h for each group that ends here.  With G = 128 a group is two tiles: `part` carries
// its sums from the first (half = 0) to the second, where it is scaled.
template <int G, int NB, int NL>
__device__ __forceinline__ void q4_tile(const uint4 w, const uint16_t (*s)[2], const uint4 (&bw)[NL],
                                        const float (*start)[NL], int half, int (&part)[NL][4], float (&acc)[NL][2]) {
    const uint32_t word[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int m = 0; m < 2; m++) {  // 32 columns
        uint32_t a[4];
#pragma unroll
        for (int i = 0; i < 2; i++) {
            a[2 * i] = word[2 * m + i] & 0x0f0f0f0fu;             // row g
            a[2 * i + 1] = (word[2 * m + i] >> 4) & 0x0f0f0f0fu;  // row g + 8
        }
        const bool begins = G <= 32 || (m == 0 && (G <= kQ4Cols || half == 0));
        const bool ends = G <= 32 || (m == 1 && (G <= kQ4Cols || half == 1));
        const int n = G <= 32 ? m : 0;
        float s0 = 0.0f, s1 = 0.0f;
        if (ends) {
            s0 = __half2float(__ushort_as_half(s[n][0]));
            s1 = __half2float(__ushort_as_half(s[n][1]));
        }
#pragma unroll
        for (int j = 0; j < NB; j++) {
            const uint32_t b0 = m ? bw[j].z : bw[j].x, b1 = m ? bw[j].w : bw[j].y;
            if (begins)
                q4_mma_zero(part[j], a, b0, b1);
            else
                q4_mma(part[j], a, b0, b1);
            if (ends) {  // at most 128 x 15 x 128 x 257 < 2^26
                acc[j][0] = fmaf(s0, (float)(part[j][0] * 256 + part[j][1]) + start[n][j], acc[j][0]);
                acc[j][1] = fmaf(s1, (float)(part[j][2] * 256 + part[j][3]) + start[n][j], acc[j][1]);
            }
        }
    }
}
// A lane's sums of its two digits, joined with the other two digits' in the neighbouring
// lane: the results of rows g (even lanes) and g + 8 (odd lanes) in fixed-point units.
__device__ __forceinline__ float q4_join(const float (&acc)[2], int lane) {
    const bool odd = lane & 1;
    const float r0 = odd ? acc[0] : acc[0] * 65536.0f, r1 = odd ? acc[1] : acc[1] * 65536.0f;
    const float other = __shfl_xor_sync(0xffffffffu, odd ? r0 : r1, 1);
    return (odd ? r1 : r0) + other;
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
// 8 experts, 2048 x 768, G = 64: 7.0 us, one chain from the ids over h's digits and 12 tiles
// a warp to the joining of the warps; the 6.7 MB alone would take 1.
constexpr int kQ4T1Warps = 16;
constexpr size_t kQ4T1Smem = 200 * 1024;

// U tiles of one row block times h; sums: of the first tile's group.
template <int G, int U>
__device__ __forceinline__ void q4_t1_batch(const Q4Tiles<G, U>& tiles, const uint32_t* hb, const float* sums, int g,
                                            int c, int (&part)[1][4], float (&acc)[1][2]) {
    constexpr int NS = Q4Tiles<G, U>::NS;
#pragma unroll
    for (int u = 0; u < U; u++) {
        uint4 bw[1] = {make_uint4(0, 0, 0, 0)};
        if (g < 4) bw[0] = *reinterpret_cast<const uint4*>(hb + u * kQ4BTile + 16 * g + 4 * c);  // column g: digit g
        float start[NS][1];
#pragma unroll
        for (int n = 0; n < NS; n++) start[n][0] = sums[(u * kQ4Cols / G + n) * 2 + (c & 1)];
        q4_tile<G, 1, 1>(tiles.w[u], tiles.s[u], bw, start, u & 1, part, acc);
    }
}

template <int G>
__global__ void __launch_bounds__(32 * kQ4T1Warps) k_q4_t1(const Q4Params P) {
    // Tiles per batch, and per step of what is left.  (8 slots, 2048 rows, G = 64, batches of 2, 4, 6, 8, us: 512
    // columns 6.40, 6.46, 6.36, 6.37; 768 columns 7.28, 7.20, 7.01, 7.19; 1,024 columns 8.12, 7.71, 7.90, 7.71; 1,408
    // columns 11.9, 11.2, 11.1, 11.0: 6 is within 0.2 us of the best at each.)
    constexpr int U = 6, V = G > kQ4Cols ? 2 : 1;
    extern __shared__ __align__(16) uint32_t s_h[];  // [K][tiles][4][16], then [K][groups][2], [row blocks][unit][16], ids, weights
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, c = lane & 3;
    const int ntiles = P.M.cols_p / kQ4Cols, nblk = P.M.nblk;
    const int nrb = (nblk - (int)blockIdx.x + (int)gridDim.x - 1) / (int)gridDim.x;  // row blocks blockIdx + i gridDim
    const int ngroups = P.M.cols_p / G;
    float* s_sum = reinterpret_cast<float*>(s_h + (size_t)P.K * P.M.cols_p);
    float* s_part = s_sum + 2 * P.K * ngroups;
    int* s_e = reinterpret_cast<int*>(s_part + (size_t)nrb * P.K * P.ksplit * kQ4Rows);
    float* s_g = reinterpret_cast<float*>(s_e + P.K);
    const int64_t bb = q4_block_bytes(P.M.cols_p, G), scale_off = (int64_t)P.M.cols_p * 8;
    for (int v = threadIdx.x; v < P.K * nrb; v += 32 * kQ4T1Warps) {
        const int e = __ldcg(P.ids + v % P.K);  // leaves no line in L1, which the loads after the wait go through
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
        const float* sums = s_sum + j * ngroups * 2;
        float scale = 1.0f;
        Q4Tiles<G, U> tiles;
        const bool batches = t1 - t0 >= U;
        if (e >= 0 && t0 < t1) {
            const uint8_t* base = P.M.blob + ((int64_t)e * nblk + blockIdx.x) * bb;
            const uint8_t* codes = base + 16 * lane;
            const uint16_t* scales = reinterpret_cast<const uint16_t*>(base + scale_off) + g;
            q4_advance<G>(codes, scales, t0);
            if (batches) tiles.load(codes, scales);
            // chunks of 16 columns, one a lane: the whole range in most layers, else the first 32 stay in registers
            const int64_t hrow = (int64_t)j * P.M.cols;
            auto h_of = [&](int ch, float(&h)[16]) {
                float v[8];
#pragma unroll
                for (int q = 0; q < 2; q++) {
                    const bool in = ch < 4 * t1 && 16 * ch + 8 * q < P.M.cols;  // columns are a multiple of 8
                    if (in) q4_h8(P.yg, P.yu, hrow + 16 * ch + 8 * q, v);
#pragma unroll
                    for (int i = 0; i < 8; i++) h[8 * q + i] = in ? v[i] : 0.0f;
                }
            };
            float kept[16];
            unsigned bits = 0u;  // of the absolute values: ordered like the values, NaN above all
            h_of(4 * t0 + lane, kept);
#pragma unroll
            for (int i = 0; i < 16; i++) bits = max(bits, __float_as_uint(fabsf(kept[i])));
            for (int ch = 4 * t0 + lane + 32; ch < 4 * t1; ch += 32) {
                float h[16];
                h_of(ch, h);
#pragma unroll
                for (int i = 0; i < 16; i++) bits = max(bits, __float_as_uint(fabsf(h[i])));
            }
            const float m = __uint_as_float(__reduce_max_sync(0xffffffffu, bits));
            const int ex = q4_exponent(m);
            scale = q4_unit(m, ex);
            const float to_fixed = q4_pow2(30 - ex);
            auto put = [&](int ch, const float(&h)[16]) {
                uint32_t w[4][4];
                int hi, lo;
                q4_digits(h, to_fixed, w, hi, lo);
                q4_group_sums<G>(hi, lo);
                if (ch >= 4 * t1) return;
#pragma unroll
                for (int d = 0; d < 4; d++)
#pragma unroll
                    for (int k = 0; k < 4; k++) hb[q4_b_at(ch, d, k)] = w[d][k];
                if (ch % (G / 16) == 0) {
                    float* sm = s_sum + (j * ngroups + ch / (G / 16)) * 2;
                    sm[0] = -7.5f * (float)hi;
                    sm[1] = -7.5f * (float)lo;
                }
            };
            put(4 * t0 + lane, kept);
            for (int c0 = 4 * t0 + 32; c0 < 4 * t1; c0 += 32) {
                float h[16];
                h_of(c0 + lane, h);
                put(c0 + lane, h);
            }
            __syncwarp();
        }
        for (int i = 0; i < nrb; i++) {
            float acc[1][2] = {};
            int part[1][4];
            if (e >= 0 && t0 < t1) {
                const uint8_t* base = P.M.blob + ((int64_t)e * nblk + blockIdx.x + (int64_t)i * gridDim.x) * bb;
                const uint8_t* codes = base + 16 * lane;
                const uint16_t* scales = reinterpret_cast<const uint16_t*>(base + scale_off) + g;
                q4_advance<G>(codes, scales, t0);
                int tb = t0;
                for (; tb + U <= t1; tb += U) {
                    if (i > 0 || tb > t0) tiles.load(codes, scales);
                    q4_t1_batch<G, U>(tiles, hb + tb * 64, sums + tb * kQ4Cols / G * 2, g, c, part, acc);
                    q4_advance<G>(codes, scales, U);
                }
                for (; tb < t1; tb += V) {
                    Q4Tiles<G, V> one;
                    one.load(codes, scales);
                    q4_t1_batch<G, V>(one, hb + tb * 64, sums + tb * kQ4Cols / G * 2, g, c, part, acc);
                    q4_advance<G>(codes, scales, V);
                }
            }
            const float r = q4_join(acc[0], lane);
            if (c < 2) s_part[((size_t)i * P.K * P.ksplit + unit) * kQ4Rows + g + 8 * c] = r * scale;
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

template <int THREADS>
__device__ void q4_group(const Q4Params& P, int32_t* s_cnt) {
    __shared__ int s_warp[32];
    __shared__ int s_carry, s_cost;
    constexpr int KEEP = 2048 / THREADS;  // pairs whose expert a thread keeps
    const int tid = threadIdx.x;
    int* s_first = s_cnt + P.E;      // the expert's first piece
    int* s_count = s_cnt + 2 * P.E;  // its pairs
    int* s_before = s_cnt + 3 * P.E; // the cost of the pieces before its own
    int mine[KEEP];
#pragma unroll
    for (int i = 0; i < KEEP; i++) {
        const int p = tid + i * THREADS;
        mine[i] = p < P.pairs ? P.ids[p] : -1;
    }
    for (int e = tid; e < P.E; e += THREADS) s_cnt[e] = 0;
    if (tid == 0) s_carry = s_cost = 0;
    __syncthreads();
    bool bad = false;
    auto each = [&](auto&& f) {  // every pair of this thread with its expert, -1 for a bad one
#pragma unroll
        for (int i = 0; i < KEEP; i++)
            if (tid + i * THREADS < P.pairs) f(tid + i * THREADS, mine[i] < P.E ? mine[i] : -1);
        for (int p = tid + KEEP * THREADS; p < P.pairs; p += THREADS) {
            const int e = P.ids[p];
            f(p, e < P.E ? e : -1);
        }
    };
    each([&](int, int e) {
        if (e >= 0)
            atomicAdd(&s_cnt[e], 1);
        else
            bad = true;
    });
    if (bad && P.status) atomicOr(P.status, BITSMOE_ST_BADEXPERT);
    __syncthreads();
    for (int e0 = 0; e0 < P.E; e0 += THREADS) {
        const int e = e0 + tid, n = e < P.E ? s_cnt[e] : 0, np = (n + P.tok - 1) / P.tok;
        const int first = cta_scan<THREADS>(np, s_warp) + s_carry - np;
        if (e < P.E) {
            s_cnt[e] = 0;  // becomes the place of the expert's next pair
            s_first[e] = first;
            s_count[e] = n;
        }
        const int cost = np > 0 ? (np - 1) * q4_cost(P.tok) + q4_cost(n - (np - 1) * P.tok) : 0;
        const int before = cta_scan<THREADS>(cost, s_warp) + s_cost - cost;
        if (e < P.E) s_before[e] = before;
        for (int i = 0; i < np; i++) {
            int32_t* rec = P.pieces + (int64_t)(1 + first + i) * kQ4Rec;
            rec[0] = e;
            rec[1] = min(P.tok, n - i * P.tok);
        }
        __syncthreads();
        if (tid == THREADS - 1) {
            s_carry = first + np;
            s_cost = before + cost;
        }
        __syncthreads();
    }
    // Runs of equal cost: CTA b starts at the first unit at or after its share of the cost
    // (units are numbered over the pieces).
    const int per_piece = P.ksplit * P.M.nblk;
    const int64_t all = (int64_t)s_cost * per_piece;  // cost of all units
    for (int b = tid; b <= P.grid; b += THREADS) {
        int unit = s_carry * per_piece;
        const int64_t at = all / P.grid * b + all % P.grid * b / P.grid;
        if (b < P.grid && s_carry > 0) {
            int lo = 0, hi = P.E;  // the last expert whose pieces start at or before `at`: it has some
            while (hi - lo > 1) {
                const int mid = (lo + hi) >> 1;
                if (s_before[mid] * (int64_t)per_piece <= at)
                    lo = mid;
                else
                    hi = mid;
            }
            const int n = s_count[lo], np = (n + P.tok - 1) / P.tok, full = q4_cost(P.tok);
            const int64_t off = at - s_before[lo] * (int64_t)per_piece;
            const int i = (int)min((int64_t)np - 1, off / ((int64_t)full * per_piece));
            const int cost = q4_cost(min(P.tok, n - i * P.tok));
            unit = (s_first[lo] + i) * per_piece + (int)((off - (int64_t)i * full * per_piece + cost - 1) / cost);
        }
        P.runs[b] = unit;
    }
    // a pair's place inside its group may vary; its result does not depend on it
    each([&](int p, int e) {
        if (e < 0) return;
        const int at = atomicAdd(&s_cnt[e], 1);
        P.pieces[(int64_t)(1 + s_first[e] + at / P.tok) * kQ4Rec + kQ4Slot0 + at % P.tok] = p;
    });
}

template <int G, int THREADS>
__global__ void __launch_bounds__(THREADS) k_q4_prep(const Q4Params P) {
    extern __shared__ int32_t s_cnt[];  // [4 E]: see q4_group
    __shared__ unsigned s_max;
    const int tid = threadIdx.x;
    pdl_wait();
    pdl_trigger();
    if (blockIdx.x == 0) {
        q4_group<THREADS>(P, s_cnt);
        return;
    }
    const int pair = (int)blockIdx.x - 1, e = P.ids[pair];
    if (e < 0 || e >= P.E) return;  // in no group
    if (tid == 0) s_max = 0u;
    __syncthreads();
    const int64_t base = (int64_t)pair * P.M.cols;
    const int nch = P.M.cols_p / 16;  // chunks of 16 columns, one a thread at a time
    auto h_of = [&](int ch, float(&h)[16]) {
        float v[8];
#pragma unroll
        for (int q = 0; q < 2; q++) {
            const bool in = 16 * ch + 8 * q < P.M.cols;  // columns are a multiple of 8
            if (in) q4_h8(P.yg, P.yu, base + 16 * ch + 8 * q, v);
#pragma unroll
            for (int i = 0; i < 8; i++) h[8 * q + i] = in ? v[i] : 0.0f;
        }
    };
    float kept[16];
    unsigned m = 0u;  // of the absolute values' bits: ordered like the values, NaN above all
    h_of(tid, kept);
#pragma unroll
    for (int i = 0; i < 16; i++) m = max(m, __float_as_uint(fabsf(kept[i])));
    for (int ch = tid + THREADS; ch < nch; ch += THREADS) {
        float v[16];
        h_of(ch, v);
#pragma unroll
        for (int i = 0; i < 16; i++) m = max(m, __float_as_uint(fabsf(v[i])));
    }
    m = __reduce_max_sync(0xffffffffu, m);
    if ((tid & 31) == 0) atomicMax(&s_max, m);
    __syncthreads();
    const float largest = __uint_as_float(s_max);
    const int ex = q4_exponent(largest);
    const float to_fixed = q4_pow2(30 - ex);
    if (tid == 0) P.hscale[pair] = q4_unit(largest, ex);
    uint32_t* hb = P.hb + (int64_t)pair * P.M.cols_p;
    auto put = [&](int ch, const float(&v)[16]) {
        uint32_t w[4][4];
        int hi, lo;
        q4_digits(v, to_fixed, w, hi, lo);
        q4_group_sums<G>(hi, lo);
        if (ch >= nch) return;
#pragma unroll
        for (int d = 0; d < 4; d++)
#pragma unroll
            for (int k = 0; k < 4; k++) hb[q4_b_at(ch, d, k)] = w[d][k];
        if (ch % (G / 16) == 0) {
            float* sm = P.hsum + ((int64_t)pair * (P.M.cols_p / G) + ch / (G / 16)) * 2;
            sm[0] = -7.5f * (float)hi;
            sm[1] = -7.5f * (float)lo;
        }
    };
    put(tid, kept);
    for (int c0 = THREADS; c0 < nch; c0 += THREADS) {  // whole warps
        float v[16];
        h_of(c0 + tid, v);
        put(c0 + tid, v);
    }
}

// Second launch: the pieces times their expert's rows.  The work is cut into units of one
// piece, one range of columns and one block of 16 rows, in that order, and every CTA takes
// a contiguous run of them of equal cost for its 8 warps: its units share a piece and a
// range, whose B operands stay in L1.  A warp streams its units' tiles through a ring of
// its own in shared memory, filled by bulk copies of up to 12 tiles, a stage ahead and
// across the borders of units (without the products this reads at HBM's rate).  Results go
// from registers to memory, a row of y per pair and range; no CTA barrier is met.
// 64 tokens, 128 experts, 2048 x 768, top 8: about 32 us of the step's 43 (108 MB); 48% of
// the issue slots are used, most by unpacking and scaling, the MMAs take 11 us.
constexpr int kQ4Warps = 8;
constexpr int kQ4Threads = 32 * kQ4Warps;
// Tiles per stage, at most: two CTAs' rings of two stages fill an SM's shared memory.  (8: 43.2 instead of 42.2 us at 64
// tokens of 128 experts, 2048 x 768, where 12 are a whole row block and one copy; 120 instead of 112 at 256 tokens.)
constexpr int kQ4CT = 12;
constexpr int kQ4StageBytes = kQ4CT * (kQ4TileBytes + 2 * 32);  // their codes, and up to 2 groups' scales each
constexpr int kQ4Stages = 2;

__device__ __forceinline__ void q4_bulk(uint32_t dst, const uint8_t* src, uint32_t bytes, uint32_t bar) {
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
                 "l"(src), "r"(bytes), "r"(bar)
                 : "memory");
}

// A warp's ring.  The producer cursor and the consumer cursor see the same sequence of
// stages; stage q uses slot q mod kQ4Stages.
template <int G>
struct Q4Ring {
    uint8_t* slots;
    uint32_t base, bars;  // shared-memory addresses of the slots and their barriers
    int in_slot, out_slot;
    uint32_t out_phase;

    __device__ __forceinline__ void init(uint8_t* smem, uint64_t* bar, int lane) {
        slots = smem;
        base = (uint32_t)__cvta_generic_to_shared(smem);
        bars = (uint32_t)__cvta_generic_to_shared(bar);
        in_slot = out_slot = 0;
        out_phase = 0;
        if (lane < kQ4Stages) asm volatile("mbarrier.init.shared::cta.b64 [%0], 1;" ::"r"(bars + 8 * lane));
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        __syncwarp();
    }
    // Tiles t .. t + n - 1 of the row block at `block`: codes, then scales; one copy when that is the whole block.
    __device__ __forceinline__ void fill(const Q4Params& P, const uint8_t* block, int t, int n, int lane) {
        const uint32_t slot = base + in_slot * kQ4StageBytes, bar = bars + 8 * in_slot;
        const uint32_t cb = n * kQ4TileBytes, sb = n * (kQ4Cols * 32) / G;
        const bool whole = n * kQ4Cols == P.M.cols_p;
        if (lane == 0) {
            asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(bar), "r"(cb + sb) : "memory");
            q4_bulk(slot, block + (int64_t)t * kQ4TileBytes, whole ? cb + sb : cb, bar);
            if (!whole) q4_bulk(slot + cb, block + (int64_t)P.M.cols_p * 8 + (int64_t)t * (kQ4Cols * 32) / G, sb, bar);
        }
        __syncwarp();
        in_slot = in_slot == kQ4Stages - 1 ? 0 : in_slot + 1;
    }
    __device__ __forceinline__ bool wait() { return warp_wait(bars + 8 * out_slot, out_phase); }
    __device__ __forceinline__ const uint8_t* slot() const { return slots + out_slot * kQ4StageBytes; }
    __device__ __forceinline__ void pop() {  // every lane has read the slot
        __syncwarp();
        if (++out_slot == kQ4Stages) {
            out_slot = 0;
            out_phase ^= 1u;
        }
    }
};

// What a lane holds of one piece: NTL blocks of 2 pairs (8 columns: 4 digits each).
template <int G, int NTL>
struct Q4Piece {
    const uint32_t* hb[NTL];  // B operands of column g: digit g mod 4 of pair g / 4; past the last pair, that one
    const float* sums[NTL];   // -7.5 sum h of the accumulator columns 2c and 2c + 1: 2 digits of pair c / 2

    // pair: out, the pair c / 2 of each block.
    __device__ __forceinline__ void set(const Q4Params& P, const int32_t* rec, int np, int t0, int lane, int (&pair)[NTL]) {
        const int g = lane >> 2, c = lane & 3;
#pragma unroll
        for (int j = 0; j < NTL; j++) {
            const int col = rec[kQ4Slot0 + min(2 * j + g / 4, np - 1)];
            pair[j] = rec[kQ4Slot0 + min(2 * j + c / 2, np - 1)];
            hb[j] = P.hb + (int64_t)col * P.M.cols_p + 16 * (g & 3) + 4 * c + t0 * kQ4BTile;
            sums[j] = P.hsum + ((int64_t)pair[j] * (P.M.cols_p / G) + t0 * kQ4Cols / G) * 2 + (c & 1);
        }
    }
    __device__ __forceinline__ void back(int n) {  // n tiles
#pragma unroll
        for (int j = 0; j < NTL; j++) {
            hb[j] -= n * kQ4BTile;
            sums[j] -= n * kQ4Cols / G * 2;
        }
    }
};

// U tiles of a stage times the first NB of NTL blocks of columns.
template <int G, int NB, int NTL, int U>
__device__ __forceinline__ void q4_tiles(const uint8_t* codes, const uint16_t* scales, Q4Piece<G, NTL>& piece,
                                         int (&part)[NTL][4], float (&acc)[NTL][2]) {
    constexpr int NS = G < kQ4Cols ? kQ4Cols / G : 1;
#pragma unroll
    for (int u = 0; u < U; u++) {
        uint4 bw[NTL];
        float start[NS][NTL];
#pragma unroll
        for (int j = 0; j < NB; j++) {
            bw[j] = *reinterpret_cast<const uint4*>(piece.hb[j] + u * kQ4BTile);
#pragma unroll
            for (int k = 0; k < NS; k++) start[k][j] = piece.sums[j][(u * kQ4Cols / G + k) * 2];
        }
        uint16_t s[NS][2];
#pragma unroll
        for (int k = 0; k < NS; k++) {
            s[k][0] = scales[(G > kQ4Cols ? u / 2 : u * NS + k) * kQ4Rows];
            s[k][1] = scales[(G > kQ4Cols ? u / 2 : u * NS + k) * kQ4Rows + 8];
        }
        const uint4 w = *reinterpret_cast<const uint4*>(codes + u * kQ4TileBytes);
        q4_tile<G, NB, NTL>(w, s, bw, start, u & 1, part, acc);
    }
#pragma unroll
    for (int j = 0; j < NTL; j++) {  // of every block: back() takes them all back
        piece.hb[j] += U * kQ4BTile;
        piece.sums[j] += U * kQ4Cols / G * 2;
    }
}
// The n tiles of a stage (codes, then scales) times the first NB of NTL blocks of columns.
template <int G, int NB, int NTL>
__device__ __forceinline__ void q4_stage(const uint8_t* slot, int n, Q4Piece<G, NTL>& piece, float (&acc)[NTL][2], int lane) {
    constexpr int U = NB > 2 ? 2 : 4, V = G > kQ4Cols ? 2 : 1;
    int part[NTL][4];
    const uint8_t* codes = slot + 16 * lane;
    const uint16_t* scales = reinterpret_cast<const uint16_t*>(slot + n * kQ4TileBytes) + (lane >> 2);
    for (; n >= U; n -= U) {
        q4_tiles<G, NB, NTL, U>(codes, scales, piece, part, acc);
        codes += U * kQ4TileBytes;
        scales += U * kQ4Cols / G * kQ4Rows;
    }
    for (; n > 0; n -= V) {
        q4_tiles<G, NB, NTL, V>(codes, scales, piece, part, acc);
        codes += V * kQ4TileBytes;
        scales += V * kQ4Cols / G * kQ4Rows;
    }
}
template <int G, int NTL>
__device__ __forceinline__ void q4_stage_any(const uint8_t* slot, int n, int np, Q4Piece<G, NTL>& piece,
                                             float (&acc)[NTL][2], int lane) {
    if (NTL > 2 && np > 4)
        q4_stage<G, NTL, NTL>(slot, n, piece, acc, lane);
    else if (np > 2)
        q4_stage<G, 2, NTL>(slot, n, piece, acc, lane);
    else
        q4_stage<G, 1, NTL>(slot, n, piece, acc, lane);
}

template <int G, int NTL>
__global__ void __launch_bounds__(kQ4Threads, 2) k_q4_mt(const Q4Params P) {
    extern __shared__ __align__(128) uint8_t s_ring[];
    __shared__ uint64_t s_bar[kQ4Warps][kQ4Stages];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, c = lane & 3;
    const int ntiles = P.M.cols_p / kQ4Cols, nblk = P.M.nblk;
    const int64_t bb = q4_block_bytes(P.M.cols_p, G);
    Q4Ring<G> ring;
    ring.init(s_ring + warp * (kQ4Stages * kQ4StageBytes), s_bar[warp], lane);
    pdl_wait();
    pdl_trigger();
    // this warp's units: block blk of part (piece, range), every kQ4Warps-th of the CTA's run
    const int* run = P.runs + blockIdx.x;
    const int u0 = run[0] + warp, left0 = (run[1] - u0 + kQ4Warps - 1) / kQ4Warps;
    if (left0 <= 0) return;
    struct Cursor {
        int left, part, blk;
        __device__ __forceinline__ bool next(int nblk) {  // true when the part changes
            left--;
            blk += kQ4Warps;
            const bool moved = blk >= nblk;
            while (blk >= nblk) {
                blk -= nblk;
                part++;
            }
            return moved;
        }
    };
    Cursor in{left0, u0 / nblk, u0 % nblk}, cur = in;
    // producer: the next stage to fill starts at tile pt (below pt1) of unit `in`
    const uint8_t* experts = nullptr;
    int pt = 0, pt1 = 0;
    auto enter = [&]() {  // the part of `in`
        experts = P.M.blob + (int64_t)P.pieces[(int64_t)(1 + in.part / P.ksplit) * kQ4Rec] * nblk * bb;
        pt = in.part % P.ksplit * P.kper;
        pt1 = min(ntiles, pt + P.kper);
    };
    enter();
    auto fill = [&]() {
        if (in.left <= 0) return;
        const int n = min(kQ4CT, pt1 - pt);
        ring.fill(P, experts + in.blk * bb, pt, n, lane);
        pt += n;
        if (pt < pt1) return;
        pt -= min(P.kper, ntiles - in.part % P.ksplit * P.kper);  // back to the range's first tile
        if (in.next(nblk) && in.left > 0) enter();
    };
    for (int i = 0; i < kQ4Stages; i++) fill();
    bool moved = true;
    int np = 0, kp = 0, t0 = 0, t1 = 0;
    Q4Piece<G, NTL> piece;
    float unit[NTL];
    float* y[NTL];
    while (cur.left > 0) {
        if (moved) {
            const int32_t* rec = P.pieces + (int64_t)(1 + cur.part / P.ksplit) * kQ4Rec;
            np = rec[1];
            kp = cur.part % P.ksplit;
            t0 = kp * P.kper;
            t1 = min(ntiles, t0 + P.kper);
            int pair[NTL];
            piece.set(P, rec, np, t0, lane, pair);
#pragma unroll
            for (int j = 0; j < NTL; j++) {
                unit[j] = P.hscale[pair[j]];
                y[j] = 2 * j + c / 2 < np ? P.y + ((int64_t)kp * P.pairs + pair[j]) * P.M.rows + g + 8 * (c & 1) : nullptr;
            }
        }
        float acc[NTL][2] = {};
        for (int t = t0; t < t1; t += kQ4CT) {
            if (!ring.wait()) {
                if (lane == 0 && P.status) atomicOr(P.status, BITSMOE_ST_TIMEOUT);
                for (int i = 1; i < kQ4Stages; i++) {  // the copies still on their way, with the same limit each
                    ring.pop();
                    ring.wait();
                }
                return;
            }
            q4_stage_any<G, NTL>(ring.slot(), min(kQ4CT, t1 - t), np, piece, acc, lane);
            ring.pop();
            fill();
        }
        piece.back(t1 - t0);
        const int row0 = cur.blk * kQ4Rows;
        const bool in_rows = row0 + g + 8 * (c & 1) < P.M.rows;
#pragma unroll
        for (int j = 0; j < NTL; j++) {
            const float r = q4_join(acc[j], lane);
            if (y[j] && in_rows) y[j][row0] = r * unit[j];
        }
        moved = cur.next(nblk);
    }
}

// Third launch: each token's sum over its slots, in order, and over a slot's ranges of columns.
__global__ void __launch_bounds__(256) k_q4_sum(const Q4Params P) {
    pdl_wait();
    pdl_trigger();
    const int64_t n = (int64_t)P.T * P.M.rows, range = (int64_t)P.pairs * P.M.rows;
    for (int64_t x = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; x < n; x += (int64_t)gridDim.x * blockDim.x) {
        const int64_t t = x / P.M.rows;
        const float* y = P.y + t * P.K * P.M.rows + x % P.M.rows;
        float acc = 0.0f;
        for (int j0 = 0; j0 < P.K; j0 += 8) {  // a slot's rows are read whether or not its id is one: they are not used then
            float v[8], w[8];
            int e[8];
#pragma unroll
            for (int j = 0; j < 8; j++) {
                const int k = min(j0 + j, P.K - 1);
                v[j] = y[(int64_t)k * P.M.rows];
                w[j] = P.gw[t * P.K + k];
                e[j] = P.ids[t * P.K + k];
            }
            for (int r = 1; r < P.ksplit; r++)
#pragma unroll
                for (int j = 0; j < 8; j++) v[j] += y[r * range + (int64_t)min(j0 + j, P.K - 1) * P.M.rows];
#pragma unroll
            for (int j = 0; j < 8; j++)
                if (j0 + j < P.K && e[j] >= 0 && e[j] < P.E) acc = fmaf(w[j], v[j], acc);
        }
        P.out[x] = acc;
    }
}

// ---------------------------------------------------------------------------
// host side
// ---------------------------------------------------------------------------
constexpr int kQ4Sms = 148;    // SMs the launches are sized for
constexpr int kQ4MaxE = 2048;  // the grouping keeps 4 numbers of each in shared memory (32 KB)

// Pairs per piece, by the expected group size.  8 at most: the sums of more do not fit the registers.  (Pieces of 4 and
// of 8, us: 128 experts, 2048 x 768, 1 pair each 23.4 and 25.0, 4 pairs 43.1 and 45.1, 8 pairs 69.2 and 69.2;
// 8 experts, 4096 x 4096, 8 pairs each 46.4 and 53.7, 16 pairs 76.0 and 73.1.)
static int q4_tok(int pairs, int E) { return pairs / E <= 8 ? 4 : 8; }
static int q4_slots(int pairs, int E) { return std::min(pairs, E) + pairs / q4_tok(pairs, E); }

// The single-token kernel: h and the partial sums of a CTA's row blocks fit its shared memory.
static size_t q4_t1_smem(const bitsmoe_ffn_dims* d, int group, int sms) {
    const int nblk = (d->d_model + kQ4Rows - 1) / kQ4Rows, grid = std::min(nblk, sms), nrb = (nblk + grid - 1) / grid;
    const size_t units = (size_t)d->top_k * std::max(1, kQ4T1Warps / d->top_k);
    const size_t cols_p = q4_cols_padded(d->d_ff, group);
    return 4ull * d->top_k * (cols_p + 2 * (cols_p / group)) + 4ull * nrb * units * kQ4Rows + 8ull * d->top_k;
}
static bool q4_single(const bitsmoe_ffn_dims* d, int group, int T) {
    return T == 1 && d->top_k <= 64 && q4_t1_smem(d, group, kQ4Sms) <= kQ4T1Smem;
}

struct Q4WS {
    int32_t* runs;
    int32_t* pieces;
    uint32_t* hb;
    float* hsum;
    float* hscale;
    float* y;
    uint64_t used;
};

// Ranges of columns of the grouped form.  Enough for 4 units for each of the 16 resident
// warps of an SM when few row blocks are touched, of 4 tiles or more each, and with
// partial sums (4 bytes per pair, row and further range) that take no more memory than
// the B operands and half a MB.
static void q4_ranges(const bitsmoe_ffn_dims* d, int group, int64_t pairs, int& ksplit, int& kper) {
    const int64_t nblk = (d->d_model + kQ4Rows - 1) / kQ4Rows, ntiles = q4_cols_padded(d->d_ff, group) / kQ4Cols;
    const int64_t units = std::min<int64_t>(pairs, d->n_experts) * nblk;
    int64_t ks = std::max<int64_t>(1, (4 * 16 * kQ4Sms + units - 1) / units);
    ks = std::min(ks, std::max<int64_t>(1, ntiles / 4));
    ks = std::min(ks, 1 + (d->d_ff + (1 << 17) / pairs) / d->d_model);
    kper = (int)roundup((uint64_t)((ntiles + ks - 1) / ks), 2);  // whole groups, also where one is two tiles
    ksplit = (int)((ntiles + kper - 1) / kper);
}

static Q4WS q4_ws(const bitsmoe_ffn_dims* d, int group, int T, uint8_t* base) {
    Q4WS w{};
    uint64_t used = 0;
    auto take = [&](uint64_t bytes) -> void* {
        const uint64_t off = roundup(used, 256);
        used = off + bytes;
        return base ? base + off : nullptr;
    };
    const uint64_t pairs = (uint64_t)T * d->top_k, dp = q4_cols_padded(d->d_ff, group);
    int ksplit, kper;
    q4_ranges(d, group, (int64_t)pairs, ksplit, kper);
    w.runs = (int32_t*)take(4ull * (2 * kQ4Sms + 1));
    w.pieces = (int32_t*)take(4ull * kQ4Rec * (1 + q4_slots((int)pairs, d->n_experts)));
    w.hb = (uint32_t*)take(4 * pairs * dp);
    w.hsum = (float*)take(8 * pairs * (dp / group));
    w.hscale = (float*)take(4 * pairs);
    w.y = (float*)take(4 * pairs * d->d_model * ksplit);
    w.used = used;
    return w;
}

static bool q4_dims_ok(const bitsmoe_ffn_dims* d, int group, int T) {
    return d && d->d_model >= 1 && d->d_ff >= 8 && d->d_ff % 8 == 0 && d->n_experts >= 1 && d->n_experts <= kQ4MaxE &&
           d->top_k >= 1 && q4_group_ok(group) && T >= 0 && (int64_t)T * d->top_k <= 0x3fffffff &&
           d->d_ff <= (1 << 30) && d->d_model <= (1 << 30);
}

// A thread per 16 columns of a pair, in one pass where 1024 threads are enough: 14,336 columns
// took 5 us more with 256.
template <int G>
static int launch_q4_prep(const Q4Params& P, cudaStream_t s) {
    const dim3 grid((unsigned)P.pairs + 1);
    const size_t smem = 16ull * P.E;
    return P.M.cols_p / 16 <= 256 ? launch_pdl(k_q4_prep<G, 256>, grid, dim3(256), smem, s, P)
                                  : launch_pdl(k_q4_prep<G, 1024>, grid, dim3(1024), smem, s, P);
}

template <int G, int NTL>
static int launch_q4_form(Q4Params& P, cudaStream_t s) {
    const int smem = kQ4Warps * kQ4Stages * kQ4StageBytes;
    const cudaError_t e = cudaFuncSetAttribute(k_q4_mt<G, NTL>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return set_cuda_error(e);
    return launch_pdl(k_q4_mt<G, NTL>, dim3((unsigned)P.grid), dim3(kQ4Threads), smem, s, P);
}

template <int G>
static int launch_q4_mt(Q4Params& P, cudaStream_t s) {
    if (P.tok == 4) return launch_q4_form<G, 2>(P, s);
    return launch_q4_form<G, 4>(P, s);
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
    P.runs = w.runs;
    P.pieces = w.pieces;
    P.hb = w.hb;
    P.hsum = w.hsum;
    P.hscale = w.hscale;
    P.y = w.y;
    P.tok = q4_tok(P.pairs, P.E);
    P.slots = q4_slots(P.pairs, P.E);
    q4_ranges(dims, group, P.pairs, P.ksplit, P.kper);
    const int64_t most = (int64_t)P.slots * P.ksplit * P.M.nblk;  // units, at least as many as there are
    if (most > 0x7fffffff) return BITSMOE_EINVAL;
    P.grid = (int)std::min<int64_t>(2 * kQ4Sms, (most + kQ4Warps - 1) / kQ4Warps);
    int rc = group == 32 ? launch_q4_prep<32>(P, s) : group == 64 ? launch_q4_prep<64>(P, s) : launch_q4_prep<128>(P, s);
    if (rc) return rc;
    rc = group == 32 ? launch_q4_mt<32>(P, s) : group == 64 ? launch_q4_mt<64>(P, s) : launch_q4_mt<128>(P, s);
    if (rc) return rc;
    const int64_t n = (int64_t)T * dims->d_model;
    return launch_pdl(k_q4_sum, dim3((unsigned)std::min<int64_t>((n + 255) / 256, 148 * 16)), dim3(256), 0, s, P);
}
