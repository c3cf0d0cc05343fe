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
// Arithmetic: q - 7.5 is exact in fp16 (one mask and one fused multiply-add per two
// codes, from the bit pattern 0x6400 | q << 4 = 1024 + 16 q).  h is split into an
// fp16 high part and the fp16 rest after a power-of-two scaling into fp16's range;
// the two are two columns of the B operand, so a product keeps fp32's precision.
// A group's fp32 sum is multiplied by its scale in fp32.
#include <algorithm>

#include "elem.cuh"

namespace bitsmoe {

int launch_route_ids(const int32_t* ids, int npairs, int E, const RouteWS& rw, int32_t* status, cudaStream_t s);
int launch_combine(const int32_t* ids, const float* gw, float* Ye, float* Ysum, int T, int K, int E, int d_out,
                   cudaStream_t s);

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
// The four registers of the A operand of one k step: q - 7.5 of the word's nibbles in
// fp16, exact: (0x6400 | 16 q) = 1024 + 16 q, times 1/16, minus 71.5.
__device__ __forceinline__ uint32_t q4_pair(uint32_t w) {
    const uint32_t v = (w & 0x00f000f0u) | 0x64006400u;
    const __half2 sixteenth = __half2half2(__ushort_as_half(0x2c00)), bias = __half2half2(__ushort_as_half(0xd478));
    const __half2 r = __hfma2(*reinterpret_cast<const __half2*>(&v), sixteenth, bias);
    return *reinterpret_cast<const uint32_t*>(&r);
}

__device__ __forceinline__ void q4_mma(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// SiLU(yg) * yu of 8 values (yu NULL: yg itself).
__device__ __forceinline__ void q4_h8(const float* yg, const float* yu, int64_t i, float (&h)[8]) {
    load_elems<8>(yg, BITSMOE_F32, i, h);
    if (!yu) return;
    float u[8];
    load_elems<8>(yu, BITSMOE_F32, i, u);
#pragma unroll
    for (int j = 0; j < 8; j++) h[j] = h[j] / (1.0f + expf(-h[j])) * u[j];
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
    RouteWS rw;          // routing groups
    uint32_t* hb;        // [pairs][cols_p / 64][2][32] B operands (high part, low part)
    float* hscale;       // [pairs]
    float* y;            // [pairs][rows]
    int E, pairs;
    int ksplit;          // warps that share a block of 16 rows along the columns
    int chunk;           // blocks of 16 rows per CTA
};

// A warp per pair: h, its scale and its B operands.
constexpr int kQ4hWarps = 8;
__global__ void __launch_bounds__(32 * kQ4hWarps) k_q4_h(const Q4Params P) {
    const int lane = threadIdx.x & 31;
    const int pair = (int)blockIdx.x * kQ4hWarps + ((int)threadIdx.x >> 5);
    pdl_wait();
    pdl_trigger();
    if (pair >= P.pairs) return;
    const int e = P.ids[pair];
    if (e < 0 || e >= P.E) return;  // in no group
    const int64_t base = (int64_t)pair * P.M.cols;
    const int nch = P.M.cols / 8;
    float m = 0.0f;
    for (int c = lane; c < nch; c += 32) {
        float h[8];
        q4_h8(P.yg, P.yu, base + 8 * c, h);
#pragma unroll
        for (int j = 0; j < 8; j++) m = fmaxf(m, fabsf(h[j]));
    }
    m = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(m)));  // non-negative: ordered like their bits
    const float scale = q4_h_scale(m), inv = 1.0f / scale;
    if (lane == 0) P.hscale[pair] = scale;
    uint32_t* hb = P.hb + (int64_t)pair * P.M.cols_p;
    for (int c = lane; c < P.M.cols_p / 8; c += 32) {
        float h[8] = {};
        if (c < nch) q4_h8(P.yg, P.yu, base + 8 * c, h);
        uint32_t* tile = hb + (int64_t)(c / 8) * 64;
#pragma unroll
        for (int j = 0; j < 8; j += 2) {
            uint32_t hi, lo;
            q4_split(h[j] * inv, h[j + 1] * inv, hi, lo);
            const int w = q4_b_word(c % 8 * 8 + j);
            tile[w] = hi;
            tile[32 + w] = lo;
        }
    }
}

constexpr int kQ4Warps = 8;
constexpr int kQ4Threads = 32 * kQ4Warps;

// Grouped pairs: CTA = (a piece of 4 NTL pairs of one expert, `chunk` blocks of 16
// rows).  Its 8 warps are 8 / ksplit row blocks at a time x ksplit ranges of columns.
template <int G, int NTL>
__global__ void __launch_bounds__(kQ4Threads) k_q4_mt(const Q4Params P) {
    constexpr int U = 4;  // tiles in flight per warp
    __shared__ float s_part[kQ4Warps][kQ4Rows][4 * NTL + 1];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, c = lane & 3;
    pdl_wait();
    pdl_trigger();
    // the piece: experts' groups cut into 4 NTL pairs, in expert order
    int e = -1, p0 = 0, np = 0;
    {
        int base = 0;
        const int nact = *P.rw.nactive;
        for (int q0 = 0; q0 < nact && e < 0; q0 += 32) {
            const int q = q0 + lane;
            int s0 = 0, s1 = 0, ex = 0;
            if (q < nact) {
                ex = P.rw.active[q];
                s0 = P.rw.start[ex];
                s1 = P.rw.start[ex + 1];
            }
            const int n = (s1 - s0 + 4 * NTL - 1) / (4 * NTL);
            int inc = n;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int u = __shfl_up_sync(0xffffffffu, inc, o);
                if (lane >= o) inc += u;
            }
            const int k = (int)blockIdx.y - (base + inc - n);
            const unsigned who = __ballot_sync(0xffffffffu, k >= 0 && k < n);
            if (who) {
                const int l = __ffs(who) - 1;
                e = __shfl_sync(0xffffffffu, ex, l);
                p0 = __shfl_sync(0xffffffffu, s0 + k * 4 * NTL, l);
                np = min(4 * NTL, __shfl_sync(0xffffffffu, s1, l) - p0);
            }
            base += __shfl_sync(0xffffffffu, inc, 31);
        }
    }
    if (e < 0) return;
    // this lane's column g of each 8-column B operand: pair g / 2, high part for even g
    const uint32_t* hb[NTL];
#pragma unroll
    for (int j = 0; j < NTL; j++) {
        const int i = 4 * j + g / 2;
        hb[j] = i < np ? P.hb + (int64_t)P.rw.pairs[p0 + i] * P.M.cols_p + 32 * (g & 1) + 8 * c : nullptr;
    }
    const int ntiles = P.M.cols_p / kQ4Cols;
    const int wk = warp % P.ksplit, wr = warp / P.ksplit, nwr = kQ4Warps / P.ksplit;
    // ranges of whole groups: a multiple of 2 tiles when a group spans 2
    constexpr int TG = G > kQ4Cols ? G / kQ4Cols : 1;
    const int per = ((ntiles / TG + P.ksplit - 1) / P.ksplit) * TG;
    const int t0 = min(ntiles, wk * per), t1 = min(ntiles, t0 + per);
    const int64_t bb = q4_block_bytes(P.M.cols_p, G);
    const int rb0 = (int)blockIdx.x * P.chunk, rb1 = min(P.M.nblk, rb0 + P.chunk);
    for (int rb = rb0; rb < rb1; rb += nwr) {
        const int blk = rb + wr;
        float acc[NTL][4];
#pragma unroll
        for (int j = 0; j < NTL; j++)
#pragma unroll
            for (int q = 0; q < 4; q++) acc[j][q] = 0.0f;
        if (blk < rb1) {
            const uint8_t* base = P.M.blob + ((int64_t)e * P.M.nblk + blk) * bb;
            const uint16_t* scales = reinterpret_cast<const uint16_t*>(base + (int64_t)P.M.cols_p * 8);
            float part[NTL][4];
#pragma unroll
            for (int j = 0; j < NTL; j++)
#pragma unroll
                for (int q = 0; q < 4; q++) part[j][q] = 0.0f;
            for (int tb = t0; tb < t1; tb += U) {
                uint4 wv[U];
#pragma unroll
                for (int u = 0; u < U; u++)
                    wv[u] = tb + u < t1 ? *reinterpret_cast<const uint4*>(base + (int64_t)(tb + u) * kQ4TileBytes + 16 * lane)
                                        : make_uint4(0, 0, 0, 0);
#pragma unroll
                for (int u = 0; u < U; u++) {
                    const int tile = tb + u;
                    if (tile >= t1) break;
                    uint32_t bw[NTL][8];
#pragma unroll
                    for (int j = 0; j < NTL; j++) {
                        uint4 lo = make_uint4(0, 0, 0, 0), hi = lo;
                        if (hb[j]) {
                            const uint4* src = reinterpret_cast<const uint4*>(hb[j] + (int64_t)tile * 64);
                            lo = src[0];
                            hi = src[1];
                        }
                        bw[j][0] = lo.x; bw[j][1] = lo.y; bw[j][2] = lo.z; bw[j][3] = lo.w;
                        bw[j][4] = hi.x; bw[j][5] = hi.y; bw[j][6] = hi.z; bw[j][7] = hi.w;
                    }
                    const uint32_t word[4] = {wv[u].x, wv[u].y, wv[u].z, wv[u].w};
#pragma unroll
                    for (int t = 0; t < 4; t++) {
                        const uint32_t a[4] = {q4_pair(word[t] << 4), q4_pair(word[t]), q4_pair(word[t] >> 4),
                                               q4_pair(word[t] >> 8)};
#pragma unroll
                        for (int j = 0; j < NTL; j++) q4_mma(part[j], a, bw[j][2 * t], bw[j][2 * t + 1]);
                        const int col = tile * kQ4Cols + 16 * (t + 1);
                        if (col % G == 0) {  // the group ends here
                            const int gr = col / G - 1;
                            const float s0 = __half2float(__ushort_as_half(scales[gr * kQ4Rows + g]));
                            const float s1 = __half2float(__ushort_as_half(scales[gr * kQ4Rows + g + 8]));
#pragma unroll
                            for (int j = 0; j < NTL; j++) {
                                acc[j][0] = fmaf(s0, part[j][0], acc[j][0]);
                                acc[j][1] = fmaf(s0, part[j][1], acc[j][1]);
                                acc[j][2] = fmaf(s1, part[j][2], acc[j][2]);
                                acc[j][3] = fmaf(s1, part[j][3], acc[j][3]);
                                part[j][0] = part[j][1] = part[j][2] = part[j][3] = 0.0f;
                            }
                        }
                    }
                }
            }
        }
        // columns 2c and 2c + 1 of a fragment are the high and the low part of pair c
#pragma unroll
        for (int j = 0; j < NTL; j++) {
            s_part[warp][g][4 * j + c] = acc[j][0] + acc[j][1];
            s_part[warp][g + 8][4 * j + c] = acc[j][2] + acc[j][3];
        }
        __syncthreads();
        for (int v = threadIdx.x; v < nwr * kQ4Rows * np; v += kQ4Threads) {
            const int r = v % kQ4Rows, i = v / kQ4Rows % np, w = v / (kQ4Rows * np);
            const int row = (rb + w) * kQ4Rows + r;
            if (rb + w < rb1 && row < P.M.rows) {
                float sum = 0.0f;
                for (int k = 0; k < P.ksplit; k++) sum += s_part[w * P.ksplit + k][r][i];
                const int pair = P.rw.pairs[p0 + i];
                P.y[(int64_t)pair * P.M.rows + row] = sum * P.hscale[pair];
            }
        }
        __syncthreads();
    }
}

// ---------------------------------------------------------------------------
// host side
// ---------------------------------------------------------------------------
struct Q4WS {
    RouteWS route;
    uint32_t* hb;
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
    const uint64_t E = d->n_experts, pairs = (uint64_t)T * d->top_k, dp = q4_cols_padded(d->d_ff, group);
    w.route.count = (int32_t*)take(4 * E);
    w.route.start = (int32_t*)take(4 * (E + 1));
    w.route.active = (int32_t*)take(4 * E);
    w.route.nactive = (int32_t*)take(4);
    w.route.pairs = (int32_t*)take(4 * pairs + 4);
    w.hb = (uint32_t*)take(4 * pairs * dp);
    w.hscale = (float*)take(4 * pairs);
    w.y = (float*)take(4 * pairs * d->d_model);
    w.used = used;
    return w;
}

static bool q4_dims_ok(const bitsmoe_ffn_dims* d, int group, int T) {
    return d && d->d_model >= 1 && d->d_ff >= 8 && d->d_ff % 8 == 0 && d->n_experts >= 1 && d->top_k >= 1 &&
           q4_group_ok(group) && T >= 0 && (int64_t)T * d->top_k <= 0x7fffffff && d->d_ff <= (1 << 30) &&
           d->d_model <= (1 << 30);
}

template <int G>
static int launch_q4_mt(const Q4Params& P, int ntl, const dim3& grid, cudaStream_t s) {
    if (ntl == 1) return launch_pdl(k_q4_mt<G, 1>, grid, dim3(kQ4Threads), 0, s, P);
    if (ntl == 2) return launch_pdl(k_q4_mt<G, 2>, grid, dim3(kQ4Threads), 0, s, P);
    return launch_pdl(k_q4_mt<G, 4>, grid, dim3(kQ4Threads), 0, s, P);
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
    if (!q4_dims_ok(dims, group, T) || T == 0) return 0;
    return q4_ws(dims, group, T, nullptr).used;
}

BITSMOE_API int bitsmoe_ffn_down_q4_launches(const bitsmoe_ffn_dims* dims, int32_t group, int32_t T) {
    if (!q4_dims_ok(dims, group, T)) return BITSMOE_EINVAL;
    return T == 0 ? 0 : 4;
}

BITSMOE_API int bitsmoe_ffn_down_q4(const bitsmoe_ffn_dims* dims, const void* blob, int32_t group, const float* Y_gate,
                                    const float* Y_up, const int32_t* topk_ids, const float* gate_w, int32_t T,
                                    float* out, void* workspace, uint64_t workspace_bytes, int32_t* status,
                                    void* stream) {
    if (!q4_dims_ok(dims, group, T)) return BITSMOE_EINVAL;
    if (T == 0) return BITSMOE_OK;
    if (!blob || !Y_gate || !topk_ids || !gate_w || !out) return BITSMOE_EINVAL;
    if ((uintptr_t)blob % 16 || (uintptr_t)Y_gate % 16 || (uintptr_t)Y_up % 16 || (uintptr_t)out % 4 ||
        (uintptr_t)topk_ids % 4 || (uintptr_t)gate_w % 4)
        return BITSMOE_EINVAL;
    const uint64_t need = bitsmoe_ffn_down_q4_workspace_bytes(dims, group, T);
    if (need > 0 && (!workspace || (uintptr_t)workspace % 256)) return BITSMOE_EINVAL;
    if (workspace_bytes < need) return BITSMOE_ESIZE;
    cudaStream_t s = (cudaStream_t)stream;
    const int E = dims->n_experts, K = dims->top_k, pairs = T * K;
    const Q4WS w = q4_ws(dims, group, T, (uint8_t*)workspace);
    Q4Params P{};
    P.M = q4_matrix(blob, dims->d_model, dims->d_ff, group);
    P.yg = Y_gate;
    P.yu = Y_up;
    P.ids = topk_ids;
    P.rw = w.route;
    P.hb = w.hb;
    P.hscale = w.hscale;
    P.y = w.y;
    P.E = E;
    P.pairs = pairs;
    int rc = launch_route_ids(topk_ids, pairs, E, w.route, status, s);
    if (rc) return rc;
    rc = launch_pdl(k_q4_h, dim3((unsigned)((pairs + kQ4hWarps - 1) / kQ4hWarps)), dim3(32 * kQ4hWarps), 0, s, P);
    if (rc) return rc;
    const int avg = pairs / E;
    const int ntl = avg <= 3 ? 1 : avg <= 6 ? 2 : 4;
    const int64_t slots = std::min(pairs, E) + pairs / (4 * ntl);
    // warps along the columns: enough of them to fill the SMs when few row blocks are touched
    const int64_t tasks = (int64_t)std::min<int64_t>(slots, std::min(pairs, E)) * P.M.nblk;
    P.ksplit = tasks >= 148 * 32 ? 1 : tasks >= 148 * 16 ? 2 : tasks >= 148 * 8 ? 4 : 8;
    P.chunk = kQ4Warps;
    if (slots > 65535) return BITSMOE_EINVAL;
    const dim3 grid((unsigned)((P.M.nblk + P.chunk - 1) / P.chunk), (unsigned)slots);
    rc = group == 32 ? launch_q4_mt<32>(P, ntl, grid, s) : group == 64 ? launch_q4_mt<64>(P, ntl, grid, s)
                                                                        : launch_q4_mt<128>(P, ntl, grid, s);
    if (rc) return rc;
    return launch_combine(topk_ids, gate_w, w.y, out, T, K, E, dims->d_model, s);
}
