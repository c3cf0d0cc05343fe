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
#include "tc_common.cuh"

namespace bitsmoe {

int launch_combine(const int32_t* ids, const float* gw, float* Ye, float* Ysum, int T, int K, int E, int d_out,
                   cudaStream_t s);

constexpr int kGmmMaxRows = 1 << 30;  // a row's index and a tile of rows behind it are ints
constexpr int kGmmMaxIn = 1 << 30;    // so are a k and a step of all warps behind it

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

// The group of expert e in ascending offsets, inside [0, P].  True when its end is below its start: the groups from it
// on are then those of group_from.
__device__ __forceinline__ bool group_range(const GmmParams& P, int e, int& i0, int& i1) {
    const int a = P.offsets[e], b = P.offsets[e + 1];
    i0 = min(max(a, 0), P.P);
    i1 = min(max(b, i0), P.P);
    if ((i0 != a || i1 != b) && P.status) atomicOr(P.status, BITSMOE_ST_BADGROUP);
    return b < a;
}
// Whatever the offsets hold, an offset counts as the largest up to it, so that no row belongs to two experts (both
// would write it): the group that starts at i0, the end of the one before, ends at i0 or at offset e + 1.
__device__ __forceinline__ int group_from(const GmmParams& P, int e, int i0) {
    return min(max(P.offsets[e + 1], i0), P.P);
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

// ---------------------------------------------------------------------------
// few rows per expert
// ---------------------------------------------------------------------------
// Bound by the weights' bytes, with too few of them for the kernel below (one token, 8 of
// 128 experts, 2048 -> 768 gated: 11.6 us, 4.3 TB/s).  A CTA owns 16 rows of one expert's
// matrix (of both, when gated) and up to 8 of its input rows; its 4 warps take a quarter of K
// each, so that every SM has enough loads in flight when only a few experts are
// touched, and add their fp32 partial tiles in warp order.  The products are
// mma.sync m16n8k16 on operands that go from global memory to registers: a lane
// loads 16 contiguous bytes of weight row g (and g + 8), eight k's that the two MMAs
// of a 32-wide step take as k = 2c, 2c+1, 2c+8, 2c+9; the input rows are loaded with
// the same order of k, so the sum over k is the same and no operand is rearranged.
//
// 4 warps, and registers for a warp's loads of 4 steps at once: 8 warps took 15.4 us
// in that case, and 10.4 instead of 7.4 for the 768 -> 2048 products of one token.
//
// Which of the two kernels (us, this one / the next; K x N matrices of E experts, pairs of rows):
//   gated 2048 x 768, E = 128:   32 pairs 33.4 / 38.1    128 pairs 81.9 / 81.3   256 pairs  106 /  105
//   768 x 2048, E = 128:         64 pairs 33.0 / 33.6    128 pairs 56.3 / 48.5
//   1024 x 4096, E = 64:         32 pairs 36.0 / 37.3     64 pairs 59.3 / 54.0
//   gated 2048 x 768, E = 8:     32 pairs 11.3 / 16.2     64 pairs 12.4 / 16.4   192 pairs 22.0 / 16.8
//   768 x 2048, E = 8:           32 pairs  6.1 /  9.1     64 pairs  9.1 /  9.1    96 pairs 10.2 /  9.1
//   gated 4096 x 14336, E = 8:    4 pairs  120 /  129     32 pairs  305 /  295    64 pairs  415 /  296
//   2048 x 256, E = 8:          256 pairs  9.6 / 15.7   1024 pairs 18.0 / 18.8
//   4096 x 64, E = 2:            32 pairs  6.1 / 24.2    512 pairs  7.1 / 30.6
//   gated 4096 x 256, E = 2:     32 pairs  7.8 / 24.0    512 pairs 27.3 / 27.1
// The next one's CTA pairs take blocks of 256 weight rows over all of K: it is slower while these are few for the SMs,
// and this one reads the weights again for every 8 rows of an expert.  So the next one takes over where its tiles are
// many and the experts have a row each on average, or more than 8 rows; but not products with few results.
constexpr int kTcTiles = 384, kTcRows = 8, kMvResults = 1 << 17;
constexpr int kMvWarps = 4;
constexpr int kMvThreads = 32 * kMvWarps;
constexpr int kMvRows = 16, kMvTok = 8;  // weight rows and input rows of a CTA
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
        asm(
            "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
            : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
            : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
    else
        asm(
            "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
            : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
            : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Expert and first sorted row of work slot `slot`: the experts' groups cut into pieces
// of `tok` rows, in expert order.  Every warp of the CTA calls it; false past the end.
__device__ __forceinline__ bool find_slot(const GmmParams& P, int slot, int tok, int& e_out, int& i0_out, int& n_out) {
    const int lane = threadIdx.x & 31;
    int base = 0;
    bool fell = false;
    for (int e0 = 0; e0 < P.E; e0 += 32) {
        const int e = e0 + lane;
        int i0 = 0, i1 = 0;
        bool falls = false;
        if (e < P.E) falls = group_range(P, e, i0, i1);
        fell = __any_sync(0xffffffffu, falls);
        if (fell) break;
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
    if (!fell) return false;
    int i0 = min(max(P.offsets[0], 0), P.P);
    base = 0;
#pragma unroll 1
    for (int e = 0; e < P.E; e++) {  // offsets that fall: one expert after the other
        const int i1 = group_from(P, e, i0), n = (i1 - i0 + tok - 1) / tok;
        if (slot < base + n) {
            e_out = e;
            i0_out = i0 + (slot - base) * tok;
            n_out = min(tok, i1 - i0_out);
            return true;
        }
        base += n;
        i0 = i1;
    }
    return false;
}

template <bool BF16, bool GATED>
__global__ void __launch_bounds__(kMvThreads, GATED ? 4 : 8) k_gmm_mv(const GmmParams P) {
    constexpr int NW = GATED ? 2 : 1;
    __shared__ float s_part[kMvWarps][NW][kMvRows][kMvTok + 1];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, c = lane & 3;
    pdl_wait();
    pdl_trigger();
    int e, i0, nt;
    if (!find_slot(P, (int)blockIdx.y, kMvTok, e, i0, nt)) return;
    const int n0 = (int)blockIdx.x * kMvRows;

    // this lane's input row and weight rows
    int64_t src = 0, dst = 0;
    const uint16_t* brow = g < nt && row_pair(P, i0 + g, src, dst) ? P.a + src * P.lda : nullptr;
    const uint16_t* wrow[NW][2];
#pragma unroll
    for (int m = 0; m < NW; m++)
#pragma unroll
        for (int r = 0; r < 2; r++) {
            const int n = n0 + g + 8 * r;
            wrow[m][r] = n < P.N ? (m ? P.w_up : P.w) + ((int64_t)e * P.N + n) * P.D : nullptr;
        }
    float acc[NW][4] = {};
    const int steps = (P.D + 31) / 32, per = (steps + kMvWarps - 1) / kMvWarps;
    const int s0 = min(steps, warp * per), s1 = min(steps, s0 + per);
    for (int s = s0; s < s1; s += kMvUnroll) {
        uint4 wv[kMvUnroll][NW][2], bv[kMvUnroll];
#pragma unroll
        for (int u = 0; u < kMvUnroll; u++) {
            const int k = (s + u) * 32 + 8 * c;  // D is a multiple of 8: a lane's 8 k's are inside or outside together
            const bool in = s + u < s1 && k < P.D;
#pragma unroll
            for (int m = 0; m < NW; m++)
#pragma unroll
                for (int r = 0; r < 2; r++)
                    wv[u][m][r] = in && wrow[m][r] ? ld_stream(wrow[m][r] + k) : make_uint4(0, 0, 0, 0);
            bv[u] = in && brow ? *reinterpret_cast<const uint4*>(brow + k) : make_uint4(0, 0, 0, 0);
        }
        // the MMA's accumulator drops what does not fit, toward zero: 128 k's at a time, joined by fp32 additions
        float part[NW][4] = {};
#pragma unroll
        for (int u = 0; u < kMvUnroll; u++)
#pragma unroll
            for (int m = 0; m < NW; m++) {
                mma16816<BF16>(part[m], wv[u][m][0].x, wv[u][m][1].x, wv[u][m][0].y, wv[u][m][1].y, bv[u].x, bv[u].y);
                mma16816<BF16>(part[m], wv[u][m][0].z, wv[u][m][1].z, wv[u][m][0].w, wv[u][m][1].w, bv[u].z, bv[u].w);
            }
#pragma unroll
        for (int m = 0; m < NW; m++)
#pragma unroll
            for (int q = 0; q < 4; q++) acc[m][q] += part[m][q];
    }
#pragma unroll
    for (int m = 0; m < NW; m++)
#pragma unroll
        for (int q = 0; q < 4; q++) s_part[warp][m][g + 8 * (q >> 1)][2 * c + (q & 1)] = acc[m][q];
    __syncthreads();
    for (int v = threadIdx.x; v < nt * kMvRows; v += kMvThreads) {
        const int i = v / kMvRows, r = v % kMvRows;
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
    const int slots = std::min(P.P, P.E) + P.P / kMvTok;  // at least the pieces of every group; at most 2^15 here
    return launch_pdl(k_gmm_mv<BF16, GATED>, dim3((P.N + kMvRows - 1) / kMvRows, slots), dim3(kMvThreads), 0, s, P);
}

// ---------------------------------------------------------------------------
// many rows per expert: the tensor cores
// ---------------------------------------------------------------------------
// The transposed product, out^T = W a^T: the weights' rows are the MMA's M, the
// expert's input rows its N, so a ragged group costs its size rounded up to 32 and not
// to a tile of 128.  Two CTAs (a cluster, one per SM) share each tile: tcgen05.mma
// cta_group::2 with M = 256 weight rows (128 per CTA; of both matrices when gated) and
// N = up to 256 (gated: 128) input rows, half of whose rows each CTA stages; an SM then
// reads 8 KB of shared memory per 128 x 256 x 16 step instead of 12.  Persistent CTA
// pairs walk the tiles -- expert, then block of 256 weight rows, then piece of the
// group, so that the pieces that share weights run at the same time and the weights
// come from HBM once.  Warp roles in each CTA: one issues the TMA loads (weights, and
// input rows when they are contiguous), one -- in the first CTA of the pair -- the
// MMAs, four move finished accumulators from tensor memory to out while the next
// tile's MMAs fill the other half of tensor memory, and with gathered input rows eight
// more fetch those by 16-byte asynchronous copies into the same swizzled layout and one
// passes their arrival on.
// The number of tiles is known on the device alone: every CTA derives it from offsets.
//
// Bound by the weights' bytes up to a few hundred rows per expert, then by the tensor
// pipe.  A few calls / a loop of seconds, in which the board's power limit lowers the clocks:
// 128 experts, 2048 -> 768 gated, gathered, 128 pairs 81 us (510 MB, 6.3 TB/s), 16,384 pairs
// 153 / 181 us (870 MB, 5.7 / 4.8 TB/s, the tensor pipe 40% busy; 1.24 GHz in the loop);
// 768 -> 2048 with fp32 results, 16,384 pairs 107 / 122 us (1.59 GHz); 8 experts, 4096 ->
// 14336, 2,050 pairs 232 to 250 / 298 us (1.04 to 0.96 / 0.81 PFLOP/s; 1.07 GHz).  The clocks are
// not all of the last: it does 0.70 to 0.76 TFLOP/s per MHz, the library's dense product of
// 8192^3 1.04, and no unit is full (tensor pipe 68%, L2 45%, DRAM 55%).  Likely the weights'
// path from L2: the pieces of one expert load the same weight tiles, each for itself.
// Tiles of one expert stand together:
// walking them by block of weight rows over all experts was 2 to 5% slower.
constexpr int kGtM = 128;                        // weight rows per CTA and matrix
constexpr int kGtK = 64;                         // K per stage: one 128-byte swizzled row
constexpr int kGtMaxStages = 12;
constexpr uint32_t kGtAStage = kGtM * kGtK * 2;  // 16 KB
constexpr int kGtRelayWarp = 2;                  // warps 0 and 1 issue loads and MMAs; 3 is idle
constexpr int kGtEpiWarp0 = 4, kGtGatherWarps = 8;
__host__ __device__ constexpr int gt_epi_warps(bool seg) { return seg ? 8 : 4; }
__host__ __device__ constexpr int gt_gather_warp0(bool seg) { return kGtEpiWarp0 + gt_epi_warps(seg); }
constexpr int gt_threads(bool gather, bool seg) { return 32 * (gt_gather_warp0(seg) + (gather ? kGtGatherWarps : 0)); }
constexpr size_t kGtSmem = 204 * 1024;           // dynamic shared memory a CTA uses at most (21 KB are static)
// Segments.  The tensor cores' fp32 accumulator cuts what does not fit, toward zero, at every step of 16 k: an
// error of about 1.2e-9 K of the results' norm (measured: 4.9e-6 at K = 4096, twice that when gated; 4e-6 of a
// sum of 768 terms of one sign), nothing beside a rounding to 16 bits but several times an fp32 sum's.  For fp32
// results it is kept under 1e-6: at most 768 k's (gated: 384) are summed in tensor memory, and fp32 additions to
// nearest in the epilogue's registers join them.  The epilogue is then 8 warps with 128 sums a thread: 384
// threads launch with 168 registers each; the 640 of the gathering kernel with 96, of which the others give up
// half: 256 x 168 + 384 x 48 = 640 x 96.  (At 16,384 pairs of 128 experts, 2048 x 768, fp32 results, three
// segments took 126 us instead of 103.)
constexpr int gt_segment(bool gated) { return gated ? 6 : 12; }

constexpr int kGtBoxes = 5;
__host__ __device__ constexpr int gt_box(int i) { return i < 3 ? 16 << i : 32 * i; }  // 16, 32, 64, 96, 128 rows
struct GtMaps {
    CUtensorMap w, u;          // weights: boxes of 128 rows
    CUtensorMap a[kGtBoxes];   // input rows
};

struct GmmTcParams {
    GmmParams p;
    int tok;          // input rows per piece, at most (a multiple of 32)
    int ntiles;       // blocks of 256 weight rows
    int nst;          // K stages
    int stages;       // ring
    int seg;          // K stages summed in tensor memory
    uint32_t stage_bytes;
    int vec;          // rows of out are whole 16-byte pieces
};

// True in one lane of a converged warp.  The warp-wide roles below run their loops in
// every lane and issue under this: ptxas then knows that one thread executes the TMA and
// MMA instructions, whose operands are warp-uniform registers, and need not serialise
// over the lanes (under `if (lane == 0)` an MMA took about 100 cycles to issue).
__device__ __forceinline__ bool gt_elect() {
    uint32_t p;
    asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}\n" : "=r"(p));
    return p != 0;
}
__device__ __forceinline__ uint32_t gt_mapa(uint32_t addr, uint32_t rank) {
    uint32_t r;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
    return r;
}
__device__ __forceinline__ void gt_arrive_cluster(uint32_t bar) {
    asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ void gt_cluster_sync() {
    asm volatile("barrier.cluster.arrive.release.aligned;\n barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// A TMA tile into this CTA's shared memory that completes on a barrier of either CTA of the pair.
__device__ __forceinline__ void gt_tma2d(uint32_t dst, const CUtensorMap* map, int x, int y, uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], "
        "[%4];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(bar)
        : "memory");
}
__device__ __forceinline__ void gt_commit_both(uint32_t bar) {
    asm volatile(
        "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(bar),
        "h"((uint16_t)3)
        : "memory");
}
__device__ __forceinline__ void gt_mma(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
    asm volatile(
        "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n}\n" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(acc)
        : "memory");
}
template <int REGS, bool MORE>
__device__ __forceinline__ void gt_regs() {
    if constexpr (MORE)
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(REGS));
    else
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(REGS));
}
__device__ __forceinline__ void gt_ld16(uint32_t addr, uint32_t (&v)[16]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
        : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7]), "=r"(v[8]),
          "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]), "=r"(v[14]), "=r"(v[15])
        : "r"(addr));
}

// 32 columns of each accumulator to, or with `more` added to, a thread's sums.
template <int NW, bool SEG>
__device__ __forceinline__ void gt_add(uint32_t addr, bool more, float (&y)[NW][32]) {
    uint32_t v[SEG ? 1 : 2 * NW][16];
#pragma unroll
    for (int m = 0; m < 2 * NW; m++) {
        uint32_t(&x)[16] = v[SEG ? 0 : m];
        gt_ld16(addr + 128u * (m >> 1) + 16u * (m & 1), x);
        if (SEG) {
            asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
            for (int j = 0; j < 16; j++) {
                float& s = y[m >> 1][16 * (m & 1) + j];
                s = more ? s + __uint_as_float(x[j]) : __uint_as_float(x[j]);
            }
        }
    }
    if (!SEG) {
        asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
        for (int m = 0; m < 2 * NW; m++)
#pragma unroll
            for (int j = 0; j < 16; j++) y[m >> 1][16 * (m & 1) + j] = __uint_as_float(v[SEG ? 0 : m][j]);
    }
}

// Column `row` of ROWS rows of out from shared memory, [ROWS][32]; dst: the rows' places, -1 for none.
template <typename T, int ROWS>
__device__ __forceinline__ void gt_store_rows(const T* src, const int* dst, void* out, int n_out, int row) {
    if (row >= n_out) return;
    T* col = static_cast<T*>(out) + row;
    const int lane = threadIdx.x & 31;
    for (int j = 0; j < ROWS; j += 8) {
        T v[8];
        int d[8];
#pragma unroll
        for (int k = 0; k < 8; k++) {
            v[k] = src[32 * (j + k) + lane];
            d[k] = dst[j + k];
        }
#pragma unroll
        for (int k = 0; k < 8; k++)
            if (d[k] >= 0) col[(int64_t)d[k] * n_out] = v[k];
    }
}

// One tile of the walk.
struct GtTile {
    int e, n0;   // expert, first weight row of the pair's block
    int i0, cnt; // first sorted row and rows of the piece
    int n_mma;   // cnt rounded up to 32
};
__device__ __forceinline__ int gt_pieces(int cnt, int tok) { return (cnt + tok - 1) / tok; }

// Tile `item`; s_tab[e]: tiles of the experts before e.
__device__ __forceinline__ GtTile gt_tile(const GmmTcParams& Q, const int* s_tab, int item) {
    int lo = 0, hi = Q.p.E;  // s_tab[lo] <= item < s_tab[hi]
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (s_tab[mid] <= item)
            lo = mid;
        else
            hi = mid;
    }
    GtTile t;
    t.e = lo;
    int i0, i1;
    group_range(Q.p, lo, i0, i1);
    const int np = gt_pieces(i1 - i0, Q.tok), within = item - s_tab[lo];
    // pieces of equal size, whole steps of 32
    const int size = (int)roundup((uint64_t)((i1 - i0 + np - 1) / np), 32);
    t.n0 = within / np * (2 * kGtM);
    t.i0 = i0 + within % np * size;
    t.cnt = max(0, min(size, i1 - t.i0));
    t.n_mma = max(32, (int)roundup((uint64_t)t.cnt, 32));
    return t;
}

// All of it by fp32 products one by one, a result per thread: for offsets that fall somewhere, which are an error of
// the caller's that need not be fast.  (With tiles that look for their groups in such offsets, every call took 1% more:
// 16,384 pairs, 768 -> 2048, 122.9 us instead of 121.4.)
template <bool GATED>
__device__ __forceinline__ void gmm_plain(const GmmParams& P) {
    int i0 = min(max(P.offsets[0], 0), P.P);
#pragma unroll 1
    for (int e = 0; e < P.E; e++) {
        const int i1 = group_from(P, e, i0);
        const int64_t n = (int64_t)(i1 - i0) * P.N;
#pragma unroll 1
        for (int64_t v = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; v < n; v += (int64_t)gridDim.x * blockDim.x) {
            int64_t src, dst;
            if (!row_pair(P, i0 + (int)(v / P.N), src, dst)) continue;
            const int64_t row = ((int64_t)e * P.N + v % P.N) * P.D;
            float y = 0.0f, u = 0.0f;
#pragma unroll 1
            for (int k = 0; k < P.D; k++) {
                const float a = half_bits(P.a[src * P.lda + k], P.type);
                y = fmaf(half_bits(P.w[row + k], P.type), a, y);
                if (GATED) u = fmaf(half_bits(P.w_up[row + k], P.type), a, u);
            }
            const float o[1] = {GATED ? silu_f(y) * u : y};
            store_elems<1>(P.out, P.out_type, dst * P.N + v % P.N, o);
        }
        i0 = i1;
    }
}

template <bool GATED, bool GATHER, bool SEG>
__global__ void __launch_bounds__(gt_threads(GATHER, SEG), 1)
    k_gmm_tc(const GmmTcParams Q, const __grid_constant__ GtMaps M) {
    constexpr int NW = GATED ? 2 : 1, EW = gt_epi_warps(SEG), kGatherWarp0 = gt_gather_warp0(SEG);
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    __shared__ uint64_t s_full[kGtMaxStages], s_empty[kGtMaxStages], s_rows[kGtMaxStages], s_afull[2], s_aempty[2];
    __shared__ uint32_t s_tmem;
    __shared__ int s_fail;
    __shared__ int s_dst[EW][1024 / EW];  // per epilogue warp: output row of each of its input rows, -1 for none
    __shared__ __align__(16) uint4 s_out[EW][1024 / EW];  // per epilogue warp: results to be stored
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    uint32_t rank;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(rank));
    const GmmParams& P = Q.p;
    const uint32_t sbase = (tc_smem(smem_raw) + 1023u) & ~1023u;
    int* s_tab = reinterpret_cast<int*>(smem_raw + (sbase - tc_smem(smem_raw)) + (size_t)Q.stages * Q.stage_bytes);  // [E+1]

    if (warp == 0) {
        asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(tc_smem(&s_tmem)), "r"(512u)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
    }
    if (tid == 32) {
        for (int i = 0; i < kGtMaxStages; i++) {
            asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(tc_smem(&s_full[i])),
                         "r"(GATHER ? 3u : 1u));  // the TMA bytes; each CTA's gathered rows
            asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(tc_smem(&s_rows[i])), "r"(32u * kGtGatherWarps));
            asm volatile("mbarrier.init.shared::cta.b64 [%0], 1;" ::"r"(tc_smem(&s_empty[i])));
        }
        for (int i = 0; i < 2; i++) {
            asm volatile("mbarrier.init.shared::cta.b64 [%0], 1;" ::"r"(tc_smem(&s_afull[i])));
            asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(tc_smem(&s_aempty[i])), "r"(2u * EW));
        }
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        s_fail = 0;
    }
    pdl_wait();
    pdl_trigger();
    // tiles of every expert, then their running sum
    int falls = 0;
    for (int e = tid; e < P.E; e += blockDim.x) {
        int i0, i1;
        falls |= group_range(P, e, i0, i1);
        s_tab[e + 1] = gt_pieces(i1 - i0, Q.tok) * Q.ntiles;
    }
    if (tid == 0) s_tab[0] = 0;
    falls = __syncthreads_or(falls);
    if (falls) gmm_plain<GATED>(P);  // and no tiles; here, where every thread still has the registers of the launch
    if (warp == 0) {
        int base = 0;
        for (int e0 = 0; e0 < P.E; e0 += 32) {
            int v = e0 + lane < P.E ? s_tab[e0 + lane + 1] : 0;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int u = __shfl_up_sync(0xffffffffu, v, o);
                if (lane >= o) v += u;
            }
            if (e0 + lane < P.E) s_tab[e0 + lane + 1] = base + v;
            base += __shfl_sync(0xffffffffu, v, 31);
        }
    }
    asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
    __syncthreads();
    gt_cluster_sync();  // both CTAs' barriers and tensor memory are ready
    asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
    const uint32_t tmem = s_tmem;
    const int total = falls ? 0 : s_tab[P.E], first = (int)blockIdx.x >> 1, step = (int)gridDim.x >> 1;
    const uint32_t b_off = NW * kGtAStage;
    volatile int* fail = &s_fail;

    if (warp >= kGtEpiWarp0 && warp < kGatherWarp0) {
        if constexpr (GATHER && SEG) gt_regs<168, true>();
        // accumulators to out: a thread owns a weight row, a column of tensor memory is an input row.  With 8 warps two
        // share 32 weight rows and take the blocks of 32 input rows in turn.
        constexpr int SHARE = EW / 4, NB = 8 / (NW * SHARE);  // NB: blocks a warp takes at most
        constexpr int PASS = SEG ? 2 : 1;  // fp32 results go through shared memory in this many passes
        const int sub = warp & 3, half = (warp - kGtEpiWarp0) >> 2;  // sub: the 32 lanes of tensor memory a warp can read
        int* dst_of = s_dst[warp - kGtEpiWarp0];
        uint4* stage_out = s_out[warp - kGtEpiWarp0];
        const uint32_t aempty0 = gt_mapa(tc_smem(&s_aempty[0]), 0);
        const bool f32 = SEG || P.out_type == BITSMOE_F32;
        const int cw = f32 ? 8 : 4, piece = lane % cw;  // 16-byte pieces of 32 results, and this lane's
        const int64_t pitch = (int64_t)P.N * (f32 ? 4 : 2);
        int buf = 0;
        uint32_t phase = 0;
        bool ok = true;
        for (int item = first; item < total && ok; item += step) {
            const GtTile t = gt_tile(Q, s_tab, item);
            for (int i = 0; i < NB; i++) {
                const int j = 32 * (SHARE * i + half) + lane;
                int64_t src, dst;
                dst_of[32 * i + lane] = j < t.cnt && row_pair(P, t.i0 + j, src, dst) ? (int)dst : -1;
            }
            __syncwarp();
            const int row = t.n0 + (int)rank * kGtM + 32 * sub, row0 = row + piece * (32 / cw);  // whole pieces inside N
            uint8_t* out0 = static_cast<uint8_t*>(P.out) + (int64_t)row0 * (f32 ? 4 : 2);
            float y[SEG ? NB : 1][NW][32];
            for (int k = 0; k < Q.nst; k += Q.seg) {
                ok = warp_wait(tc_smem(&s_afull[buf]), phase);
                if (!ok) break;
                asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
                const uint32_t tl = tmem + 256u * buf + ((uint32_t)(32 * sub) << 16);
#pragma unroll(SEG ? NB : 1)
                for (int i = 0; i < NB; i++) {
                    const int c0 = 32 * (SHARE * i + half), cols = min(32, t.cnt - c0);
                    if (cols <= 0) break;
                    float(&yb)[NW][32] = y[SEG ? i : 0];
                    gt_add<NW, SEG>(tl + (uint32_t)c0, k > 0, yb);
                    if (SEG && k + Q.seg < Q.nst) continue;
                    if (GATED) {
#pragma unroll
                        for (int j = 0; j < 32; j++) yb[0][j] = silu_f(yb[0][j]) * yb[NW - 1][j];
                    }
                    // through shared memory, [input row][32 weight rows]: then 16 bytes per thread and store, or, where rows
                    // of out are not whole 16-byte pieces, a weight row per thread, 8 stores behind their 8 loads (one by
                    // one, each under its branch, 4,737 rows x 206 took 28 us, and 208 columns 12)
#pragma unroll
                    for (int p = 0; p < PASS; p++) {
                        if (!f32 && p > 0) break;
                        __syncwarp();
                        if (f32) {
                            float* f = reinterpret_cast<float*>(stage_out);
#pragma unroll
                            for (int j = 0; j < 32 / PASS; j++) f[32 * j + lane] = yb[0][32 / PASS * p + j];
                        } else {
                            uint16_t* h = reinterpret_cast<uint16_t*>(stage_out);
                            if (P.type == BITSMOE_F16) {
#pragma unroll
                                for (int j = 0; j < 32; j++) h[32 * j + lane] = (uint16_t)to_half_bits(yb[0][j], BITSMOE_F16);
                            } else {
#pragma unroll
                                for (int j = 0; j < 32; j++) h[32 * j + lane] = (uint16_t)to_half_bits(yb[0][j], BITSMOE_BF16);
                            }
                        }
                        __syncwarp();
                        const int j0 = 32 / PASS * p, n = f32 ? min(32 / PASS, cols - j0) : cols;
                        const int* dsts = dst_of + 32 * i + j0;  // -1 past the last row
                        if (Q.vec) {
#pragma unroll 4
                            for (int j = lane / cw; j < n; j += 32 / cw) {
                                const int dst = dsts[j];
                                const uint4 w = stage_out[j * cw + piece];
                                if (dst >= 0 && row0 < P.N) *reinterpret_cast<uint4*>(out0 + dst * pitch) = w;
                            }
                        } else if (f32) {
                            gt_store_rows<float, 32 / PASS>(reinterpret_cast<const float*>(stage_out), dsts, P.out, P.N, row + lane);
                        } else {
                            gt_store_rows<uint16_t, 32>(reinterpret_cast<const uint16_t*>(stage_out), dsts, P.out, P.N, row + lane);
                        }
                    }
                }
                asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
                __syncwarp();
                if (lane == 0) gt_arrive_cluster(aempty0 + 8u * (uint32_t)buf);
                buf ^= 1;
                if (buf == 0) phase ^= 1u;
            }
        }
        if (!ok) *fail = 1;
    } else {
        if constexpr (GATHER && SEG) gt_regs<48, false>();
        if (warp == 0) {
            // the weights' tiles, and contiguous input rows; the pair's bytes complete on the first CTA's barrier
            const uint32_t full0 = gt_mapa(tc_smem(&s_full[0]), 0);
            int s = 0;
            uint32_t phase = 1;  // parity of the stage's last release: nothing to wait for in the first round
            bool ok = true;
            for (int item = first; item < total && ok; item += step) {
                const GtTile t = gt_tile(Q, s_tab, item);
                const int half = t.n_mma / 2, row_w = t.e * P.N + t.n0 + (int)rank * kGtM;
                const int row_a = t.i0 + (int)rank * half;
                // one box of at least the half's rows: an issued TMA costs more than the rows behind them
                const int bi = half <= 16 ? 0 : half <= 32 ? 1 : half <= 64 ? 2 : half <= 96 ? 3 : 4;
                const CUtensorMap* tmA = &M.a[bi];
                const uint32_t bytes = 2u * (NW * kGtAStage + (GATHER ? 0u : 128u * (uint32_t)gt_box(bi)));
                for (int k = 0; k < Q.nst; k++) {
                    ok = warp_wait(tc_smem(&s_empty[s]), phase);
                    if (!ok) break;
                    if (gt_elect()) {
                        const uint32_t st = sbase + (uint32_t)s * Q.stage_bytes, bar = full0 + 8u * (uint32_t)s;
                        if (rank == 0)
                            asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(tc_smem(&s_full[s])),
                                         "r"(bytes)
                                         : "memory");
                        gt_tma2d(st, &M.w, k * kGtK, row_w, bar);
                        if (GATED) gt_tma2d(st + kGtAStage, &M.u, k * kGtK, row_w, bar);
                        if (!GATHER) gt_tma2d(st + b_off, tmA, k * kGtK, row_a, bar);
                    }
                    __syncwarp();
                    if (++s == Q.stages) {
                        s = 0;
                        phase ^= 1u;
                    }
                }
            }
            if (!ok) *fail = 1;
        } else if (warp == 1) {
            if (rank == 0) {
                int s = 0, buf = 0;
                uint32_t phase = 0, aphase = 1;
                bool ok = true;
                for (int item = first; item < total && ok; item += step) {
                    const GtTile t = gt_tile(Q, s_tab, item);
                    const uint32_t idesc = tc_idesc(2 * kGtM, t.n_mma) | (P.type == BITSMOE_BF16 ? (1u << 7) | (1u << 10) : 0u);
                    int left = 0;  // stages left in the segment
                    for (int k = 0; k < Q.nst; k++) {
                        const uint32_t d = tmem + 256u * buf;
                        const bool begin = left == 0;
                        if (begin) {
                            left = min(Q.seg, Q.nst - k);
                            ok = warp_wait(tc_smem(&s_aempty[buf]), aphase);
                            if (!ok) break;
                        }
                        const bool end = --left == 0;
                        ok = warp_wait(tc_smem(&s_full[s]), phase);
                        if (!ok) break;
                        asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
                        if (gt_elect()) {
                            const uint32_t st = sbase + (uint32_t)s * Q.stage_bytes;
                            // a K step of 16 elements is 32 bytes further in the swizzled row: 2 in the descriptor's address
                            const uint64_t ad = tc_desc_sw128(st), bd = tc_desc_sw128(st + b_off);
#pragma unroll
                            for (int kk = 0; kk < kGtK / 16; kk++)
#pragma unroll
                                for (int m = 0; m < NW; m++)
                                    gt_mma(d + 128u * m, ad + (uint64_t)(m * (kGtAStage >> 4) + 2 * kk), bd + 2u * kk, idesc,
                                           (!begin || kk > 0) ? 1u : 0u);
                            gt_commit_both(tc_smem(&s_empty[s]));
                            if (end) gt_commit_both(tc_smem(&s_afull[buf]));
                        }
                        __syncwarp();
                        if (++s == Q.stages) {
                            s = 0;
                            phase ^= 1u;
                        }
                        if (end) {
                            buf ^= 1;
                            if (buf == 0) aphase ^= 1u;
                        }
                    }
                }
                if (!ok) *fail = 1;
            }
        } else if (GATHER && warp == kGtRelayWarp) {
            // A stage's gathered rows have arrived: the copies wrote shared memory as ordinary
            // stores do, the MMAs read it as the asynchronous proxy; then tell the first CTA.
            // (A gathering thread that fenced would wait for its later copies as well.)
            const uint32_t full0 = gt_mapa(tc_smem(&s_full[0]), 0);
            int s = 0;
            uint32_t phase = 0;
            bool ok = true;
            for (int item = first; item < total && ok; item += step)
                for (int k = 0; k < Q.nst; k++) {
                    ok = warp_wait(tc_smem(&s_rows[s]), phase);
                    if (!ok) break;
                    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                    if (gt_elect()) gt_arrive_cluster(full0 + 8u * (uint32_t)s);
                    __syncwarp();
                    if (++s == Q.stages) {
                        s = 0;
                        phase ^= 1u;
                    }
                }
            if (!ok) *fail = 1;
        } else if (GATHER && warp >= kGatherWarp0) {
            // this CTA's half of the piece's input rows: 8 threads a row, 16 bytes each, chunk ch of row r at ch ^ (r mod 8)
            const int gt = tid - 32 * kGatherWarp0, ch = gt & 7, r0 = gt >> 3;
            constexpr int RS = 4 * kGtGatherWarps, RPT = kGtM / RS;  // rows a thread fetches: r0 + RS i of up to 128
            const uint32_t b0 = sbase + b_off + 128u * r0 + ((uint32_t)(ch ^ (r0 & 7)) << 4);  // RS is a multiple of 8
            int s = 0;
            uint32_t phase = 1;
            bool ok = true;
            for (int item = first; item < total && ok; item += step) {
                const GtTile t = gt_tile(Q, s_tab, item);
                const int half = t.n_mma / 2;
                const uint16_t* src_row[RPT];  // NULL: zeros
#pragma unroll
                for (int i = 0; i < RPT; i++) {
                    const int r = r0 + RS * i, j = (int)rank * half + r;
                    int64_t src = 0, dst;
                    src_row[i] = r < half && j < t.cnt && row_pair(P, t.i0 + j, src, dst) ? P.a + src * P.lda + 8 * ch : nullptr;
                }
                for (int k = 0; k < Q.nst; k++) {
                    ok = warp_wait(tc_smem(&s_empty[s]), phase);
                    if (!ok) break;
                    const uint32_t b = b0 + (uint32_t)s * Q.stage_bytes;
                    const bool in_k = k * kGtK + 8 * ch < P.D;
#pragma unroll
                    for (int i = 0; i < RPT; i++)
                        if (r0 + RS * i < half) {
                            const bool in = src_row[i] != nullptr && in_k;
                            asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(b + 128u * RS * i),
                                         "l"(in ? src_row[i] + k * kGtK : P.a), "r"(in ? 16 : 0)
                                         : "memory");
                        }
                    asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(tc_smem(&s_rows[s])) : "memory");
                    if (++s == Q.stages) {
                        s = 0;
                        phase ^= 1u;
                    }
                }
            }
            asm volatile("cp.async.wait_all;" ::: "memory");
            if (!ok) *fail = 1;
        }
    }
    __syncwarp();
    if (*fail && lane == 0 && P.status) atomicOr(P.status, BITSMOE_ST_TIMEOUT);
    asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
    __syncthreads();
    gt_cluster_sync();  // neither CTA leaves while the other may signal its barriers or use its shared memory
    asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
    if (warp == 0)
        asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512u) : "memory");
}

template <bool GATED, bool GATHER, bool SEG>
static int launch_gmm_tc(const GmmParams& P, cudaStream_t s) {
    GmmTcParams Q{};
    Q.p = P;
    // input rows per piece: fewer keep the ring deeper, more share the weights' tiles (64 experts, 768 x 2048, pieces of
    // 128 and 256, us: 48 rows per expert 41.5 and 42.7, 64 rows 43.8 and 44.5, 128 rows 62.4 and 51.7)
    Q.tok = GATED || P.P <= 64 * (int64_t)P.E ? 128 : 256;
    Q.ntiles = (P.N + 2 * kGtM - 1) / (2 * kGtM);
    Q.nst = (P.D + kGtK - 1) / kGtK;
    const int segs = SEG ? (Q.nst + gt_segment(GATED) - 1) / gt_segment(GATED) : 1;
    Q.seg = (Q.nst + segs - 1) / segs;
    Q.stage_bytes = (GATED ? 2 : 1) * kGtAStage + (uint32_t)Q.tok / 2 * 128u;
    const size_t tab = roundup(4ull * (P.E + 1), 16);
    Q.stages = (int)std::min<size_t>(kGtMaxStages, (kGtSmem - 1024 - tab) / Q.stage_bytes);
    const size_t smem = 1024 + (size_t)Q.stages * Q.stage_bytes + tab;
    Q.vec = (uintptr_t)P.out % 16 == 0 && P.N % (16 / elem_bytes(P.out_type)) == 0;
    GtMaps M;
    int rc = tc_tensor_map(&M.w, P.w, P.D, P.E * P.N, kGtM);
    if (!rc && GATED) rc = tc_tensor_map(&M.u, P.w_up, P.D, P.E * P.N, kGtM);
    for (int i = 0; i < kGtBoxes && !rc && !GATHER; i++)
        rc = tc_tensor_map_ld(&M.a[i], P.a, P.D, P.n_a, P.lda, gt_box(i));
    if (rc) return rc;
    int dev = 0, sms = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    if (e == cudaSuccess)
        e = cudaFuncSetAttribute(k_gmm_tc<GATED, GATHER, SEG>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kGtSmem);
    if (e != cudaSuccess) return set_cuda_error(e);
    const int64_t tiles = (int64_t)Q.ntiles * (std::min(P.P, P.E) + P.P / Q.tok);  // at least as many as there are
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)(2 * std::min<int64_t>(sms / 2, tiles)));
    cfg.blockDim = dim3(gt_threads(GATHER, SEG));
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = 2;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    e = cudaLaunchKernelEx(&cfg, k_gmm_tc<GATED, GATHER, SEG>, Q, M);
    return e == cudaSuccess ? BITSMOE_OK : set_cuda_error(e);
}

template <bool GATED, bool GATHER>
static int launch_gmm_seg(const GmmParams& P, cudaStream_t s) {
    return P.out_type == BITSMOE_F32 && P.D > kGtK * gt_segment(GATED) ? launch_gmm_tc<GATED, GATHER, true>(P, s)
                                                                       : launch_gmm_tc<GATED, GATHER, false>(P, s);
}

}  // namespace bitsmoe

using namespace bitsmoe;

static int gmm_refusal(const bitsmoe_gmm_args& d) {
    if (d.n_rows < 0 || d.n_rows > kGmmMaxRows || d.n_a_rows < 0 || d.n_out < 1 || d.n_in < 8 || d.n_in > kGmmMaxIn || d.n_in % 8 || d.n_experts < 1 ||
        d.n_experts > BITSMOE_GMM_MAX_EXPERTS || (d.in_type != BITSMOE_F16 && d.in_type != BITSMOE_BF16) ||
        (d.out_type != BITSMOE_F32 && d.out_type != d.in_type) || d.rows_per_a < 1 || d.reserved ||
        (int64_t)d.n_experts * d.n_out > 0x7fffffff - 2 * kGtM)  // a tile's last weight row is an int
        return BITSMOE_EINVAL;
    if (!d.rows && (d.scatter || d.rows_per_a != 1 || d.n_a_rows < d.n_rows)) return BITSMOE_EINVAL;
    if (d.n_rows == 0) return BITSMOE_OK;
    if (!d.A || !d.W || !d.offsets || !d.out || d.a_stride < d.n_in || d.a_stride % 8) return BITSMOE_EINVAL;
    if ((uintptr_t)d.A % 16 || (uintptr_t)d.W % 16 || (uintptr_t)d.W_up % 16 || (uintptr_t)d.offsets % 4 ||
        (uintptr_t)d.rows % 4 || (uintptr_t)d.out % elem_bytes(d.out_type))
        return BITSMOE_EINVAL;
    return BITSMOE_OK;
}

static int launch_gmm(const bitsmoe_gmm_args& d, void* stream) {
    GmmParams P{};
    P.a = (const uint16_t*)d.A;
    P.w = (const uint16_t*)d.W;
    P.w_up = (const uint16_t*)d.W_up;
    P.offsets = d.offsets;
    P.rows = d.rows;
    P.out = d.out;
    P.status = d.status;
    P.lda = d.a_stride;
    P.P = d.n_rows;
    P.N = d.n_out;
    P.D = d.n_in;
    P.E = d.n_experts;
    P.n_a = d.n_a_rows;
    P.div = d.rows_per_a;
    P.type = d.in_type;
    P.out_type = d.out_type;
    P.scatter = d.scatter != 0;
    cudaStream_t s = (cudaStream_t)stream;
    const int64_t tiles = (int64_t)((P.N + 2 * kGtM - 1) / (2 * kGtM)) * std::min(P.P, P.E);  // were no two pairs of one expert
    const bool few = (int64_t)P.N * P.P * (P.w_up ? 2 : 1) <= kMvResults;
    if (!few && ((tiles >= kTcTiles && P.P >= P.E) || P.P > kTcRows * P.E)) {
        if (d.rows) return d.W_up ? launch_gmm_seg<true, true>(P, s) : launch_gmm_seg<false, true>(P, s);
        return d.W_up ? launch_gmm_seg<true, false>(P, s) : launch_gmm_seg<false, false>(P, s);
    }
    if (d.in_type == BITSMOE_BF16) return d.W_up ? launch_gmm_mv<true, true>(P, s) : launch_gmm_mv<true, false>(P, s);
    return d.W_up ? launch_gmm_mv<false, true>(P, s) : launch_gmm_mv<false, false>(P, s);
}

BITSMOE_API int bitsmoe_grouped_matmul(const bitsmoe_gmm_args* args, void* stream) {
    if (!args) return BITSMOE_EINVAL;
    const int rc = gmm_refusal(*args);
    return rc || args->n_rows == 0 ? rc : launch_gmm(*args, stream);
}

// ---------------------------------------------------------------------------
// the routed FFN of dense experts
// ---------------------------------------------------------------------------
static bool dense_dims_ok(const bitsmoe_ffn_dims* d, int32_t T) {
    return d && T >= 0 && d->d_model >= 8 && d->d_model % 8 == 0 && d->d_ff >= 8 && d->d_ff % 8 == 0 && d->n_experts >= 1 &&
           d->n_experts <= BITSMOE_GMM_MAX_EXPERTS && d->top_k >= 1 && (int64_t)T * d->top_k <= kGmmMaxRows;
}

BITSMOE_API uint64_t bitsmoe_dense_ffn_workspace_bytes(const bitsmoe_ffn_dims* dims, int32_t T) {
    if (!dense_dims_ok(dims, T) || T == 0) return 0;
    const uint64_t pairs = (uint64_t)T * dims->top_k;
    return roundup(2 * pairs * dims->d_ff, 256) + 4 * pairs * dims->d_model;  // h, then every pair's output row
}

BITSMOE_API int bitsmoe_dense_ffn_forward(const bitsmoe_dense_ffn_args* args, void* stream) {
    if (!args) return BITSMOE_EINVAL;
    const bitsmoe_dense_ffn_args& a = *args;
    const bitsmoe_ffn_dims& d = a.dims;
    if (!dense_dims_ok(&d, a.tokens) || (a.type != BITSMOE_F16 && a.type != BITSMOE_BF16)) return BITSMOE_EINVAL;
    if (a.tokens == 0) return BITSMOE_OK;
    if (!a.x || !a.W_gate || !a.W_up || !a.W_down || !a.topk_ids || !a.gate_w || !a.offsets || !a.order || !a.out)
        return BITSMOE_EINVAL;
    if ((uintptr_t)a.topk_ids % 4 || (uintptr_t)a.gate_w % 4 || (uintptr_t)a.out % 4 || !a.workspace ||
        (uintptr_t)a.workspace % 256)
        return BITSMOE_EINVAL;
    if (a.workspace_bytes < bitsmoe_dense_ffn_workspace_bytes(&d, a.tokens)) return BITSMOE_ESIZE;
    const int pairs = a.tokens * d.top_k;
    uint8_t* h = (uint8_t*)a.workspace;
    float* y = (float*)(h + roundup(2ull * pairs * d.d_ff, 256));
    bitsmoe_gmm_args g{};
    g.A = a.x;
    g.W = a.W_gate;
    g.W_up = a.W_up;
    g.offsets = a.offsets;
    g.rows = a.order;
    g.out = h;
    g.status = a.status;
    g.a_stride = a.x_stride;
    g.n_rows = pairs;
    g.n_a_rows = a.tokens;
    g.n_out = d.d_ff;
    g.n_in = d.d_model;
    g.n_experts = d.n_experts;
    g.in_type = g.out_type = a.type;
    g.rows_per_a = d.top_k;
    g.scatter = 1;
    bitsmoe_gmm_args down = g;
    down.A = h;
    down.W = a.W_down;
    down.W_up = nullptr;
    down.out = y;
    down.a_stride = d.d_ff;
    down.n_a_rows = pairs;
    down.n_out = d.d_model;
    down.n_in = d.d_ff;
    down.out_type = BITSMOE_F32;
    down.rows_per_a = 1;
    int rc = gmm_refusal(g);
    if (!rc) rc = gmm_refusal(down);  // before the first launch
    if (!rc) rc = launch_gmm(g, stream);
    if (!rc) rc = launch_gmm(down, stream);
    if (rc) return rc;
    return launch_combine(a.topk_ids, a.gate_w, y, a.out, a.tokens, d.top_k, d.n_experts, d.d_model, (cudaStream_t)stream);
}
