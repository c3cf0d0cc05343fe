// elem.cuh -- element types of the block operators (norms, routing, grouped
// products): loads and stores that convert between fp32 arithmetic and fp32, fp16
// or bf16 memory, the type chosen at run time (uniform over a launch), and the
// launch helper that lets a kernel's start overlap the end of the kernel before it.
#pragma once

#include <cuda_bf16.h>

#include "common.cuh"

namespace bitsmoe {

__host__ __device__ constexpr int elem_bytes(int type) { return type == BITSMOE_F32 ? 4 : 2; }
inline bool elem_ok(int type) { return type == BITSMOE_F32 || type == BITSMOE_F16 || type == BITSMOE_BF16; }

__device__ __forceinline__ float half_bits(uint32_t b, int type) {
    return type == BITSMOE_F16 ? __half2float(__ushort_as_half((unsigned short)b)) : __uint_as_float(b << 16);
}
__device__ __forceinline__ uint32_t to_half_bits(float v, int type) {
    return type == BITSMOE_F16 ? (uint32_t)__half_as_ushort(__float2half_rn(v))
                               : (uint32_t)__bfloat16_as_ushort(__float2bfloat16_rn(v));
}
// A pair of elements in a word, low half first.
template <bool F16>
__device__ __forceinline__ uint32_t pack2(float a, float b) {
    if constexpr (F16) {
        const __half2 h = __floats2half2_rn(a, b);
        return *reinterpret_cast<const uint32_t*>(&h);
    } else {
        const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
        return *reinterpret_cast<const uint32_t*>(&h);
    }
}
template <bool F16>
__device__ __forceinline__ float2 unpack2(uint32_t w) {
    if constexpr (F16) return __half22float2(*reinterpret_cast<const __half2*>(&w));
    return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
}
__device__ __forceinline__ void unpack4(uint2 w, int type, float (&v)[4]) {
    const float2 a = type == BITSMOE_F16 ? unpack2<true>(w.x) : unpack2<false>(w.x);
    const float2 b = type == BITSMOE_F16 ? unpack2<true>(w.y) : unpack2<false>(w.y);
    v[0] = a.x; v[1] = a.y; v[2] = b.x; v[3] = b.y;
}

// 4 elements, F32 or 16-bit of `type` (16 and 8 bytes, aligned).
template <bool F32>
__device__ __forceinline__ void load4(const void* p, int type, int64_t i, float (&v)[4]) {
    if constexpr (F32) {
        const float4 a = *reinterpret_cast<const float4*>(static_cast<const float*>(p) + i);
        v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
    } else {
        unpack4(*reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(p) + i), type, v);
    }
}
template <bool F32>
__device__ __forceinline__ void store4(void* p, int type, int64_t i, const float (&v)[4]) {
    if constexpr (F32) {
        *reinterpret_cast<float4*>(static_cast<float*>(p) + i) = make_float4(v[0], v[1], v[2], v[3]);
    } else {
        const uint2 w = type == BITSMOE_F16 ? make_uint2(pack2<true>(v[0], v[1]), pack2<true>(v[2], v[3]))
                                            : make_uint2(pack2<false>(v[0], v[1]), pack2<false>(v[2], v[3]));
        *reinterpret_cast<uint2*>(static_cast<uint16_t*>(p) + i) = w;
    }
}

// V neighbouring elements, one by one, from element i of p on.
template <int V>
__device__ __forceinline__ void load_elems(const void* p, int type, int64_t i, float (&v)[V]) {
#pragma unroll
    for (int j = 0; j < V; j++)
        v[j] = type == BITSMOE_F32 ? static_cast<const float*>(p)[i + j]
                                   : half_bits(static_cast<const uint16_t*>(p)[i + j], type);
}
template <int V>
__device__ __forceinline__ void store_elems(void* p, int type, int64_t i, const float (&v)[V]) {
#pragma unroll
    for (int j = 0; j < V; j++) {
        if (type == BITSMOE_F32)
            static_cast<float*>(p)[i + j] = v[j];
        else
            static_cast<uint16_t*>(p)[i + j] = (uint16_t)to_half_bits(v[j], type);
    }
}

// SiLU.  The approximate division (2 units of the last place) has no branch; its denominator is
// at least 1, and it gives 0 where that leaves the range (v below about -88).
__device__ __forceinline__ float silu_f(float v) { return __fdividef(v, 1.0f + expf(-v)); }

// Inclusive scan over a CTA of THREADS threads, one value each; s_warp [32].
template <int THREADS>
__device__ __forceinline__ int cta_scan(int v, int* s_warp) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int u = __shfl_up_sync(0xffffffffu, v, o);
        if (lane >= o) v += u;
    }
    if (lane == 31) s_warp[warp] = v;
    __syncthreads();
    if (warp == 0) {
        int w = lane < THREADS / 32 ? s_warp[lane] : 0;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int u = __shfl_up_sync(0xffffffffu, w, o);
            if (lane >= o) w += u;
        }
        s_warp[lane] = w;
    }
    __syncthreads();
    if (warp > 0) v += s_warp[warp - 1];
    __syncthreads();
    return v;
}

// A bounded wait of a whole warp on an mbarrier phase; every lane gets the same answer.
// The clock is read once in 64 tries.
constexpr long long kWarpWaitNs = 2000000000LL;  // 2 s, then BITSMOE_ST_TIMEOUT
__device__ __forceinline__ bool warp_wait(uint32_t bar, uint32_t parity) {
    long long t0 = 0;
    for (int i = 1;; i++) {
        uint32_t ok;
        asm volatile(
            "{\n .reg .pred p;\n mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n selp.u32 %0, 1, 0, p;\n}\n"
            : "=r"(ok)
            : "r"(bar), "r"(parity)
            : "memory");
        if (__all_sync(0xffffffffu, ok)) return true;
        if (i % 64 == 0) {
            long long t;
            asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(t));
            t = __shfl_sync(0xffffffffu, t, 0);
            if (t0 == 0)
                t0 = t;
            else if (t - t0 > kWarpWaitNs)
                return false;
        }
    }
}

// Programmatic dependent launch: the wait returns when every kernel before this one
// in the stream has finished and its writes are visible; the trigger lets the next
// kernel (if it was launched the same way) start its own pre-wait part.
__device__ __forceinline__ void pdl_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void pdl_trigger() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

template <typename... KArgs, typename... Args>
inline int launch_pdl(void (*kernel)(KArgs...), dim3 grid, dim3 block, size_t smem, cudaStream_t s, Args&&... args) {
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = grid;
    cfg.blockDim = block;
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, std::forward<Args>(args)...);
    return e == cudaSuccess ? BITSMOE_OK : set_cuda_error(e);
}

}  // namespace bitsmoe
