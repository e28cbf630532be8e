// ft_vec.cuh -- eight-element vectors of bf16 or FP32 rows, and reductions,
// for the streaming kernels around the linears.
#pragma once

#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

namespace ft {

// Eight consecutive elements as loaded: 16 bytes of bf16 or 32 of FP32.
template <typename T>
struct Raw8;
template <>
struct Raw8<__nv_bfloat16> {
    uint4 a;
};
template <>
struct Raw8<float> {
    uint4 a, b;
};

// Streamed rows are read once: they bypass L1, which keeps the vectors that
// every row reads.  Not the non-coherent path: an output may be in place.
__device__ __forceinline__ uint4 ld_stream_v4(const void* p) {
    uint4 v;
    asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "l"(p)
                 : "memory");
    return v;
}
__device__ __forceinline__ void load8(Raw8<__nv_bfloat16>& r, const __nv_bfloat16* p) { r.a = ld_stream_v4(p); }
__device__ __forceinline__ void load8(Raw8<float>& r, const float* p) {
    r.a = ld_stream_v4(p);
    r.b = ld_stream_v4(p + 4);
}

__device__ __forceinline__ float bf16_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }
__device__ __forceinline__ void unpack8(const uint4& v, float (&f)[8]) {
    f[0] = bf16_lo(v.x), f[1] = bf16_hi(v.x), f[2] = bf16_lo(v.y), f[3] = bf16_hi(v.y);
    f[4] = bf16_lo(v.z), f[5] = bf16_hi(v.z), f[6] = bf16_lo(v.w), f[7] = bf16_hi(v.w);
}
__device__ __forceinline__ void unpack8(const Raw8<__nv_bfloat16>& r, float (&f)[8]) { unpack8(r.a, f); }
__device__ __forceinline__ void unpack8(const Raw8<float>& r, float (&f)[8]) {
    f[0] = __uint_as_float(r.a.x), f[1] = __uint_as_float(r.a.y), f[2] = __uint_as_float(r.a.z);
    f[3] = __uint_as_float(r.a.w), f[4] = __uint_as_float(r.b.x), f[5] = __uint_as_float(r.b.y);
    f[6] = __uint_as_float(r.b.z), f[7] = __uint_as_float(r.b.w);
}

// Two floats to packed bf16, each rounded to nearest even, `lo` in the low half.
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
    uint32_t w;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(w) : "f"(hi), "f"(lo));
    return w;
}
__device__ __forceinline__ uint4 pack8(const float (&f)[8]) {
    return make_uint4(pack_bf16(f[0], f[1]), pack_bf16(f[2], f[3]), pack_bf16(f[4], f[5]), pack_bf16(f[6], f[7]));
}
// Stores eight values rounded to T and leaves them in f as stored.
__device__ __forceinline__ void store8(__nv_bfloat16* p, float (&f)[8]) {
    const uint4 v = pack8(f);
    *reinterpret_cast<uint4*>(p) = v;
    unpack8(v, f);
}
__device__ __forceinline__ void store8(float* p, float (&f)[8]) {
    *reinterpret_cast<float4*>(p) = make_float4(f[0], f[1], f[2], f[3]);
    *reinterpret_cast<float4*>(p + 4) = make_float4(f[4], f[5], f[6], f[7]);
}

// Eight values of a parameter vector (bf16 or FP32, 16-byte aligned), cached.
__device__ __forceinline__ void load_param8(const void* p, int64_t i, bool f32, float (&f)[8]) {
    if (f32) {
        const float4 a = __ldg(reinterpret_cast<const float4*>(static_cast<const float*>(p) + i));
        const float4 b = __ldg(reinterpret_cast<const float4*>(static_cast<const float*>(p) + i + 4));
        f[0] = a.x, f[1] = a.y, f[2] = a.z, f[3] = a.w, f[4] = b.x, f[5] = b.y, f[6] = b.z, f[7] = b.w;
    } else {
        unpack8(__ldg(reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(p) + i)), f);
    }
}
__device__ __forceinline__ float load_param(const void* p, int64_t i, bool f32) {
    return f32 ? __ldg(static_cast<const float*>(p) + i)
               : __bfloat162float(static_cast<const __nv_bfloat16*>(p)[i]);
}

__device__ __forceinline__ float max_abs8(const float (&f)[8], float m) {
#pragma unroll
    for (int i = 0; i < 8; ++i) m = fmaxf(m, fabsf(f[i]));
    return m;
}

// Raises *out to the block's largest m (all threads of the block call it;
// `red` holds a float per warp).  Non-negative floats order like their bits,
// so an integer max is exact and independent of the order of arrival; a block
// that would not raise the word sends no atomic.
__device__ __forceinline__ void raise_amax(float* out, float m, float* red) {
    if (!out) return;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, nw = (blockDim.x + 31) >> 5;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
    __syncthreads();  // red may still be read as something else
    if (lane == 0) red[warp] = m;
    __syncthreads();
    if (warp == 0) {
        m = lane < nw ? red[lane] : 0.0f;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
        if (lane == 0 && m > *reinterpret_cast<volatile float*>(out))
            atomicMax(reinterpret_cast<int*>(out), __float_as_int(m));
    }
}

}  // namespace ft
