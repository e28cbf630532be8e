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
__device__ __forceinline__ uint2 ld_stream_v2(const void* p) {
    uint2 v;
    asm volatile("ld.global.L1::no_allocate.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "l"(p) : "memory");
    return v;
}

__device__ __forceinline__ float bf16_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }
__device__ __forceinline__ void unpack8(const uint4& v, float (&f)[8]) {
    f[0] = bf16_lo(v.x), f[1] = bf16_hi(v.x), f[2] = bf16_lo(v.y), f[3] = bf16_hi(v.y);
    f[4] = bf16_lo(v.z), f[5] = bf16_hi(v.z), f[6] = bf16_lo(v.w), f[7] = bf16_hi(v.w);
}

// Asynchronous 16-byte copies into a thread's own shared-memory slots: what a
// thread copied it may read after its own wait, without a barrier.
__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async8(uint32_t dst, const void* src) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int kLeft>  // until at most kLeft of the thread's groups are in flight
__device__ __forceinline__ void cp_async_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(kLeft) : "memory");
}

// Pairs of floats as the two lanes of one instruction.
__device__ __forceinline__ unsigned long long bits2(float2 a) {
    return (unsigned long long)__float_as_uint(a.y) << 32 | __float_as_uint(a.x);
}
__device__ __forceinline__ float2 pair2(unsigned long long v) {
    return make_float2(__uint_as_float((uint32_t)v), __uint_as_float((uint32_t)(v >> 32)));
}
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
    unsigned long long d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(bits2(a)), "l"(bits2(b)), "l"(bits2(c)));
    return pair2(d);
}
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
    unsigned long long d;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(bits2(a)), "l"(bits2(b)));
    return pair2(d);
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
    unsigned long long d;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(bits2(a)), "l"(bits2(b)));
    return pair2(d);
}
__device__ __forceinline__ float2 both(float a) { return make_float2(a, a); }

// Eight values as four pairs.
struct F8 {
    float2 p[4];
};
__device__ __forceinline__ F8 widen(const uint4& v) {
    return {{make_float2(bf16_lo(v.x), bf16_hi(v.x)), make_float2(bf16_lo(v.y), bf16_hi(v.y)),
             make_float2(bf16_lo(v.z), bf16_hi(v.z)), make_float2(bf16_lo(v.w), bf16_hi(v.w))}};
}
__device__ __forceinline__ F8 widen(const Raw8<__nv_bfloat16>& r) { return widen(r.a); }
__device__ __forceinline__ F8 widen(const Raw8<float>& r) {
    return {{make_float2(__uint_as_float(r.a.x), __uint_as_float(r.a.y)),
             make_float2(__uint_as_float(r.a.z), __uint_as_float(r.a.w)),
             make_float2(__uint_as_float(r.b.x), __uint_as_float(r.b.y)),
             make_float2(__uint_as_float(r.b.z), __uint_as_float(r.b.w))}};
}
__device__ __forceinline__ F8 zero8() { return {{both(0.0f), both(0.0f), both(0.0f), both(0.0f)}}; }
__device__ __forceinline__ F8 mul(const F8& a, const F8& b) {
    return {{mul2(a.p[0], b.p[0]), mul2(a.p[1], b.p[1]), mul2(a.p[2], b.p[2]), mul2(a.p[3], b.p[3])}};
}
__device__ __forceinline__ F8 mul(const F8& a, float b) {
    const float2 c = both(b);
    return {{mul2(a.p[0], c), mul2(a.p[1], c), mul2(a.p[2], c), mul2(a.p[3], c)}};
}
__device__ __forceinline__ F8 add(const F8& a, const F8& b) {
    return {{add2(a.p[0], b.p[0]), add2(a.p[1], b.p[1]), add2(a.p[2], b.p[2]), add2(a.p[3], b.p[3])}};
}
__device__ __forceinline__ F8 add(const F8& a, float b) {
    const float2 c = both(b);
    return {{add2(a.p[0], c), add2(a.p[1], c), add2(a.p[2], c), add2(a.p[3], c)}};
}
__device__ __forceinline__ F8 fma(const F8& a, const F8& b, const F8& c) {
    return {{fma2(a.p[0], b.p[0], c.p[0]), fma2(a.p[1], b.p[1], c.p[1]), fma2(a.p[2], b.p[2], c.p[2]),
             fma2(a.p[3], b.p[3], c.p[3])}};
}
__device__ __forceinline__ F8 fma(const F8& a, float b, const F8& c) {
    const float2 d = both(b);
    return {{fma2(a.p[0], d, c.p[0]), fma2(a.p[1], d, c.p[1]), fma2(a.p[2], d, c.p[2]), fma2(a.p[3], d, c.p[3])}};
}
// a value's eight lanes added into a running pair
__device__ __forceinline__ float2 gather(float2 s, const F8& a) {
    return add2(s, add2(add2(a.p[0], a.p[1]), add2(a.p[2], a.p[3])));
}
__device__ __forceinline__ float2 gather(float2 s, const F8& a, const F8& b) {  // of products
    return fma2(a.p[3], b.p[3], fma2(a.p[2], b.p[2], fma2(a.p[1], b.p[1], fma2(a.p[0], b.p[0], s))));
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
__device__ __forceinline__ void put8(__nv_bfloat16* p, const Raw8<__nv_bfloat16>& r) {
    *reinterpret_cast<uint4*>(p) = r.a;
}
__device__ __forceinline__ void put8(float* p, const Raw8<float>& r) {
    *reinterpret_cast<uint4*>(p) = r.a;
    *reinterpret_cast<uint4*>(p + 4) = r.b;
}
// Rounds eight values to T as they would be loaded again.
__device__ __forceinline__ void round8(Raw8<__nv_bfloat16>& r, const F8& f) {
    r.a = make_uint4(pack_bf16(f.p[0].x, f.p[0].y), pack_bf16(f.p[1].x, f.p[1].y), pack_bf16(f.p[2].x, f.p[2].y),
                     pack_bf16(f.p[3].x, f.p[3].y));
}
__device__ __forceinline__ void round8(Raw8<float>& r, const F8& f) {
    r.a = make_uint4(__float_as_uint(f.p[0].x), __float_as_uint(f.p[0].y), __float_as_uint(f.p[1].x),
                     __float_as_uint(f.p[1].y));
    r.b = make_uint4(__float_as_uint(f.p[2].x), __float_as_uint(f.p[2].y), __float_as_uint(f.p[3].x),
                     __float_as_uint(f.p[3].y));
}
// Stores eight values as bf16 and raises the two lanes of m to the largest
// stored magnitudes.  m's lanes carry a sign that means nothing (amax_of drops
// it); NaN is passed over.
__device__ __forceinline__ uint32_t max_mag2(uint32_t m, uint32_t w) {
    uint32_t d;
    asm("max.xorsign.abs.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(m), "r"(w));
    return d;
}
__device__ __forceinline__ uint32_t max_mag8(uint32_t m, const uint4& v) {
    return max_mag2(max_mag2(m, v.x), max_mag2(max_mag2(v.y, v.z), v.w));
}
__device__ __forceinline__ float amax_of(uint32_t m) { return fmaxf(fabsf(bf16_lo(m)), fabsf(bf16_hi(m))); }
__device__ __forceinline__ uint32_t store8_max(__nv_bfloat16* p, const F8& f, uint32_t m) {
    Raw8<__nv_bfloat16> r;
    round8(r, f);
    *reinterpret_cast<uint4*>(p) = r.a;
    return max_mag8(m, r.a);
}
__device__ __forceinline__ uint32_t store8_max(__nv_bfloat16* p, const float (&f)[8], uint32_t m) {
    const uint4 v = pack8(f);
    *reinterpret_cast<uint4*>(p) = v;
    return max_mag8(m, v);
}

// Eight values of a parameter vector (bf16 or FP32, 16-byte aligned), cached.
template <bool k32>
__device__ __forceinline__ F8 load_param8(const void* p, int64_t i) {
    if constexpr (k32) {
        Raw8<float> r;
        r.a = __ldg(reinterpret_cast<const uint4*>(static_cast<const float*>(p) + i));
        r.b = __ldg(reinterpret_cast<const uint4*>(static_cast<const float*>(p) + i + 4));
        return widen(r);
    } else {
        return widen(__ldg(reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(p) + i)));
    }
}
__device__ __forceinline__ float load_param(const void* p, int64_t i, bool f32) {
    return f32 ? __ldg(static_cast<const float*>(p) + i)
               : __bfloat162float(static_cast<const __nv_bfloat16*>(p)[i]);
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
