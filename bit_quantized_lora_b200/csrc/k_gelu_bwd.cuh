// k_gelu_bwd.cuh -- the backward of GELU on bf16:
//
//     dy = dh GELU'(y),   GELU'(y) = Phi(y) + y phi(y)
//
// with Phi(y) = erfc(-y / sqrt 2) / 2, which keeps its relative accuracy for
// y << 0 (1 + erf would cancel).  The slope is FP32 and the product is
// rounded to bf16 once.
//
// HBM bounds it, 6 B per element, once the slope is no longer computed per
// element: a bf16 y with 2^-12 <= |y| < 2^4 takes one of 4096 values, whose
// slopes each block tabulates first (16 KB of shared memory): 60 us for
// 4608 x 12288 values, 0.86 of the measured HBM rate, where computing every
// slope took 143 us.  Blocks that would tabulate more than they look up
// compute instead.
#pragma once

#include "ft_ptx.cuh"
#include "ft_vec.cuh"

namespace ft {
namespace gelub {

constexpr int kThreads = 1024;
constexpr int kTab = 4096;
constexpr int kU = 2;  // vectors of eight in flight per thread, of y and of dh

// GELU'(y).  From |y| = 16 on the slope is 1 or 0 to more than FP32 shows
// (y phi(y) < 2^-180 there, below the smallest subnormal); at the infinities
// these are its limits.
__device__ __forceinline__ float slope(float y) {
    if (fabsf(y) >= 16.0f) return y > 0.0f ? 1.0f : 0.0f;
    const float phi = __fmul_rn(0.39894228040143268f, expf(-0.5f * y * y));
    return fmaf(y, phi, 0.5f * erfcf(-0.70710678118654752f * y));  // NaN goes on
}

// Entry s << 11 | (e - 115) << 7 | m: the slope at the bf16 of sign s, biased
// exponent e (115 to 130) and mantissa m.
__device__ __forceinline__ void build(float* tab) {
    for (int i = threadIdx.x; i < kTab; i += blockDim.x)
        tab[i] = slope(__uint_as_float((uint32_t)(i >> 11) << 31 | (115u + ((uint32_t)i >> 7 & 15u)) << 23 |
                                       ((uint32_t)i & 127u) << 16));
}
__device__ __noinline__ float2 slope2_rare(uint32_t w) { return make_float2(slope(bf16_lo(w)), slope(bf16_hi(w))); }

// The slopes at two packed values.  Both exponents are offset by 141 within
// their own 16 bits, so that a value of the table's range lands in [256, 272);
// the indices are in range whatever the exponents.
__device__ __forceinline__ float2 slope2(uint32_t w, const float* tab) {
    const uint32_t v = ((w >> 7) & 0x00FF00FFu) + 0x008D008Du;
    const uint32_t i = ((w >> 4) & 0x08000800u) | ((v & 0x000F000Fu) << 7) | (w & 0x007F007Fu);
    float2 s = make_float2(tab[i & 0xFFFFu], tab[i >> 16]);
    if ((v & 0xFFF0FFF0u) != 0x01000100u) s = slope2_rare(w);
    return s;
}

template <bool kTable>
__global__ void __launch_bounds__(kThreads) k_gelu_bwd_bf16(const __nv_bfloat16* y, const __nv_bfloat16* dh,
                                                            __nv_bfloat16* dy, int64_t n, float* amax_out) {
    __shared__ float tab[kTable ? kTab : 1];
    __shared__ float red[32];
    if (kTable) build(tab);
    grid_dep_wait();
    const int64_t n8 = n / 8, stride = (int64_t)gridDim.x * blockDim.x;
    uint4 a[kU], d[kU];
    auto fetch = [&](int64_t i) {
#pragma unroll
        for (int u = 0; u < kU; ++u) {
            const int64_t j = i + u * stride;
            if (j < n8) {
                a[u] = ld_stream_v4(y + 8 * j);
                d[u] = ld_stream_v4(dh + 8 * j);
            }
        }
    };
    int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
    fetch(i);
    __syncthreads();
    uint32_t amax = 0;
    for (; i < n8; i += kU * stride) {
        uint4 ca[kU], cd[kU];
#pragma unroll
        for (int u = 0; u < kU; ++u) ca[u] = a[u], cd[u] = d[u];
        fetch(i + kU * stride);
#pragma unroll
        for (int u = 0; u < kU; ++u) {
            const int64_t j = i + u * stride;
            if (j >= n8) break;
            const uint32_t w[4] = {ca[u].x, ca[u].y, ca[u].z, ca[u].w};
            float f[8];
            unpack8(cd[u], f);
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const float2 s = kTable ? slope2(w[k], tab) : make_float2(slope(bf16_lo(w[k])), slope(bf16_hi(w[k])));
                f[2 * k] *= s.x;
                f[2 * k + 1] *= s.y;
            }
            amax = store8_max(dy + 8 * j, f, amax);
        }
    }
    raise_amax(amax_out, amax_of(amax), red);
}

}  // namespace gelub
}  // namespace ft
