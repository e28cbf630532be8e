// k_gelu_bwd.cuh -- the backward of GELU on bf16:
//
//     dy = dh GELU'(y),   GELU'(y) = Phi(y) + y phi(y)
//
// with Phi(y) = erfc(-y / sqrt 2) / 2, which keeps its relative accuracy for
// y << 0 (1 + erf would cancel).  The slope is FP32 and the product is
// rounded to bf16 once.
#pragma once

#include "ft_ptx.cuh"
#include "ft_vec.cuh"

namespace ft {
namespace gelub {

// GELU'(y).  From |y| = 16 on the slope is 1 or 0 to more than FP32 shows
// (y phi(y) < 2^-180 there, and its product with any bf16 underflows).
__device__ __forceinline__ float slope(float y) {
    if (fabsf(y) >= 16.0f) return y > 0.0f ? 1.0f : 0.0f;  // NaN goes on
    const float phi = __fmul_rn(0.39894228040143268f, expf(-0.5f * y * y));
    return fmaf(y, phi, 0.5f * erfcf(-0.70710678118654752f * y));
}

__global__ void __launch_bounds__(256) k_gelu_bwd_bf16(const __nv_bfloat16* y, const __nv_bfloat16* dh,
                                                       __nv_bfloat16* dy, int64_t n, float* amax_out) {
    __shared__ float red[32];
    grid_dep_wait();
    float amax = 0.0f;
    for (int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; i < n / 8;
         i += (int64_t)gridDim.x * blockDim.x) {
        float a[8], d[8];
        unpack8(ld_stream_v4(y + 8 * i), a);
        unpack8(ld_stream_v4(dh + 8 * i), d);
#pragma unroll
        for (int k = 0; k < 8; ++k) d[k] *= slope(a[k]);
        store8(dy + 8 * i, d);
        amax = max_abs8(d, amax);
    }
    raise_amax(amax_out, amax, red);
}

}  // namespace gelub
}  // namespace ft
