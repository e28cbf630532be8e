// k_adamw.cuh -- one AdamW step over many tensors.
//
//     m = b1 m + (1 - b1) g,  v = b2 v + (1 - b2) g^2
//     p = p (1 - lr wd) - lr / (1 - b1^t) m / (sqrt(v / (1 - b2^t)) + eps)
//
// Eight-bit states hold, per block of 256 elements with top = its largest
// |m| (v):  m ~ sign (c / 127)^2 top,  v ~ (c / 255)^4 top.  Every step
// between a stored state and the next is one IEEE FP32 operation without
// contraction, so the codes are the same wherever they are computed.
//
// HBM bounds it: 30 B per element with FP32 states (p, m, v read and
// written, g read, the bf16 copy written), 18 B with 8-bit ones.  The tensor
// list travels in the launch's parameters, so one launch serves all tensors,
// a captured step owns its list, and nothing is copied to the device first.
#pragma once

#include "../../include/ft.h"
#include "ft_ptx.cuh"
#include "ft_vec.cuh"

namespace ft {
namespace adamw {

constexpr int kBlock = 256;            // elements that share a scale
constexpr int kWarps = 8;
constexpr int kUnit = kBlock * kWarps;  // elements of one turn of a block of threads

struct Tensor {
    float* p;
    __nv_bfloat16* p16;
    const void* g;
    void* m;
    void* v;
    float* ms;
    float* vs;
    long long n;
    float wd;
    unsigned first;  // units before this tensor
    int g16, vec;
};
template <int kMax>
struct Params {
    int count, last;  // last: this launch ends the step
    unsigned units;
    float b1, c1, b2, c2, eps;  // c = 1 - b, rounded from double
    double lr, log_b1, log_b2;
    const float* lr_dev;
    const float* grad_scale;
    long long* step;
    Tensor t[kMax];
};

__device__ __forceinline__ float decode_m(int c, float top) {
    return __fmul_rn(__fmul_rn((float)(c * abs(c)), 1.0f / 16129.0f), top);
}
__device__ __forceinline__ float decode_v(int c, float top) {
    const float r = __fmul_rn((float)(c * c), 1.0f / 65025.0f);
    return __fmul_rn(__fmul_rn(r, r), top);
}
__device__ __forceinline__ float recip_top(float top) { return top >= 1.17549435e-38f ? __frcp_rn(top) : 0.0f; }
__device__ __forceinline__ int encode_m(float m, float inv) {
    const int c = __float2int_rn(__fmul_rn(__fsqrt_rn(__fmul_rn(fabsf(m), inv)), 127.0f));
    return m < 0.0f ? -c : c;
}
__device__ __forceinline__ int encode_v(float v, float inv) {
    return __float2int_rn(__fmul_rn(__fsqrt_rn(__fsqrt_rn(__fmul_rn(v, inv))), 255.0f));
}
// the largest of a and b, NaN if one of them is
__device__ __forceinline__ float max_nan(float a, float b) { return a != a || a > b ? a : b; }

template <bool k8, int kMax>
__global__ void __launch_bounds__(32 * kWarps) k_adamw(const __grid_constant__ Params<kMax> p) {
    __shared__ float coef[2];
    grid_dep_wait();
    const float gs = p.grad_scale ? *p.grad_scale : 1.0f;
    const double lr = p.lr_dev ? (double)*p.lr_dev : p.lr;
    if (threadIdx.x == 0) {
        // 1 - b^t in FP64: it cancels for small t
        const double t = (double)(*p.step + 1);
        coef[0] = (float)(lr / -expm1(t * p.log_b1));
        coef[1] = (float)rsqrt(-expm1(t * p.log_b2));
    }
    __syncthreads();
    const float rate = coef[0], rc2 = coef[1];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    for (unsigned unit = blockIdx.x; unit < p.units; unit += gridDim.x) {
        // the last tensor whose first unit is not above this one
        int lo = 0, hi = p.count - 1;
        while (lo < hi) {
            const int mid = (lo + hi + 1) >> 1;
            if (p.t[mid].first <= unit)
                lo = mid;
            else
                hi = mid - 1;
        }
        const Tensor& T = p.t[lo];
        const long long block = (long long)(unit - T.first) * kWarps + warp;
        const long long at = block * kBlock + lane * 8;
        if (block * kBlock >= T.n) continue;
        const int live = (int)max(0ll, min(8ll, T.n - at));
        const bool vec = T.vec && live == 8;
        float g[8] = {}, w[8] = {}, m[8] = {}, v[8] = {};
        float mtop = 0.0f, vtop = 0.0f;
        if (k8) {
            mtop = T.ms[block];
            vtop = T.vs[block];
        }
        if (vec) {
            if (T.g16) {
                unpack8(ld_stream_v4(static_cast<const __nv_bfloat16*>(T.g) + at), g);
            } else {
                Raw8<float> r;
                load8(r, static_cast<const float*>(T.g) + at);
                unpack8(r, g);
            }
            if (T.p) {
                Raw8<float> r;
                load8(r, T.p + at);
                unpack8(r, w);
            } else {
                unpack8(ld_stream_v4(T.p16 + at), w);
            }
            if (k8) {
                const uint2 a = *reinterpret_cast<const uint2*>(static_cast<const uint8_t*>(T.m) + at);
                const uint2 b = *reinterpret_cast<const uint2*>(static_cast<const uint8_t*>(T.v) + at);
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    m[i] = decode_m((int)(int8_t)((i < 4 ? a.x : a.y) >> (8 * (i & 3))), mtop);
                    v[i] = decode_v((int)(((i < 4 ? b.x : b.y) >> (8 * (i & 3))) & 255u), vtop);
                }
            } else {
                Raw8<float> r;
                load8(r, static_cast<const float*>(T.m) + at);
                unpack8(r, m);
                load8(r, static_cast<const float*>(T.v) + at);
                unpack8(r, v);
            }
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                if (i >= live) continue;
                g[i] = T.g16 ? __bfloat162float(static_cast<const __nv_bfloat16*>(T.g)[at + i])
                             : static_cast<const float*>(T.g)[at + i];
                w[i] = T.p ? T.p[at + i] : __bfloat162float(T.p16[at + i]);
                m[i] = k8 ? decode_m(static_cast<const int8_t*>(T.m)[at + i], mtop)
                          : static_cast<const float*>(T.m)[at + i];
                v[i] = k8 ? decode_v(static_cast<const uint8_t*>(T.v)[at + i], vtop)
                          : static_cast<const float*>(T.v)[at + i];
            }
        }
        const float decay = (float)(1.0 - lr * (double)T.wd);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float gi = __fmul_rn(g[i], gs);
            m[i] = __fadd_rn(__fmul_rn(m[i], p.b1), __fmul_rn(gi, p.c1));
            v[i] = __fadd_rn(__fmul_rn(v[i], p.b2), __fmul_rn(__fmul_rn(gi, p.c2), gi));
            w[i] = fmaf(-rate, __fdiv_rn(m[i], fmaf(__fsqrt_rn(v[i]), rc2, p.eps)), w[i] * decay);
        }
        uint2 cm = make_uint2(0, 0), cv = make_uint2(0, 0);
        if (k8) {
            mtop = vtop = 0.0f;
#pragma unroll
            for (int i = 0; i < 8; ++i)
                if (i < live) {
                    mtop = max_nan(fabsf(m[i]), mtop);
                    vtop = max_nan(v[i], vtop);
                }
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) {
                mtop = max_nan(__shfl_xor_sync(0xFFFFFFFFu, mtop, o), mtop);
                vtop = max_nan(__shfl_xor_sync(0xFFFFFFFFu, vtop, o), vtop);
            }
            // a non-finite block: no code can stand for its values
            const float bad = __int_as_float(0x7FC00000);
            if (!(mtop <= 3.4028234e38f)) mtop = bad;
            if (!(vtop <= 3.4028234e38f)) vtop = bad;
            const float mi = recip_top(mtop), vi = recip_top(vtop);
            uint32_t am[2] = {0, 0}, av[2] = {0, 0};
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                am[i >> 2] |= (uint32_t)(uint8_t)encode_m(m[i], mi) << (8 * (i & 3));
                av[i >> 2] |= (uint32_t)(uint8_t)encode_v(v[i], vi) << (8 * (i & 3));
            }
            cm = make_uint2(am[0], am[1]);
            cv = make_uint2(av[0], av[1]);
            if (lane == 0) {
                T.ms[block] = mtop;
                T.vs[block] = vtop;
            }
        }
        if (vec) {
            if (T.p) store8(T.p + at, w);
            if (T.p16) store8(T.p16 + at, w);
            if (k8) {
                *reinterpret_cast<uint2*>(static_cast<uint8_t*>(T.m) + at) = cm;
                *reinterpret_cast<uint2*>(static_cast<uint8_t*>(T.v) + at) = cv;
            } else {
                store8(static_cast<float*>(T.m) + at, m);
                store8(static_cast<float*>(T.v) + at, v);
            }
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                if (i >= live) continue;
                if (T.p) T.p[at + i] = w[i];
                if (T.p16) T.p16[at + i] = __float2bfloat16_rn(w[i]);
                if (k8) {
                    static_cast<uint8_t*>(T.m)[at + i] = (uint8_t)((i < 4 ? cm.x : cm.y) >> (8 * (i & 3)));
                    static_cast<uint8_t*>(T.v)[at + i] = (uint8_t)((i < 4 ? cv.x : cv.y) >> (8 * (i & 3)));
                } else {
                    static_cast<float*>(T.m)[at + i] = m[i];
                    static_cast<float*>(T.v)[at + i] = v[i];
                }
            }
        }
    }
    // The last block to get here has seen every block read the count: it
    // counts the step and leaves the arrival word as it found it.
    if (p.last) {
        __syncthreads();
        if (threadIdx.x == 0) {
            unsigned long long* word = reinterpret_cast<unsigned long long*>(p.step + 1);
            if (atomicAdd(word, 1ull) == gridDim.x - 1) {
                *word = 0;
                *p.step += 1;
            }
        }
    }
}

__global__ void __launch_bounds__(256) k_adamw_decode(const uint8_t* codes, const float* scales, long long n,
                                                      int second, float* out) {
    grid_dep_wait();
    for (long long i = (long long)blockIdx.x * blockDim.x + threadIdx.x; i < n; i += (long long)gridDim.x * blockDim.x) {
        const float top = __ldg(scales + i / kBlock);
        out[i] = second ? decode_v(codes[i], top) : decode_m((int8_t)codes[i], top);
    }
}

}  // namespace adamw
}  // namespace ft
