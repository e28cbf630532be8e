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
// 24.5 M parameters in 64 tensors with 8-bit states take 86 us (a launch by
// itself, which ends with 57 of its 441 MB still to leave L2; the floor is
// 67.6), now bound by the 66 instructions of an element: IEEE
// roots and divisions for every code took 132 us, and a lane's eight values
// side by side (16-byte halves of the same sectors) instead of in two runs
// made the decoding of a state 32 instead of 22 us.
#pragma once

#include <type_traits>

#include "../../include/ft.h"
#include "ft_ptx.cuh"
#include "ft_vec.cuh"

namespace ft {
namespace adamw {

constexpr int kBlock = 256;  // elements that share a scale; a warp's at a time, eight per lane
constexpr int kWarps = 8;
constexpr int kUnit = kBlock * kWarps;  // elements that a block of threads takes at a time, within one tensor
constexpr int kPerSm = 5;               // blocks of threads that an SM holds

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
    int g16, vec, usual;
};
template <int kMax>
struct Params {
    int count, last;  // last: this launch ends the step
    unsigned units;
    bool exact;  // eps does not cover what the fast division leaves out
    float b1, c1, b2, c2, eps;  // c = 1 - b, rounded from double
    double lr, log_b1, log_b2;
    const float* lr_dev;
    const float* grad_scale;
    long long* step;
    Tensor t[kMax];
};

// A byte of w as the float 2^23 + byte: its bits are the byte under the
// exponent of 2^23.
__device__ __forceinline__ float byte_as_float(uint32_t w, int i) {
    return __uint_as_float(__byte_perm(w, 0x4B000000u, 0x7650u | (uint32_t)i));
}
// The values of the codes in bytes i, i + 1 of w (m: two's complement, v:
// unsigned).
__device__ __forceinline__ float2 decode_m(uint32_t w, int i, float top) {
    w ^= 0x80808080u;  // 2^23 + (c + 128), exact
    const float2 c = add2(make_float2(byte_as_float(w, i), byte_as_float(w, i + 1)), both(-8388736.0f));
    const float2 q = mul2(c, make_float2(fabsf(c.x), fabsf(c.y)));
    return mul2(mul2(q, both(1.0f / 16129.0f)), both(top));
}
__device__ __forceinline__ float2 decode_v(uint32_t w, int i, float top) {
    const float2 c = add2(make_float2(byte_as_float(w, i), byte_as_float(w, i + 1)), both(-8388608.0f));
    const float2 r = mul2(mul2(c, c), both(1.0f / 65025.0f));
    return mul2(mul2(r, r), both(top));
}
__device__ __forceinline__ float recip_top(float top) { return top >= 1.17549435e-38f ? __frcp_rn(top) : 0.0f; }

// Codes as defined: every step rounded once.
__device__ __forceinline__ float scaled_m(float m, float inv) {
    return copysignf(__fmul_rn(__fsqrt_rn(__fmul_rn(fabsf(m), inv)), 127.0f), m);
}
__device__ __forceinline__ float scaled_v(float v, float inv) {
    return __fmul_rn(__fsqrt_rn(__fsqrt_rn(__fmul_rn(v, inv))), 255.0f);
}
// Hardware square root and reciprocal: to 2^-23, 0 (infinity) for what is
// below 2^-126.
__device__ __forceinline__ float2 sqrt_near(float2 x) {
    asm("sqrt.approx.ftz.f32 %0, %0;" : "+f"(x.x));
    asm("sqrt.approx.ftz.f32 %0, %0;" : "+f"(x.y));
    return x;
}
__device__ __forceinline__ float2 recip_near(float2 x) {
    asm("rcp.approx.ftz.f32 %0, %0;" : "+f"(x.x));
    asm("rcp.approx.ftz.f32 %0, %0;" : "+f"(x.y));
    return x;
}
// With hardware square roots the scaled values are off by less than kNear:
// m's, up to 127, by one root, the defined root's own rounding and two
// products' (2.5 2^-23 127 = 3.8e-5), v's, up to 255, by two roots, the second
// halving the first's error (3.3 2^-23 255 = 1.0e-4).  Where a value is that
// close to the border of two codes, the lane's eight are taken by the
// definition (one warp in fourteen has one).
constexpr float kNear = 1.25e-4f;

// Adding 1.5 2^23 rounds to the nearest integer (ties to even) and leaves it
// in the low byte, negative ones in two's complement.  `edge` grows to the
// largest distance from the integer.
__device__ __forceinline__ float2 rounded(float2 t, float& edge) {
    const float2 r = add2(t, both(12582912.0f));
    const float2 n = add2(r, both(-12582912.0f));
    const float2 d = fma2(n, both(-1.0f), t);
    edge = fmaxf(edge, fmaxf(fabsf(d.x), fabsf(d.y)));
    return r;
}
__device__ __forceinline__ uint32_t low_bytes(float2 a, float2 b) {
    return __byte_perm(__byte_perm(__float_as_uint(a.x), __float_as_uint(a.y), 0x0040),
                       __byte_perm(__float_as_uint(b.x), __float_as_uint(b.y), 0x0040), 0x5410);
}
template <bool kSecond>
__device__ __noinline__ uint2 codes_defined(float2 a, float2 b, float2 c, float2 d, float inv) {
    float2 t[4] = {a, b, c, d};
    float edge = 0.0f;
    for (int i = 0; i < 4; ++i) {
        t[i] = kSecond ? make_float2(scaled_v(t[i].x, inv), scaled_v(t[i].y, inv))
                       : make_float2(scaled_m(t[i].x, inv), scaled_m(t[i].y, inv));
        t[i] = rounded(t[i], edge);
    }
    return make_uint2(low_bytes(t[0], t[1]), low_bytes(t[2], t[3]));
}
template <bool kSecond>
__device__ __forceinline__ uint2 codes(const float2 (&x)[4], float inv, bool defined) {
    float2 t[4];
    float edge = 0.0f;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if (kSecond) {
            t[i] = mul2(sqrt_near(sqrt_near(mul2(x[i], both(inv)))), both(255.0f));
        } else {
            t[i] = mul2(sqrt_near(mul2(make_float2(fabsf(x[i].x), fabsf(x[i].y)), both(inv))), both(127.0f));
            t[i] = make_float2(copysignf(t[i].x, x[i].x), copysignf(t[i].y, x[i].y));
        }
        t[i] = rounded(t[i], edge);
    }
    if (defined || !(edge < 0.5f - kNear)) return codes_defined<kSecond>(x[0], x[1], x[2], x[3], inv);
    return make_uint2(low_bytes(t[0], t[1]), low_bytes(t[2], t[3]));
}

// The sum of two products that were each rounded: a two-lane sum would be
// contracted with the two-lane product before it.
__device__ __forceinline__ float2 sum_of(float2 a, float2 b) {
    return make_float2(__fadd_rn(a.x, b.x), __fadd_rn(a.y, b.y));
}

// A lane's eight values of a block: 4 l .. 4 l + 3 and the same 128 further,
// so that every access of a warp is one run of bytes whatever the type.  at:
// the lane's first; vec: all are there and aligned, else those before `left`.
constexpr int kHalf = kBlock / 2;
__device__ __forceinline__ bool there(int i, int left) { return (i & 3) + (i >> 2) * kHalf < left; }
__device__ __forceinline__ void load_pairs(float2 (&f)[4], const float* at, bool vec, int left) {
    if (vec) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const uint4 r = ld_stream_v4(at + h * kHalf);
            f[2 * h] = make_float2(__uint_as_float(r.x), __uint_as_float(r.y));
            f[2 * h + 1] = make_float2(__uint_as_float(r.z), __uint_as_float(r.w));
        }
    } else {
        float t[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) t[i] = there(i, left) ? at[(i & 3) + (i >> 2) * kHalf] : 0.0f;
#pragma unroll
        for (int i = 0; i < 4; ++i) f[i] = make_float2(t[2 * i], t[2 * i + 1]);
    }
}
__device__ __forceinline__ void load_pairs(float2 (&f)[4], const __nv_bfloat16* at, bool vec, int left) {
    if (vec) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const uint2 r = ld_stream_v2(at + h * kHalf);
            f[2 * h] = make_float2(bf16_lo(r.x), bf16_hi(r.x));
            f[2 * h + 1] = make_float2(bf16_lo(r.y), bf16_hi(r.y));
        }
    } else {
        float t[8];
#pragma unroll
        for (int i = 0; i < 8; ++i)
            t[i] = there(i, left) ? __bfloat162float(at[(i & 3) + (i >> 2) * kHalf]) : 0.0f;
#pragma unroll
        for (int i = 0; i < 4; ++i) f[i] = make_float2(t[2 * i], t[2 * i + 1]);
    }
}
__device__ __forceinline__ void put_quad(float* p, float2 a, float2 b) {
    *reinterpret_cast<float4*>(p) = make_float4(a.x, a.y, b.x, b.y);
}
__device__ __forceinline__ void put_quad(__nv_bfloat16* p, float2 a, float2 b) {
    *reinterpret_cast<uint2*>(p) = make_uint2(pack_bf16(a.x, a.y), pack_bf16(b.x, b.y));
}
template <typename T>
__device__ __forceinline__ void store_pairs(T* at, const float2 (&f)[4], bool vec, int left) {
    if (vec) {
        put_quad(at, f[0], f[1]);
        put_quad(at + kHalf, f[2], f[3]);
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (there(i, left)) at[(i & 3) + (i >> 2) * kHalf] = (T)(i & 1 ? f[i >> 1].y : f[i >> 1].x);
    }
}
__device__ __forceinline__ uint2 load_codes(const uint8_t* at, bool vec, int left) {
    if (vec) return make_uint2(*reinterpret_cast<const uint32_t*>(at), *reinterpret_cast<const uint32_t*>(at + kHalf));
    uint32_t w[2] = {0, 0};
#pragma unroll
    for (int i = 0; i < 8; ++i)
        if (there(i, left)) w[i >> 2] |= (uint32_t)at[(i & 3) + (i >> 2) * kHalf] << (8 * (i & 3));
    return make_uint2(w[0], w[1]);
}
__device__ __forceinline__ void store_codes(uint8_t* at, uint2 c, bool vec, int left) {
    if (vec) {
        *reinterpret_cast<uint32_t*>(at) = c.x;
        *reinterpret_cast<uint32_t*>(at + kHalf) = c.y;
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (there(i, left)) at[(i & 3) + (i >> 2) * kHalf] = (uint8_t)((i < 4 ? c.x : c.y) >> (8 * (i & 3)));
    }
}

template <bool k8, int kMax>
__global__ void __launch_bounds__(32 * kWarps, kPerSm) k_adamw(const __grid_constant__ Params<kMax> p) {
    __shared__ float coef[2];
    grid_dep_launch();
    grid_dep_wait();
    const float gs = p.grad_scale ? *p.grad_scale : 1.0f;
    const double lr = p.lr_dev ? (double)*p.lr_dev : p.lr;
    if (threadIdx.x == 0) {
        // 1 - b^t by expm1, which does not cancel for small t; the exponent
        // is formed in FP64 (FP64 expm1 too would hold every block back by
        // 3 us)
        const double t = (double)(*p.step + 1);
        coef[0] = (float)lr / -expm1f((float)(t * p.log_b1));
        coef[1] = 1.0f / sqrtf(-expm1f((float)(t * p.log_b2)));
    }
    __syncthreads();
    const float rate = coef[0], rc2 = coef[1];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    int tensor = 0;
    for (unsigned unit = blockIdx.x; unit < p.units; unit += gridDim.x) {
        while (tensor + 1 < p.count && p.t[tensor + 1].first <= unit) ++tensor;
        const Tensor& T = p.t[tensor];
        const long long n = T.n;
        const long long block = (long long)(unit - T.first) * kWarps + warp;
        if (block * kBlock >= n) continue;
        const long long at = block * kBlock + lane * 4;
        const int live = (int)max(0ll, min((long long)kBlock, n - at));  // of the block from this lane's first on
        const float decay = (float)(1.0 - lr * (double)T.wd);
        // kUsual: FP32 masters with a bf16 copy and FP32 gradients, all there
        // and aligned, known to the compiler
        auto step = [&](auto usual) {
            constexpr bool kUsual = decltype(usual)::value;
            const bool vec = kUsual || (T.vec && live >= kHalf + 4);
            const bool g16 = !kUsual && T.g16, has_p = kUsual || T.p, has_16 = kUsual || T.p16;
            float2 g[4], w[4], m[4], v[4];
            float mtop = 0.0f, vtop = 0.0f;
            if (g16)
                load_pairs(g, static_cast<const __nv_bfloat16*>(T.g) + at, vec, live);
            else
                load_pairs(g, static_cast<const float*>(T.g) + at, vec, live);
            if (has_p)
                load_pairs(w, T.p + at, vec, live);
            else
                load_pairs(w, T.p16 + at, vec, live);
            if (k8) {
                mtop = T.ms[block];
                vtop = T.vs[block];
                const uint2 a = load_codes(static_cast<const uint8_t*>(T.m) + at, vec, live);
                const uint2 b = load_codes(static_cast<const uint8_t*>(T.v) + at, vec, live);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    m[i] = decode_m(i < 2 ? a.x : a.y, 2 * (i & 1), mtop);
                    v[i] = decode_v(i < 2 ? b.x : b.y, 2 * (i & 1), vtop);
                }
            } else {
                load_pairs(m, static_cast<const float*>(T.m) + at, vec, live);
                load_pairs(v, static_cast<const float*>(T.v) + at, vec, live);
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                g[i] = mul2(g[i], both(gs));
                m[i] = sum_of(mul2(m[i], both(p.b1)), mul2(g[i], both(p.c1)));
                v[i] = sum_of(mul2(v[i], both(p.b2)), mul2(mul2(g[i], both(p.c2)), g[i]));
                // hardware root and reciprocal, 2^-23 each: a few 2^-23 of the
                // step, below the weight's own rounding unless the weight is
                // small next to its step (a factor that starts at zero).  IEEE
                // root and division took 138.6 instead of 135.7 us for the
                // stack above with its decodings, 95.5 instead of 82.6 for
                // bf16 weights without master, 6.2 instead of 5.4 for two small
                // tensors.  A subnormal v counts as zero next to eps
                float2 u = mul2(m[i], recip_near(fma2(sqrt_near(v[i]), both(rc2), both(p.eps))));
                if (p.exact)
                    u = make_float2(m[i].x / fmaf(sqrtf(v[i].x), rc2, p.eps), m[i].y / fmaf(sqrtf(v[i].y), rc2, p.eps));
                w[i] = fma2(u, both(-rate), mul2(w[i], both(decay)));
            }
            if (has_p) store_pairs(T.p + at, w, vec, live);
            if (has_16) store_pairs(T.p16 + at, w, vec, live);
            if (k8) {
                // magnitudes order like their bits, NaN above infinity; what
                // is not there is zero
                uint32_t mb = 0, vb = 0;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    mb = max(mb, max(__float_as_uint(m[i].x) & 0x7FFFFFFFu, __float_as_uint(m[i].y) & 0x7FFFFFFFu));
                    vb = max(vb, max(__float_as_uint(v[i].x) & 0x7FFFFFFFu, __float_as_uint(v[i].y) & 0x7FFFFFFFu));
                }
                mb = __reduce_max_sync(0xFFFFFFFFu, mb);
                vb = __reduce_max_sync(0xFFFFFFFFu, vb);
                // a non-finite block: no code can stand for its values
                const bool bad = max(mb, vb) >= 0x7F800000u;
                mtop = __uint_as_float(mb >= 0x7F800000u ? 0x7FC00000u : mb);
                vtop = __uint_as_float(vb >= 0x7F800000u ? 0x7FC00000u : vb);
                const uint2 cm = codes<false>(m, recip_top(mtop), bad);
                const uint2 cv = codes<true>(v, recip_top(vtop), bad);
                store_codes(static_cast<uint8_t*>(T.m) + at, cm, vec, live);
                store_codes(static_cast<uint8_t*>(T.v) + at, cv, vec, live);
                if (lane == 0) {
                    T.ms[block] = mtop;
                    T.vs[block] = vtop;
                }
            } else {
                store_pairs(static_cast<float*>(T.m) + at, m, vec, live);
                store_pairs(static_cast<float*>(T.v) + at, v, vec, live);
            }
        };
        if (T.usual && block * kBlock + kBlock <= n)  // uniform over the warp
            step(std::true_type());
        else
            step(std::false_type());
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

// A block of codes per warp at a time, four of them in flight.
__global__ void __launch_bounds__(256) k_adamw_decode(const uint8_t* codes, const float* scales, long long n,
                                                      int second, float* out, int aligned) {
    constexpr int U = 4;
    const int lane = threadIdx.x & 31;
    grid_dep_launch();
    grid_dep_wait();
    const long long blocks = (n + kBlock - 1) / kBlock, step = (long long)gridDim.x * (blockDim.x >> 5);
    for (long long b = (long long)blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5); b < blocks; b += U * step) {
        uint2 c[U];
        float top[U];
        int live[U];
        bool vec[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const long long at = (b + u * step) * kBlock + lane * 4;
            live[u] = (int)max(0ll, min((long long)kBlock, n - at));
            vec[u] = aligned && live[u] >= kHalf + 4;
            if (b + u * step < blocks) {
                c[u] = load_codes(codes + at, vec[u], live[u]);
                top[u] = __ldg(scales + b + u * step);
            }
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (b + u * step >= blocks) break;
            float2 f[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const uint32_t w = k < 2 ? c[u].x : c[u].y;
                f[k] = second ? decode_v(w, 2 * (k & 1), top[u]) : decode_m(w, 2 * (k & 1), top[u]);
            }
            store_pairs(out + (b + u * step) * kBlock + lane * 4, f, vec[u], live[u]);
        }
    }
}

}  // namespace adamw
}  // namespace ft
