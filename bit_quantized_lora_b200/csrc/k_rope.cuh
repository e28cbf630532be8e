// k_rope.cuh -- rotary positions with several axes on the queries and keys
// of a QKV linear's output, with the RMS norm of each head before it, and
// their backward.
//
// A query or key head x [hd]:  n = x rstd w,  rstd = 1 / sqrt(mean(x^2) + eps),
// then its pairs (a, b) turn:  (a cos - b sin, b cos + a sin), pair j of row
// m by pos[m, axis(j)] freqs[j].  Backward: turn by the negative angle, then
//     dw = sum over rows and heads of d x rstd
//     dx = rstd (z - xh mean(z xh)),  z = d w, xh = x rstd
//
// The angle is formed in FP64 in turns and reduced by its nearest integer:
// p f / 2 pi carries 2^-53 of up to 2^31 turns, so what is left is exact to
// 2^-22 of a turn at the farthest position and to FP32 at a million.
//
// A row's cosines and sines are shared by all of its heads: a block takes a
// few rows, forms their table in shared memory and walks their heads, a
// power of two of lanes per head with eight values (four pairs) each.  HBM
// bounds both: 4 B per element of qkv (6 B backward with a norm).
#pragma once

#include "../../include/ft.h"
#include "ft_ptx.cuh"
#include "ft_vec.cuh"

namespace ft {
namespace rope {

constexpr int kThreads = 256;
constexpr int kRows = 4;      // rows of a block's table
constexpr int kMaxPairs = 128;
constexpr int kU = 4;         // heads in flight per thread

struct Heads {
    __nv_bfloat16* p;
    int64_t sb, sh, st;
};

struct Params {
    int M, S, Hq, Hk, hd, heads;  // heads: those walked (without the values when they are not copied)
    int rot, halves, norm, pos_f32, p32, n_axes;
    int axis_end[4];  // pairs up to and including axis a
    int lanes;        // per head
    float eps, inv_hd;
    const void* pos;
    const double* freqs;
    const void *w_q, *w_k;
    const __nv_bfloat16* x;  // qkv
    int64_t ld;
    __nv_bfloat16* dx;  // backward: dqkv
    int64_t lddx;
    Heads q, k, v;
    float* partial;  // backward: [blocks][2][hd], or null
    float* amax;
};

struct Table {
    float2 cs[kRows][kMaxPairs];  // (cos, sin); (1, 0) beyond the rotated pairs
    int b[kRows], s[kRows];       // sample and token of a row
};

__device__ __forceinline__ void fill_table(Table& tab, const Params& p, int row0, int rows, float sign) {
    const int pairs = p.lanes * 4;
    for (int i = threadIdx.x; i < rows * pairs; i += kThreads) {
        const int r = i / pairs, j = i - r * pairs;
        float2 cs = make_float2(1.0f, 0.0f);
        if (j < p.rot / 2) {
            int a = 0;
            while (a + 1 < p.n_axes && j >= p.axis_end[a]) ++a;
            const int64_t at = (int64_t)(row0 + r) * p.n_axes + a;
            const double pos = p.pos_f32 ? (double)static_cast<const float*>(p.pos)[at]
                                         : (double)static_cast<const int32_t*>(p.pos)[at];
            const double turns = pos * __ldg(p.freqs + j) * 0.15915494309189533577;
            float s, c;
            sincospif((float)(2.0 * (turns - rint(turns))), &s, &c);
            cs = make_float2(c, sign * s);
        }
        tab.cs[r][j] = cs;
    }
    if (threadIdx.x < rows) {
        const int m = row0 + threadIdx.x;
        tab.b[threadIdx.x] = m / p.S;
        tab.s[threadIdx.x] = m - m / p.S * p.S;
    }
}

// A lane's eight values of a head.  Pairs: 8 l .. 8 l + 7, pair i at (2i,
// 2i + 1).  Halves, below rot / 8: 4 l .. 4 l + 3 and the same behind rot / 2,
// pair i at (i, i + 4); above: 8 l .. 8 l + 7, not rotated.
struct Lane {
    int lo, hi;  // where the first and the second four values are
    bool on, split;
    __device__ Lane(const Params& p, int l) {
        on = 8 * l < p.hd;
        split = p.halves && 8 * l < p.rot;
        lo = split ? 4 * l : 8 * l;
        hi = split ? p.rot / 2 + 4 * l : 8 * l + 4;
    }
};

__device__ __forceinline__ uint4 load_lane(const __nv_bfloat16* head, const Lane& l) {
    if (!l.on) return make_uint4(0, 0, 0, 0);
    if (!l.split) return ld_stream_v4(head + l.lo);
    const uint2 a = *reinterpret_cast<const uint2*>(head + l.lo);
    const uint2 b = *reinterpret_cast<const uint2*>(head + l.hi);
    return make_uint4(a.x, a.y, b.x, b.y);
}
__device__ __forceinline__ void store_lane(__nv_bfloat16* head, const Lane& l, const uint4& v) {
    if (!l.on) return;
    if (!l.split) {
        *reinterpret_cast<uint4*>(head + l.lo) = v;
    } else {
        *reinterpret_cast<uint2*>(head + l.lo) = make_uint2(v.x, v.y);
        *reinterpret_cast<uint2*>(head + l.hi) = make_uint2(v.z, v.w);
    }
}

__device__ __forceinline__ void turn(float (&f)[8], const float2* cs, bool split) {
    float2 c[4];
#pragma unroll
    for (int i = 0; i < 4; i += 2) {
        const float4 w = *reinterpret_cast<const float4*>(cs + i);
        c[i] = make_float2(w.x, w.y);
        c[i + 1] = make_float2(w.z, w.w);
    }
    if (split) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float a = f[i], b = f[i + 4];
            f[i] = fmaf(a, c[i].x, -b * c[i].y);
            f[i + 4] = fmaf(b, c[i].x, a * c[i].y);
        }
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float a = f[2 * i], b = f[2 * i + 1];
            f[2 * i] = fmaf(a, c[i].x, -b * c[i].y);
            f[2 * i + 1] = fmaf(b, c[i].x, a * c[i].y);
        }
    }
}

__device__ __forceinline__ float head_sum(float v, int lanes) {
    for (int o = lanes >> 1; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
    return v;
}

__device__ __forceinline__ void head_weights(float (&w)[8], const void* p, bool f32, const Lane& l) {
#pragma unroll
    for (int i = 0; i < 8; ++i)
        w[i] = p && l.on ? load_param(p, i < 4 ? l.lo + i : l.hi + i - 4, f32) : 1.0f;
}

__device__ __forceinline__ __nv_bfloat16* head_of(const Params& p, const Table& tab, int r, int h) {
    const Heads& t = h < p.Hq ? p.q : h < p.Hq + p.Hk ? p.k : p.v;
    const int i = h < p.Hq ? h : h < p.Hq + p.Hk ? h - p.Hq : h - p.Hq - p.Hk;
    return t.p + tab.b[r] * t.sb + i * t.sh + tab.s[r] * t.st;
}

template <bool kBwd>
__global__ void __launch_bounds__(kThreads) k_qk_rope(const __grid_constant__ Params p) {
    __shared__ __align__(16) Table tab;
    __shared__ float red[32];
    const int group = threadIdx.x / p.lanes, groups = kThreads / p.lanes;
    const int l = threadIdx.x - group * p.lanes;
    const Lane lane(p, l);
    grid_dep_wait();
    float wq[8], wk[8];
    head_weights(wq, p.w_q, p.p32, lane);
    head_weights(wk, p.w_k, p.p32, lane);
    float dwq[8] = {}, dwk[8] = {};
    float amax = 0.0f;
    for (int row0 = blockIdx.x * kRows; row0 < p.M; row0 += gridDim.x * kRows) {
        const int rows = min(kRows, p.M - row0);
        __syncthreads();
        fill_table(tab, p, row0, rows, kBwd ? -1.0f : 1.0f);
        __syncthreads();
        // heads of the table's rows, in turn over the groups; blockIdx.y
        // shares them out further when there are few rows
        const int total = rows * p.heads, step = groups * gridDim.y;
        for (int first = blockIdx.y * groups; first < total; first += step * kU) {
            uint4 in[kU], ix[kU];
            int r[kU], h[kU];
#pragma unroll
            for (int u = 0; u < kU; ++u) {
                const int item = first + group + u * step;
                const bool live = item < total;
                r[u] = live ? item / p.heads : 0;
                h[u] = live ? item - r[u] * p.heads : -1;
                in[u] = ix[u] = make_uint4(0, 0, 0, 0);
                if (live) {
                    const __nv_bfloat16* x = p.x + (int64_t)(row0 + r[u]) * p.ld + h[u] * p.hd;
                    if (!kBwd) {
                        in[u] = load_lane(x, lane);
                    } else {
                        in[u] = load_lane(head_of(p, tab, r[u], h[u]), lane);
                        if (p.norm && h[u] < p.Hq + p.Hk) ix[u] = load_lane(x, lane);
                    }
                }
            }
#pragma unroll
            for (int u = 0; u < kU; ++u) {
                const bool turned = h[u] >= 0 && h[u] < p.Hq + p.Hk, isq = h[u] < p.Hq;
                float f[8];
                unpack8(in[u], f);
                if (!kBwd) {
                    if (p.norm) {
                        float q = 0.0f;
#pragma unroll
                        for (int i = 0; i < 8; ++i) q = fmaf(f[i], f[i], q);
                        const float rstd = 1.0f / sqrtf(fmaf(head_sum(q, p.lanes), p.inv_hd, p.eps));
                        if (turned) {
#pragma unroll
                            for (int i = 0; i < 8; ++i) f[i] *= rstd * (isq ? wq[i] : wk[i]);
                        }
                    }
                    if (turned) turn(f, &tab.cs[r[u]][4 * l], lane.split);
                    if (h[u] >= 0)
                        store_lane(head_of(p, tab, r[u], h[u]), lane, turned ? pack8(f) : in[u]);
                } else {
                    if (turned) turn(f, &tab.cs[r[u]][4 * l], lane.split);
                    if (p.norm) {
                        float x[8], q = 0.0f, z = 0.0f;
                        unpack8(ix[u], x);
#pragma unroll
                        for (int i = 0; i < 8; ++i) q = fmaf(x[i], x[i], q);
                        const float rstd = 1.0f / sqrtf(fmaf(head_sum(q, p.lanes), p.inv_hd, p.eps));
#pragma unroll
                        for (int i = 0; i < 8; ++i) {
                            x[i] *= rstd;
                            z = fmaf(f[i] * (isq ? wq[i] : wk[i]), x[i], z);
                        }
                        z = head_sum(z, p.lanes) * p.inv_hd;
                        if (turned) {
#pragma unroll
                            for (int i = 0; i < 8; ++i) {
                                if (isq)
                                    dwq[i] = fmaf(f[i], x[i], dwq[i]);
                                else
                                    dwk[i] = fmaf(f[i], x[i], dwk[i]);
                                f[i] = rstd * fmaf(-x[i], z, f[i] * (isq ? wq[i] : wk[i]));
                            }
                        }
                    }
                    if (h[u] >= 0) {
                        const uint4 v = turned ? pack8(f) : in[u];
                        store_lane(p.dx + (int64_t)(row0 + r[u]) * p.lddx + h[u] * p.hd, lane, v);
                        unpack8(v, f);
                        if (lane.on) amax = max_abs8(f, amax);
                    }
                }
            }
        }
    }
    if constexpr (kBwd) {
        raise_amax(p.amax, amax, red);
        if (p.partial) {
            // the groups' sums of a column, added in order
            float* buf = reinterpret_cast<float*>(&tab);
            static_assert(sizeof(Table) >= 4 * 8 * kThreads / 2, "half of the block's sums fit the table");
            float* out = p.partial + ((int64_t)blockIdx.y * gridDim.x + blockIdx.x) * 2 * p.hd;
            for (int k = 0; k < 2; ++k) {
                float s = 0.0f;
                for (int half = 0; half < 2; ++half) {
                    __syncthreads();
                    if (group / ((groups + 1) / 2) == half)
#pragma unroll
                        for (int i = 0; i < 8; ++i) {
                            const int at = (group - half * ((groups + 1) / 2)) * p.lanes * 8;
                            if (lane.on) buf[at + (i < 4 ? lane.lo + i : lane.hi + i - 4)] = k ? dwk[i] : dwq[i];
                        }
                    __syncthreads();
                    const int n = half ? groups - (groups + 1) / 2 : (groups + 1) / 2;
                    if (threadIdx.x < p.hd)
                        for (int g = 0; g < n; ++g) s += buf[g * p.lanes * 8 + threadIdx.x];
                }
                if (threadIdx.x < p.hd) out[k * p.hd + threadIdx.x] = s;
            }
        }
    }
}

// dw_q, dw_k from the blocks' partial sums: a warp per column.
__global__ void __launch_bounds__(256) k_qk_rope_reduce(const float* partial, int blocks, int hd, float* dw_q,
                                                        float* dw_k) {
    grid_dep_wait();
    const int c = blockIdx.x * 8 + (threadIdx.x >> 5), lane = threadIdx.x & 31;
    if (c >= 2 * hd) return;
    float s = 0.0f;
    for (int b = lane; b < blocks; b += 32) s += partial[(int64_t)b * 2 * hd + c];
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xFFFFFFFFu, s, o);
    float* out = c < hd ? dw_q : dw_k;
    if (lane == 0 && out) out[c < hd ? c : c - hd] = s;
}

}  // namespace rope
}  // namespace ft
