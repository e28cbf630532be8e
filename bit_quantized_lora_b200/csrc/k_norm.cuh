// k_norm.cuh -- a block's boundary: gated residual and modulated norm, and
// their backward.
//
// Forward, row i of sample b (every reduction over the D channels):
//     u = y  or  N_post(y) w_post
//     r = x + alpha gate_b u                       stored as XT
//     h = (N_pre(r) w + bias)(1 + scale_b) + shift_b
// Backward, with xh = (r - mean) rstd, yh = (y - mean_y) rstd_y and
// z = dh (1 + scale_b) w:
//     d  = dr + rstd (z - xh mean(z xh) - mean(z))         (RMS: no mean(z))
//     e  = alpha gate_b w_post d
//     dy = rstd_y (e - yh mean(e yh) - mean(e))            (no post norm: e)
//     S0_b = sum dh,  S1_b = sum dh xh,  T_b = sum d yh    over b's rows
//     dshift = S0, dscale = w S1 + bias S0, dgate = alpha w_post T
//     dw = sum_b (1 + scale_b) S1_b, dbias = sum_b (1 + scale_b) S0_b,
//     dw_post = sum_b alpha gate_b T_b
//
// A row stays in registers between its one load and its one store, the
// variance is taken about the mean (no cancellation), and the next row's
// loads are in flight while a row is reduced.  HBM bounds both kernels: 8 B
// per element forward (x, y, r, h in bf16), 12 B backward (dh, dr, r, y, dx,
// dy).
#pragma once

#include "../../include/ft.h"
#include "ft_ptx.cuh"
#include "ft_vec.cuh"

namespace ft {
namespace norm {

struct FwdParams {
    int M, D, B, S;  // S: rows per sample when there are no offsets
    const int32_t* offsets;
    int pre, post;
    float eps_pre, eps_post, alpha, inv_d;
    bool p32;
    int64_t ld_gate, ld_scale, ld_shift;
    const void *gate, *scale, *shift, *w_post, *w, *bias;
    const void* x;
    int64_t ldx;
    const __nv_bfloat16* y;
    int64_t ldy;
    void* r;
    int64_t ldr;
    __nv_bfloat16* h;
    int64_t ldh;
    float4* stats;
    float* amax;
    int tpr;  // threads of a row when rows share a warp (8, 16, 32)
};

struct BwdParams {
    int M, D, B, S;
    const int32_t* offsets;
    int pre, post;
    float alpha, inv_d;
    bool p32;
    int64_t ld_gate, ld_scale;
    const void *gate, *scale, *w_post, *w;
    const __nv_bfloat16* dh;
    int64_t lddh;
    const void* dr;
    int64_t lddr;
    const void* r;
    int64_t ldr;
    const __nv_bfloat16* y;
    int64_t ldy;
    const float4* stats;
    void* dx;
    int64_t lddx;
    __nv_bfloat16* dy;
    int64_t lddy;
    float* amax;
    float* partial;  // [chunks + B][3][D], or null
    bool need_s, need_t;
    int chunk;  // rows of a block
    int tpr;
};

// The sample of a row, or -1 behind the last one.  With offsets: the first b
// whose end lies above the row (an empty sample's end never is the first).
__device__ __forceinline__ int sample_of(int row, const int32_t* offsets, int B, int S) {
    if (!offsets) return row / S;
    int lo = 0, hi = B;
    while (lo < hi) {
        const int mid = (lo + hi) >> 1;
        if (__ldg(offsets + mid + 1) > row)
            hi = mid;
        else
            lo = mid + 1;
    }
    return lo < B ? lo : -1;
}

// Sum over the threads of a row: within groups of `tpr` lanes (kWide false)
// or over the block (kWide true; `red` has two halves used in turn, so one
// barrier per reduction suffices: a half is written again only after the
// barrier of the reduction between).
template <bool kWide>
struct RowSum {
    float* red;
    int tpr, half = 0;
    __device__ RowSum(float* r, int t) : red(r), tpr(t) {}
    __device__ __forceinline__ float operator()(float v) {
        if constexpr (!kWide) {
            for (int o = tpr >> 1; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
            return v;
        } else {
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
            float* s = red + half * 16;
            half ^= 1;
            if ((threadIdx.x & 31) == 0) s[threadIdx.x >> 5] = v;
            __syncthreads();
            const int nw = blockDim.x >> 5;
            v = 0.0f;
            for (int i = 0; i < nw; ++i) v += s[i];
            return v;
        }
    }
    // two sums at once
    __device__ __forceinline__ float2 operator()(float a, float b) {
        if constexpr (!kWide) {
            for (int o = tpr >> 1; o > 0; o >>= 1) {
                a += __shfl_xor_sync(0xFFFFFFFFu, a, o);
                b += __shfl_xor_sync(0xFFFFFFFFu, b, o);
            }
            return make_float2(a, b);
        } else {
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) {
                a += __shfl_xor_sync(0xFFFFFFFFu, a, o);
                b += __shfl_xor_sync(0xFFFFFFFFu, b, o);
            }
            float2* s = reinterpret_cast<float2*>(red + 32) + half * 16;
            half ^= 1;
            if ((threadIdx.x & 31) == 0) s[threadIdx.x >> 5] = make_float2(a, b);
            __syncthreads();
            const int nw = blockDim.x >> 5;
            a = b = 0.0f;
            for (int i = 0; i < nw; ++i) a += s[i].x, b += s[i].y;
            return make_float2(a, b);
        }
    }
};
constexpr int kRedFloats = 32 + 64;

// Mean and 1/deviation of a row held as V vectors of eight (`ok[v]`: this
// thread has a vector v; absent ones hold zeros).
template <int V, bool kWide>
__device__ __forceinline__ float2 row_stats(const float (&x)[V][8], const bool (&ok)[V], int kind, float eps,
                                            float inv_d, RowSum<kWide>& sum) {
    float mean = 0.0f;
    if (kind == FT_NORM_NONE) return make_float2(0.0f, 1.0f);
    if (kind == FT_NORM_LAYER) {
        float s = 0.0f;
#pragma unroll
        for (int v = 0; v < V; ++v)
#pragma unroll
            for (int i = 0; i < 8; ++i) s += x[v][i];
        mean = sum(s) * inv_d;
    }
    float q = 0.0f;
#pragma unroll
    for (int v = 0; v < V; ++v)
        if (ok[v])
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float c = x[v][i] - mean;
                q = fmaf(c, c, q);
            }
    return make_float2(mean, 1.0f / sqrtf(fmaf(sum(q), inv_d, eps)));
}

template <typename XT, int V, bool kWide>
__global__ void __launch_bounds__(512) k_gated_norm_fwd(const __grid_constant__ FwdParams p) {
    __shared__ float red[kRedFloats];
    const int tpr = kWide ? blockDim.x : p.tpr;
    const int group = kWide ? 0 : threadIdx.x / tpr, groups = kWide ? 1 : blockDim.x / tpr;
    const int t = kWide ? threadIdx.x : threadIdx.x % tpr;
    RowSum<kWide> sum(red, tpr);
    int col[V];
    bool ok[V];
#pragma unroll
    for (int v = 0; v < V; ++v) {
        col[v] = 8 * (t + v * tpr);
        ok[v] = col[v] < p.D;
    }
    grid_dep_wait();
    const XT* x = static_cast<const XT*>(p.x);
    Raw8<XT> nx[V];
    Raw8<__nv_bfloat16> ny[V];
    auto fetch = [&](int row) {
#pragma unroll
        for (int v = 0; v < V; ++v) {
            nx[v] = {};
            ny[v] = {};
            if (ok[v] && row < p.M) {
                load8(nx[v], x + (int64_t)row * p.ldx + col[v]);
                if (p.y) load8(ny[v], p.y + (int64_t)row * p.ldy + col[v]);
            }
        }
    };
    float amax = 0.0f;
    fetch(blockIdx.x * groups + group);
    // every thread of a block takes the same number of turns: the reductions
    // are the whole warp's or block's
    for (int first = blockIdx.x * groups; first < p.M; first += gridDim.x * groups) {
        const int row = first + group;
        const int b = row < p.M ? sample_of(row, p.offsets, p.B, p.S) : -1;
        float xv[V][8], u[V][8];
#pragma unroll
        for (int v = 0; v < V; ++v) {
            unpack8(nx[v], xv[v]);
            unpack8(ny[v], u[v]);
        }
        fetch(row + gridDim.x * groups);
        if (kWide && b < 0) continue;  // uniform over the block
        const int64_t sample = b < 0 ? 0 : b;
        float2 post = make_float2(0.0f, 1.0f);
        if (p.y) {
            post = row_stats<V, kWide>(u, ok, p.post, p.eps_post, p.inv_d, sum);
#pragma unroll
            for (int v = 0; v < V; ++v) {
                if (!ok[v]) continue;
                if (p.post != FT_NORM_NONE) {
#pragma unroll
                    for (int i = 0; i < 8; ++i) u[v][i] = (u[v][i] - post.x) * post.y;
                }
                float c[8];
                if (p.w_post) {
                    load_param8(p.w_post, col[v], p.p32, c);
#pragma unroll
                    for (int i = 0; i < 8; ++i) u[v][i] *= c[i];
                }
                if (p.gate) {
                    load_param8(p.gate, sample * p.ld_gate + col[v], p.p32, c);
#pragma unroll
                    for (int i = 0; i < 8; ++i) u[v][i] *= c[i];
                }
#pragma unroll
                for (int i = 0; i < 8; ++i) xv[v][i] = fmaf(p.alpha, u[v][i], xv[v][i]);
                if (b >= 0) {
                    store8(static_cast<XT*>(p.r) + (int64_t)row * p.ldr + col[v], xv[v]);
                }
            }
        }
        const float2 pre = row_stats<V, kWide>(xv, ok, p.pre, p.eps_pre, p.inv_d, sum);
        if (b < 0) continue;
        if (p.pre != FT_NORM_NONE) {
#pragma unroll
            for (int v = 0; v < V; ++v) {
                if (!ok[v]) continue;
                float c[8], f[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) f[i] = (xv[v][i] - pre.x) * pre.y;
                if (p.w) {
                    load_param8(p.w, col[v], p.p32, c);
#pragma unroll
                    for (int i = 0; i < 8; ++i) f[i] *= c[i];
                }
                if (p.bias) {
                    load_param8(p.bias, col[v], p.p32, c);
#pragma unroll
                    for (int i = 0; i < 8; ++i) f[i] += c[i];
                }
                if (p.scale) {
                    load_param8(p.scale, sample * p.ld_scale + col[v], p.p32, c);
#pragma unroll
                    for (int i = 0; i < 8; ++i) f[i] *= 1.0f + c[i];
                }
                if (p.shift) {
                    load_param8(p.shift, sample * p.ld_shift + col[v], p.p32, c);
#pragma unroll
                    for (int i = 0; i < 8; ++i) f[i] += c[i];
                }
                store8(p.h + (int64_t)row * p.ldh + col[v], f);
                amax = max_abs8(f, amax);
            }
        }
        if (p.stats && t == 0) p.stats[row] = make_float4(pre.x, pre.y, post.x, post.y);
    }
    raise_amax(p.amax, amax, red);
}

// Backward.  A block takes `chunk` consecutive rows (its groups one each in
// turn) and keeps its columns' sums of the current sample in registers; at a
// sample's last row in the chunk they go to the partial row chunk + sample --
// a number that no other (chunk, sample) pair met by these ascending steps
// has, since every step raises one of the two.
template <typename XT, int V, bool kWide, bool kAcc>
__global__ void __launch_bounds__(512) k_gated_norm_bwd(const __grid_constant__ BwdParams p) {
    __shared__ float red[kRedFloats];
    __shared__ float flush_buf[kWide || !kAcc ? 1 : 256 * 8];
    const int tpr = kWide ? blockDim.x : p.tpr;
    const int group = kWide ? 0 : threadIdx.x / tpr, groups = kWide ? 1 : blockDim.x / tpr;
    const int t = kWide ? threadIdx.x : threadIdx.x % tpr;
    RowSum<kWide> sum(red, tpr);
    int col[V];
    bool ok[V];
#pragma unroll
    for (int v = 0; v < V; ++v) {
        col[v] = 8 * (t + v * tpr);
        ok[v] = col[v] < p.D;
    }
    const int begin = blockIdx.x * p.chunk, end = min(p.M, begin + p.chunk);
    grid_dep_wait();
    Raw8<__nv_bfloat16> ndh[V], ny[V];
    Raw8<XT> ndr[V], nr[V];
    float4 nst = make_float4(0.0f, 1.0f, 0.0f, 1.0f);
    auto fetch = [&](int row) {
#pragma unroll
        for (int v = 0; v < V; ++v) {
            ndh[v] = {};
            ny[v] = {};
            ndr[v] = {};
            nr[v] = {};
            if (ok[v] && row < end) {
                if (p.dh) load8(ndh[v], p.dh + (int64_t)row * p.lddh + col[v]);
                if (p.dr) load8(ndr[v], static_cast<const XT*>(p.dr) + (int64_t)row * p.lddr + col[v]);
                if (p.r) load8(nr[v], static_cast<const XT*>(p.r) + (int64_t)row * p.ldr + col[v]);
                if (p.y) load8(ny[v], p.y + (int64_t)row * p.ldy + col[v]);
            }
        }
        if (p.stats && row < end) nst = __ldg(p.stats + row);
    };
    float acc[kAcc ? 3 : 1][V][8];
#pragma unroll
    for (int k = 0; k < (kAcc ? 3 : 1); ++k)
#pragma unroll
        for (int v = 0; v < V; ++v)
#pragma unroll
            for (int i = 0; i < 8; ++i) acc[k][v][i] = 0.0f;
    float amax = 0.0f;
    // writes the sums of sample b over the block and clears them
    auto flush = [&](int b) {
        if constexpr (kAcc) {
            float* out = p.partial + ((int64_t)blockIdx.x + b) * 3 * p.D;
#pragma unroll
            for (int k = 0; k < 3; ++k) {
                const bool wanted = k < 2 ? p.need_s : p.need_t;
                if (!wanted) continue;  // uniform
                if constexpr (kWide) {
#pragma unroll
                    for (int v = 0; v < V; ++v)
                        if (ok[v]) store8(out + (int64_t)k * p.D + col[v], acc[k][v]);
                } else {
                    __syncthreads();
#pragma unroll
                    for (int i = 0; i < 8; ++i) flush_buf[threadIdx.x * 8 + i] = acc[k][0][i];
                    __syncthreads();
                    for (int c = threadIdx.x; c < p.D; c += blockDim.x) {
                        float s = 0.0f;
                        for (int g = 0; g < groups; ++g) s += flush_buf[g * tpr * 8 + c];
                        out[(int64_t)k * p.D + c] = s;
                    }
                }
#pragma unroll
                for (int v = 0; v < V; ++v)
#pragma unroll
                    for (int i = 0; i < 8; ++i) acc[k][v][i] = 0.0f;
            }
        }
    };
    fetch(begin + group);
    int row0 = begin;
    while (row0 < end) {
        // the run of rows of one sample that starts at row0
        const int b = sample_of(row0, p.offsets, p.B, p.S);
        if (b < 0) break;  // behind the last sample: the rest is too
        const int stop = min(end, max(row0 + 1, p.offsets ? __ldg(p.offsets + b + 1) : (b + 1) * p.S));
        const int64_t sample = b;
        for (int first = row0; first < stop; first += groups) {
            const int row = first + group;
            const bool live = row < stop;
            float xh[V][8], yh[V][8], d[V][8], dh[V][8];
            const float4 st = nst;
#pragma unroll
            for (int v = 0; v < V; ++v) {
                unpack8(ndh[v], dh[v]);
                unpack8(ndr[v], d[v]);
                unpack8(nr[v], xh[v]);
                unpack8(ny[v], yh[v]);
                if (!kWide && !live) {  // the row belongs to the next run: no part of the sums
#pragma unroll
                    for (int i = 0; i < 8; ++i) dh[v][i] = d[v][i] = xh[v][i] = yh[v][i] = 0.0f;
                }
            }
            // the next row of this run, or the first of the next run
            fetch(first + groups < stop ? row + groups : stop + group);
            if (p.pre != FT_NORM_NONE) {
                float s0 = 0.0f, s1 = 0.0f;
#pragma unroll
                for (int v = 0; v < V; ++v) {
                    if (!ok[v]) continue;
                    float c[8], z[8];
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        xh[v][i] = (xh[v][i] - st.x) * st.y;
                        z[i] = dh[v][i];
                    }
                    if constexpr (kAcc) {
                        if (live)
#pragma unroll
                            for (int i = 0; i < 8; ++i) {
                                acc[0][v][i] += dh[v][i];
                                acc[1][v][i] = fmaf(dh[v][i], xh[v][i], acc[1][v][i]);
                            }
                    }
                    if (p.scale) {
                        load_param8(p.scale, sample * p.ld_scale + col[v], p.p32, c);
#pragma unroll
                        for (int i = 0; i < 8; ++i) z[i] *= 1.0f + c[i];
                    }
                    if (p.w) {
                        load_param8(p.w, col[v], p.p32, c);
#pragma unroll
                        for (int i = 0; i < 8; ++i) z[i] *= c[i];
                    }
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        s0 += z[i];
                        s1 = fmaf(z[i], xh[v][i], s1);
                        dh[v][i] = z[i];
                    }
                }
                const float2 m = sum(s0, s1);
                const float m0 = p.pre == FT_NORM_LAYER ? m.x * p.inv_d : 0.0f, m1 = m.y * p.inv_d;
#pragma unroll
                for (int v = 0; v < V; ++v)
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        d[v][i] = fmaf(st.y, dh[v][i] - fmaf(xh[v][i], m1, m0), d[v][i]);
            }
            if (p.y || p.dy) {
                float s0 = 0.0f, s1 = 0.0f;
                float e[V][8];
#pragma unroll
                for (int v = 0; v < V; ++v) {
                    if (!ok[v]) continue;
                    float c[8];
                    if (p.post != FT_NORM_NONE) {
#pragma unroll
                        for (int i = 0; i < 8; ++i) yh[v][i] = (yh[v][i] - st.z) * st.w;
                    }
                    if constexpr (kAcc) {
                        if (live)
#pragma unroll
                            for (int i = 0; i < 8; ++i) acc[2][v][i] = fmaf(d[v][i], yh[v][i], acc[2][v][i]);
                    }
#pragma unroll
                    for (int i = 0; i < 8; ++i) e[v][i] = p.alpha * d[v][i];
                    if (p.gate) {
                        load_param8(p.gate, sample * p.ld_gate + col[v], p.p32, c);
#pragma unroll
                        for (int i = 0; i < 8; ++i) e[v][i] *= c[i];
                    }
                    if (p.w_post) {
                        load_param8(p.w_post, col[v], p.p32, c);
#pragma unroll
                        for (int i = 0; i < 8; ++i) e[v][i] *= c[i];
                    }
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        s0 += e[v][i];
                        s1 = fmaf(e[v][i], yh[v][i], s1);
                    }
                }
                if (p.dy && p.post != FT_NORM_NONE) {
                    const float2 m = sum(s0, s1);
                    const float m0 = p.post == FT_NORM_LAYER ? m.x * p.inv_d : 0.0f, m1 = m.y * p.inv_d;
#pragma unroll
                    for (int v = 0; v < V; ++v)
#pragma unroll
                        for (int i = 0; i < 8; ++i) e[v][i] = st.w * (e[v][i] - fmaf(yh[v][i], m1, m0));
                }
                if (p.dy && live) {
#pragma unroll
                    for (int v = 0; v < V; ++v)
                        if (ok[v]) {
                            store8(p.dy + (int64_t)row * p.lddy + col[v], e[v]);
                            amax = max_abs8(e[v], amax);
                        }
                }
            }
            if (p.dx && live) {
#pragma unroll
                for (int v = 0; v < V; ++v)
                    if (ok[v]) store8(static_cast<XT*>(p.dx) + (int64_t)row * p.lddx + col[v], d[v]);
            }
        }
        flush(b);
        row0 = stop;
    }
    raise_amax(p.amax, amax, red);
}

struct ReduceParams {
    int M, D, B, S, chunk, chunks;
    const int32_t* offsets;
    float alpha;
    bool p32;
    int64_t ld_gate, ld_scale;
    const void *gate, *scale, *w_post, *w, *bias;
    const float* partial;
    float *dgate, *dscale, *dshift, *dw_post, *dw, *dbias;
    bool need_s, need_t;
    bool all_samples;  // one block row walks every sample (the weights' gradients sum over them)
};

// Adds the partial rows of each sample, in ascending order: 32 columns per
// block, kGroups threads per column.  Sample b's partial rows are those of
// the chunks that hold its rows.
constexpr int kReduceGroups = 16;
__global__ void __launch_bounds__(32 * kReduceGroups) k_gated_norm_reduce(const __grid_constant__ ReduceParams p) {
    __shared__ float part[3][kReduceGroups][33];
    const int lane = threadIdx.x & 31, g = threadIdx.x >> 5;
    const int c = blockIdx.x * 32 + lane;
    const bool ok = c < p.D;
    grid_dep_wait();
    float dw = 0.0f, db = 0.0f, dwp = 0.0f;
    const float w = p.w && ok ? load_param(p.w, c, p.p32) : 1.0f;
    const float bias = p.bias && ok ? load_param(p.bias, c, p.p32) : 0.0f;
    const float wp = p.w_post && ok ? load_param(p.w_post, c, p.p32) : 1.0f;
    const int step = p.all_samples ? 1 : gridDim.y;
    for (int b = p.all_samples ? 0 : blockIdx.y; b < p.B; b += step) {
        int lo = p.offsets ? __ldg(p.offsets + b) : b * p.S;
        int hi = p.offsets ? __ldg(p.offsets + b + 1) : (b + 1) * p.S;
        lo = max(lo, 0);
        hi = min(hi, p.M);
        float s[3] = {0.0f, 0.0f, 0.0f};
        if (ok && lo < hi) {
            const int c0 = lo / p.chunk, c1 = (hi - 1) / p.chunk;
            for (int k = c0 + g; k <= c1; k += kReduceGroups) {
                const float* q = p.partial + ((int64_t)k + b) * 3 * p.D + c;
                if (p.need_s) {
                    s[0] += __ldg(q);
                    s[1] += __ldg(q + p.D);
                }
                if (p.need_t) s[2] += __ldg(q + 2 * (int64_t)p.D);
            }
        }
        __syncthreads();
#pragma unroll
        for (int k = 0; k < 3; ++k) part[k][g][lane] = s[k];
        __syncthreads();
        if (g == 0 && ok) {
#pragma unroll
            for (int k = 0; k < 3; ++k) {
                s[k] = 0.0f;
                for (int i = 0; i < kReduceGroups; ++i) s[k] += part[k][i][lane];
            }
            const int64_t at = (int64_t)b * p.D + c;
            if (p.dshift) p.dshift[at] = s[0];
            if (p.dscale) p.dscale[at] = fmaf(w, s[1], bias * s[0]);
            if (p.dgate) p.dgate[at] = p.alpha * wp * s[2];
            if (p.all_samples) {
                const float a = p.scale ? 1.0f + load_param(p.scale, (int64_t)b * p.ld_scale + c, p.p32) : 1.0f;
                dw = fmaf(a, s[1], dw);
                db = fmaf(a, s[0], db);
                const float gate = p.gate ? load_param(p.gate, (int64_t)b * p.ld_gate + c, p.p32) : 1.0f;
                dwp = fmaf(p.alpha * gate, s[2], dwp);
            }
        }
    }
    if (g == 0 && ok && p.all_samples) {
        if (p.dw) p.dw[c] = dw;
        if (p.dbias) p.dbias[c] = db;
        if (p.dw_post) p.dw_post[c] = dwp;
    }
}

}  // namespace norm
}  // namespace ft
