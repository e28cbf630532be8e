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
// A row stays on chip between its one load and its one store, the variance is
// taken about the mean (no cancellation), and the next rows' loads are in
// flight while a row is reduced.  HBM bounds both kernels for many rows, 8 B
// per element forward (x, y, r, h in bf16), 12 B backward (dh, dr, r, y, dx,
// dy): from 4736 to 18944 rows of 3072 channels, 1000 more cost 4.0 us and 5.8
// us, 93 and 98 % of the measured 6.53 TB/s.  At 4608 rows (30 us forward and
// 44 us backward with its sums, replayed back to back, against 17.4 and 26.0)
// what bounds them is the start, the drain and the instructions of a row, 27
// and 47 per element: hence a thread holds four vectors forward (fewer barriers
// and addresses per element; one vector per thread took 41 us), sums come off
// in two-lane arithmetic, and the usual modulated boundary is compiled apart
// (kMod: 30 us against 38 us forward, 44 against 55 backward).  Backward a thread holds one vector up to
// 4096 channels, 80 registers and two blocks of 384 threads per SM at 3072
// (two vectors and three blocks of 192: 45 against 44 us).
#pragma once

#include "../../include/ft.h"
#include "ft_ptx.cuh"
#include "ft_vec.cuh"

namespace ft {
namespace norm {

// What a call has, as bits: one test of a word each, where comparing pointers
// and kinds took the general kernels a third of their instructions.
enum Has : uint32_t {
    kDh = 1, kDr = 2, kR = 4, kY = 8, kGate = 16, kScale = 32, kShift = 64, kW = 128, kBias = 256, kWPost = 512,
    kPre = 1024, kPreMean = 2048, kPost = 4096, kPostMean = 8192, kDx = 16384, kDy = 32768, kStats = 65536
};

struct FwdParams {
    uint32_t has;
    int M, D, B, S;  // S: rows per sample when there are no offsets
    const int32_t* offsets;
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
    uint32_t has;
    int M, D, B, S;
    const int32_t* offsets;
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
// or over the block (kWide true).  A block's warps leave their sums in one of
// two halves of `red` in turn, so one barrier per reduction suffices: a half
// is written again only after the barrier of the reduction between.  Every
// thread then adds all 16 places (the absent warps' hold zeros) in a tree.
constexpr int kRedFloats = 64;
template <bool kWide>
struct RowSum {
    float2* red;
    int tpr, half = 0;
    __device__ RowSum(float* r, int t) : red(reinterpret_cast<float2*>(r)), tpr(t) {
        if (kWide) {
            for (int i = threadIdx.x; i < kRedFloats; i += blockDim.x) r[i] = 0.0f;
            __syncthreads();
        }
    }
    __device__ __forceinline__ float operator()(float v) { return (*this)(make_float2(v, 0.0f)).x; }
    // two sums at once
    __device__ __forceinline__ float2 operator()(float2 v) {
        if constexpr (!kWide) {
            for (int o = tpr >> 1; o > 0; o >>= 1)
                v = add2(v, make_float2(__shfl_xor_sync(0xFFFFFFFFu, v.x, o), __shfl_xor_sync(0xFFFFFFFFu, v.y, o)));
            return v;
        } else {
#pragma unroll
            for (int o = 16; o > 0; o >>= 1)
                v = add2(v, make_float2(__shfl_xor_sync(0xFFFFFFFFu, v.x, o), __shfl_xor_sync(0xFFFFFFFFu, v.y, o)));
            float2* s = red + half * 16;
            half ^= 1;
            if ((threadIdx.x & 31) == 0) s[threadIdx.x >> 5] = v;
            __syncthreads();
            float2 w[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float4 q = reinterpret_cast<const float4*>(s)[i];
                w[i] = add2(make_float2(q.x, q.y), make_float2(q.z, q.w));
            }
#pragma unroll
            for (int n = 4; n > 0; n >>= 1)
#pragma unroll
                for (int i = 0; i < n; ++i) w[i] = add2(w[i], w[i + n]);
            return w[0];
        }
    }
};

// Rows come through a ring of shared-memory stages.  Every thread copies
// (cp.async) and reads its own 16-byte slots only, stages - 1 turns ahead:
// loads in flight cost no registers, and no barrier guards the ring.  Slots
// that are never filled (columns behind the row's last) hold zeros.
template <int kSlots, int V>
struct Ring {
    uint32_t base;
    int slot_stride, stage_bytes;
    __device__ Ring(const void* smem) {
        base = smem_u32(smem) + threadIdx.x * 16;
        slot_stride = blockDim.x * 16;
        stage_bytes = bytes(blockDim.x);
    }
    __device__ void clear(int stages) const {
        for (int i = 0; i < stages * kSlots * V; ++i) st_shared_v4(base + i * slot_stride, make_uint4(0, 0, 0, 0));
    }
    __host__ __device__ static constexpr int bytes(int threads) { return kSlots * V * threads * 16; }
    __device__ __forceinline__ uint32_t at(int stage, int v, int k) const {
        return base + stage * stage_bytes + (v * kSlots + k) * slot_stride;
    }
    // slots k.. of a vector, or zeros
    __device__ __forceinline__ F8 get(int stage, int v, int k, bool there, __nv_bfloat16) const {
        return there ? widen(ld_shared_v4(at(stage, v, k))) : zero8();
    }
    __device__ __forceinline__ F8 get(int stage, int v, int k, bool there, float) const {
        if (!there) return zero8();
        Raw8<float> w;
        w.a = ld_shared_v4(at(stage, v, k));
        w.b = ld_shared_v4(at(stage, v, k + 1));
        return widen(w);
    }
};
template <typename T>
__device__ __forceinline__ void ring_copy(uint32_t dst, int slot_stride, const T* src) {
    cp_async16(dst, src);
    if constexpr (sizeof(T) == 4) cp_async16(dst + slot_stride, src + 4);
}

// Mean and 1/deviation of a row held as V vectors of eight (`ok[v]`: this
// thread has a vector v); leaves x - mean in x.
template <int V, bool kWide>
__device__ __forceinline__ float2 center(F8 (&x)[V], const bool (&ok)[V], bool about_mean, float eps, float inv_d,
                                         RowSum<kWide>& sum) {
    float mean = 0.0f;
    if (about_mean) {
        float2 s = both(0.0f);
#pragma unroll
        for (int v = 0; v < V; ++v) s = gather(s, x[v]);  // absent vectors are zeros
        mean = sum(s.x + s.y) * inv_d;
#pragma unroll
        for (int v = 0; v < V; ++v) x[v] = add(x[v], -mean);
    }
    float2 q = both(0.0f);
#pragma unroll
    for (int v = 0; v < V; ++v) {
        const float2 more = gather(q, x[v], x[v]);
        q = ok[v] ? more : q;
    }
    return make_float2(mean, 1.0f / sqrtf(fmaf(sum(q.x + q.y), inv_d, eps)));
}

constexpr int kFwdStages = 2;
template <typename XT>
constexpr int kFwdSlots = sizeof(XT) / 2 + 1;  // x, y

// kMod: the modulated residual boundary -- y, gate, scale and shift given, no
// weights, no post norm -- with these facts known to the compiler: what a row
// spends on asking for each part is then a third of its instructions less.
template <typename XT, int V, bool kWide, bool k32, bool kMod>
__global__ void __launch_bounds__(256) k_gated_norm_fwd(const __grid_constant__ FwdParams p) {
    constexpr int kYSlot = sizeof(XT) / 2;
    extern __shared__ __align__(16) uint8_t smem[];
    __shared__ __align__(16) float red[kRedFloats];
    const int tpr = kWide ? blockDim.x : p.tpr;
    const int group = kWide ? 0 : threadIdx.x / tpr, groups = kWide ? 1 : blockDim.x / tpr;
    const int t = kWide ? threadIdx.x : threadIdx.x % tpr;
    RowSum<kWide> sum(red, tpr);
    const Ring<kFwdSlots<XT>, V> ring(smem);
    int col[V], at[V];  // at: where a parameter is read; in range for absent vectors too
    bool ok[V];
#pragma unroll
    for (int v = 0; v < V; ++v) {
        col[v] = 8 * (t + v * tpr);
        ok[v] = col[v] < p.D;
        at[v] = ok[v] ? col[v] : 0;
    }
    ring.clear(kFwdStages);
    const uint32_t has = p.has;
    const bool has_y = kMod || has & kY, has_gate = kMod || has & kGate, has_scale = kMod || has & kScale;
    const bool has_shift = kMod || has & kShift, has_w = !kMod && has & kW, has_bias = !kMod && has & kBias;
    const bool has_wp = !kMod && has & kWPost, has_post = !kMod && has & kPost, has_pre = kMod || has & kPre;
    grid_dep_launch();
    grid_dep_wait();
    const int step = gridDim.x * groups;
    auto fetch = [&](int row, int stage) {
        if (row < p.M) {
            const XT* x = static_cast<const XT*>(p.x) + (int64_t)row * p.ldx;
            const __nv_bfloat16* y = p.y + (int64_t)row * p.ldy;
#pragma unroll
            for (int v = 0; v < V; ++v)
                if (ok[v]) {
                    ring_copy(ring.at(stage, v, 0), ring.slot_stride, x + col[v]);
                    if (has_y) ring_copy(ring.at(stage, v, kYSlot), ring.slot_stride, y + col[v]);
                }
        }
        cp_async_commit();
    };
    uint32_t amax = 0;
    fetch(blockIdx.x * groups + group, 0);
    int stage = 0;
    // every thread of a block takes the same number of turns: the reductions
    // are the whole warp's or block's
    for (int first = blockIdx.x * groups; first < p.M; first += step, stage ^= 1) {
        const int row = first + group;
        const int b = row < p.M ? sample_of(row, p.offsets, p.B, p.S) : -1;
        fetch(row + step, stage ^ 1);
        cp_async_wait<1>();
        if (kWide && b < 0) continue;  // uniform over the block
        const bool live = kWide || b >= 0;
        const int64_t sample = live ? b : 0;
        float2 post = make_float2(0.0f, 1.0f);
        F8 f[V];
        if (has_y) {
#pragma unroll
            for (int v = 0; v < V; ++v) f[v] = ring.get(stage, v, kYSlot, live, __nv_bfloat16());
            if (has_post) post = center<V, kWide>(f, ok, has & kPostMean, p.eps_post, p.inv_d, sum);
#pragma unroll
            for (int v = 0; v < V; ++v) {
                if (has_post) f[v] = mul(f[v], post.y);
                if (has_wp) f[v] = mul(f[v], load_param8<k32>(p.w_post, at[v]));
                if (has_gate) f[v] = mul(f[v], load_param8<k32>(p.gate, sample * p.ld_gate + at[v]));
                f[v] = fma(f[v], p.alpha, ring.get(stage, v, 0, live, XT()));
                Raw8<XT> r;
                round8(r, f[v]);
                if (live && ok[v]) put8(static_cast<XT*>(p.r) + (int64_t)row * p.ldr + col[v], r);
                f[v] = widen(r);  // the norm reads the stream as it is stored
                if (!ok[v]) f[v] = zero8();
            }
        } else {
#pragma unroll
            for (int v = 0; v < V; ++v) f[v] = ring.get(stage, v, 0, live, XT());
        }
        const float2 pre = has_pre ? center<V, kWide>(f, ok, has & kPreMean, p.eps_pre, p.inv_d, sum)
                                   : make_float2(0.0f, 1.0f);
        if (!live) continue;
        if (has_pre) {
#pragma unroll
            for (int v = 0; v < V; ++v) {
                if (kMod) {
                    // f rstd (1 + scale) + shift, the scale's part first
                    const F8 c = load_param8<k32>(p.scale, sample * p.ld_scale + at[v]);
                    const F8 a = add(mul(c, pre.y), pre.y);
                    f[v] = fma(f[v], a, load_param8<k32>(p.shift, sample * p.ld_shift + at[v]));
                } else {
                    f[v] = mul(f[v], pre.y);
                    if (has_w) f[v] = mul(f[v], load_param8<k32>(p.w, at[v]));
                    if (has_bias) f[v] = add(f[v], load_param8<k32>(p.bias, at[v]));
                    if (has_scale) f[v] = fma(f[v], load_param8<k32>(p.scale, sample * p.ld_scale + at[v]), f[v]);
                    if (has_shift) f[v] = add(f[v], load_param8<k32>(p.shift, sample * p.ld_shift + at[v]));
                }
                if (ok[v]) amax = store8_max(p.h + (int64_t)row * p.ldh + col[v], f[v], amax);
            }
        }
        if (has & kStats && t == 0) p.stats[row] = make_float4(pre.x, pre.y, post.x, post.y);
    }
    cp_async_wait<0>();
    raise_amax(p.amax, amax_of(amax), red);
}

// Backward.  A block takes `chunk` consecutive rows (its groups one each per
// turn) and keeps its columns' sums of the current sample in registers; at a
// sample's last row in the chunk they go to the partial row chunk + sample --
// a number that no other (chunk, sample) pair met by these ascending steps
// has, since every step raises one of the two.
template <typename XT>
constexpr int kBwdSlots = 2 + 2 * (sizeof(XT) / 2);  // dh, y, dr, r
constexpr int kBwdStages = 2;
template <int V, bool kWide, bool kMod>
constexpr int kBwdRegs = V == 2 ? 96 : kWide ? (kMod ? 80 : 64) : 128;

// kMod: dh, dr, r, y, gate and scale given, dx and dy wanted, no weights, no
// post norm; as in the forward.
template <typename XT, int V, bool kWide, bool k32, bool kMod>
__global__ void __maxnreg__((kBwdRegs<V, kWide, kMod>)) k_gated_norm_bwd(const __grid_constant__ BwdParams p) {
    constexpr int kStages = kBwdStages, kDrSlot = 2, kRSlot = 2 + sizeof(XT) / 2;
    extern __shared__ __align__(16) uint8_t smem[];
    __shared__ __align__(16) float red[kRedFloats];
    __shared__ __align__(16) float flush_buf[kWide ? 1 : 256 * 8];
    const int tpr = kWide ? blockDim.x : p.tpr;
    const int group = kWide ? 0 : threadIdx.x / tpr, groups = kWide ? 1 : blockDim.x / tpr;
    const int t = kWide ? threadIdx.x : threadIdx.x % tpr;
    RowSum<kWide> sum(red, tpr);
    const Ring<kBwdSlots<XT>, V> ring(smem);
    int col[V], pat[V];  // pat: where a parameter is read; in range for absent vectors too
    bool ok[V];
#pragma unroll
    for (int v = 0; v < V; ++v) {
        col[v] = 8 * (t + v * tpr);
        ok[v] = col[v] < p.D;
        pat[v] = ok[v] ? col[v] : 0;
    }
    ring.clear(kStages);
    const uint32_t has = p.has;
    const bool has_dh = kMod || has & kDh, has_dr = kMod || has & kDr, has_r = kMod || has & kR, has_y = kMod || has & kY;
    const bool has_gate = kMod || has & kGate, has_scale = kMod || has & kScale, has_w = !kMod && has & kW;
    const bool has_wp = !kMod && has & kWPost, pre = kMod || has & kPre, post = !kMod && has & kPost;
    const bool want_dx = kMod || has & kDx, want_dy = kMod || has & kDy, through = want_dy && post;
    const int begin = blockIdx.x * p.chunk, end = min(p.M, begin + p.chunk);
    const int turns = (end - begin + groups - 1) / groups;
    grid_dep_launch();
    grid_dep_wait();
    auto fetch = [&](int turn, int stage) {
        const int row = begin + turn * groups + group;
        if (row < end) {
#pragma unroll
            for (int v = 0; v < V; ++v) {
                if (!ok[v]) continue;
                if (has_dh) ring_copy(ring.at(stage, v, 0), 0, p.dh + (int64_t)row * p.lddh + col[v]);
                if (has_y) ring_copy(ring.at(stage, v, 1), 0, p.y + (int64_t)row * p.ldy + col[v]);
                if (has_dr)
                    ring_copy(ring.at(stage, v, kDrSlot), ring.slot_stride,
                              static_cast<const XT*>(p.dr) + (int64_t)row * p.lddr + col[v]);
                if (has_r)
                    ring_copy(ring.at(stage, v, kRSlot), ring.slot_stride,
                              static_cast<const XT*>(p.r) + (int64_t)row * p.ldr + col[v]);
            }
        }
        cp_async_commit();
    };
    float4 nst = make_float4(0.0f, 1.0f, 0.0f, 1.0f);
    auto fetch_stats = [&](int turn) {
        const int row = begin + turn * groups + group;
        if ((kMod || has & kStats) && row < end) nst = __ldg(p.stats + row);
    };
    F8 acc[3][V];
#pragma unroll
    for (int k = 0; k < 3; ++k)
#pragma unroll
        for (int v = 0; v < V; ++v) acc[k][v] = zero8();
    uint32_t amax = 0;
    // writes the sums of sample b over the block and clears them
    auto flush = [&](int b) {
        float* out = p.partial + ((int64_t)blockIdx.x + b) * 3 * p.D;
#pragma unroll
        for (int k = 0; k < 3; ++k) {
            const bool wanted = k < 2 ? p.need_s : p.need_t;
            if (!wanted) continue;  // uniform
            if constexpr (kWide) {
#pragma unroll
                for (int v = 0; v < V; ++v)
                    if (ok[v]) {
                        Raw8<float> w;
                        round8(w, acc[k][v]);
                        put8(out + (int64_t)k * p.D + col[v], w);
                    }
            } else {
                __syncthreads();
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    *reinterpret_cast<float2*>(flush_buf + threadIdx.x * 8 + 2 * i) = acc[k][0].p[i];
                __syncthreads();
                for (int c = threadIdx.x; c < p.D; c += blockDim.x) {
                    float s = 0.0f;
                    for (int g = 0; g < groups; ++g) s += flush_buf[g * tpr * 8 + c];
                    out[(int64_t)k * p.D + c] = s;
                }
            }
#pragma unroll
            for (int v = 0; v < V; ++v) acc[k][v] = zero8();
        }
    };
#pragma unroll
    for (int k = 0; k < kStages - 1; ++k) fetch(k, k);
    fetch_stats(0);
    int b = 0, stop = begin;  // the current sample, and where its rows (in this chunk) end
    int stage = 0, ahead = kStages - 1;
    for (int turn = 0; turn < turns; ++turn) {
        const int row = begin + turn * groups + group;
        const int turn_end = min(end, begin + (turn + 1) * groups);
        const float4 st = nst;
        fetch_stats(turn + 1);
        // the stage read in the turn before takes the turn stages - 1 ahead:
        // only this thread reads its slots
        fetch(turn + kStages - 1, ahead);
        cp_async_wait<kStages - 1>();
        // one pass over the turn's rows for each sample that has some of them
        int at = begin + turn * groups;
        while (at < turn_end) {
            if (at >= stop) {
                b = sample_of(at, p.offsets, p.B, p.S);
                if (b < 0) break;
                stop = min(end, max(at + 1, p.offsets ? __ldg(p.offsets + b + 1) : (b + 1) * p.S));
            }
            const int upto = min(stop, turn_end);
            // rows of other samples and stale slots count as zeros
            const bool live = kWide || (row >= at && row < upto);
            const int64_t sample = b;
            float a0 = 0.0f, a1 = 0.0f;  // d = dr + rstd z + a1 (r - mean) + a0
            F8 z[V];  // dh (1 + scale) w
            if (pre) {
                float2 s0 = both(0.0f), s1 = both(0.0f);
#pragma unroll
                for (int v = 0; v < V; ++v) {
                    const F8 xh = mul(add(ring.get(stage, v, kRSlot, live, XT()), live ? -st.x : 0.0f), live ? st.y : 0.0f);
                    z[v] = ring.get(stage, v, 0, live, __nv_bfloat16());
                    acc[0][v] = add(acc[0][v], z[v]);
                    acc[1][v] = fma(z[v], xh, acc[1][v]);
                    if (has_scale) z[v] = fma(z[v], load_param8<k32>(p.scale, sample * p.ld_scale + pat[v]), z[v]);
                    if (has_w) z[v] = mul(z[v], load_param8<k32>(p.w, pat[v]));
                    s0 = gather(s0, z[v]);  // an absent vector's z is zero
                    s1 = gather(s1, z[v], xh);
                }
                const float2 m = sum(make_float2(s0.x + s0.y, s1.x + s1.y));
                a0 = has & kPreMean && live ? -m.x * p.inv_d * st.y : 0.0f;
                a1 = live ? -m.y * p.inv_d * st.y * st.y : 0.0f;
            }
            auto normed_y = [&](int v) {
                const F8 y = ring.get(stage, v, 1, live, __nv_bfloat16());
                return post ? mul(add(y, live ? -st.z : 0.0f), live ? st.w : 0.0f) : y;
            };
            float2 s0 = both(0.0f), s1 = both(0.0f);
            F8 e[V];
#pragma unroll
            for (int v = 0; v < V; ++v) {
                e[v] = has_dr ? ring.get(stage, v, kDrSlot, live, XT()) : zero8();
                if (pre) {
                    // the row is read again rather than kept: registers set how many blocks an SM holds
                    const F8 xc = add(ring.get(stage, v, kRSlot, live, XT()), live ? -st.x : 0.0f);
                    e[v] = add(fma(xc, a1, fma(z[v], live ? st.y : 0.0f, e[v])), a0);
                }
                F8 yh = zero8();
                if (has_y) {
                    yh = normed_y(v);
                    acc[2][v] = fma(e[v], yh, acc[2][v]);
                }
                if (want_dx && live && ok[v]) {
                    Raw8<XT> w;
                    round8(w, e[v]);
                    put8(static_cast<XT*>(p.dx) + (int64_t)row * p.lddx + col[v], w);
                }
                if (want_dy) {
                    if (has_gate) {
                        e[v] = mul(e[v], mul(load_param8<k32>(p.gate, sample * p.ld_gate + pat[v]), p.alpha));
                    } else {
                        e[v] = mul(e[v], p.alpha);
                    }
                    if (has_wp) e[v] = mul(e[v], load_param8<k32>(p.w_post, pat[v]));
                    if (through) {
                        if (!ok[v]) e[v] = zero8();
                        s0 = gather(s0, e[v]);
                        s1 = gather(s1, e[v], yh);
                    } else if (live && ok[v]) {
                        amax = store8_max(p.dy + (int64_t)row * p.lddy + col[v], e[v], amax);
                    }
                }
            }
            if (through) {
                const float2 m = sum(make_float2(s0.x + s0.y, s1.x + s1.y));
                const float e0 = has & kPostMean ? m.x * p.inv_d : 0.0f, e1 = m.y * p.inv_d;
#pragma unroll
                for (int v = 0; v < V; ++v) {
                    if (!ok[v] || !live) continue;
                    amax = store8_max(p.dy + (int64_t)row * p.lddy + col[v],
                                      mul(add(fma(normed_y(v), -e1, e[v]), -e0), st.w), amax);
                }
            }
            if (stop <= turn_end) flush(b);
            at = upto;
        }
        if (b < 0) break;  // behind the last sample: the rest is too
        stage = stage + 1 == kStages ? 0 : stage + 1;
        ahead = ahead + 1 == kStages ? 0 : ahead + 1;
    }
    cp_async_wait<0>();
    raise_amax(p.amax, amax_of(amax), red);
}

struct ReduceParams {
    int M, D, B, S, chunk;
    const int32_t* offsets;
    float alpha;
    bool p32;
    int64_t ld_gate, ld_scale;
    const void *gate, *scale, *w_post, *w, *bias;
    const float* partial;  // [chunks + B][3][D]
    float* sums;           // [B][3][D] for the weights' gradients, or null
    float *dgate, *dscale, *dshift, *dw_post, *dw, *dbias;
    bool need_s, need_t;
};

// Adds the partial rows of each sample in a fixed order: 32 columns per
// block, a thread per column and every kGroups-th partial row (32, or 4 where
// samples have few), so that a thread's loads are in flight at once.  Sample
// b's partial rows are those of the chunks that hold its rows.
template <int kGroups>
__global__ void __launch_bounds__(32 * kGroups) k_gated_norm_reduce(const __grid_constant__ ReduceParams p) {
    __shared__ float part[3][kGroups][33];
    const int lane = threadIdx.x & 31, g = threadIdx.x >> 5;
    const int c = blockIdx.x * 32 + lane;
    const bool ok = c < p.D;
    grid_dep_launch();
    grid_dep_wait();
    const float w = p.w && ok ? load_param(p.w, c, p.p32) : 1.0f;
    const float bias = p.bias && ok ? load_param(p.bias, c, p.p32) : 0.0f;
    const float wp = p.w_post && ok ? load_param(p.w_post, c, p.p32) : 1.0f;
    for (int b = blockIdx.y; b < p.B; b += gridDim.y) {
        int lo = p.offsets ? __ldg(p.offsets + b) : b * p.S;
        int hi = p.offsets ? __ldg(p.offsets + b + 1) : (b + 1) * p.S;
        lo = max(lo, 0);
        hi = min(hi, p.M);
        float s[3] = {0.0f, 0.0f, 0.0f};
        if (ok && lo < hi) {
            const int c0 = lo / p.chunk, c1 = (hi - 1) / p.chunk;
            const float* q = p.partial + ((int64_t)c0 + b + g) * 3 * p.D + c;
            const int64_t step = (int64_t)kGroups * 3 * p.D;
#pragma unroll 4
            for (int k = c0 + g; k <= c1; k += kGroups, q += step) {
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
        if (g < 3) {  // warp k adds sum k
            float t = 0.0f;
#pragma unroll
            for (int i = 0; i < kGroups; ++i) t += part[g][i][lane];
            part[g][0][lane] = t;
        }
        __syncthreads();
        if (g == 0 && ok) {
            const float s0 = part[0][0][lane], s1 = part[1][0][lane], s2 = part[2][0][lane];
            const int64_t at = (int64_t)b * p.D + c;
            if (p.dshift) p.dshift[at] = s0;
            if (p.dscale) p.dscale[at] = fmaf(w, s1, bias * s0);
            if (p.dgate) p.dgate[at] = p.alpha * wp * s2;
            if (p.sums) {
                float* o = p.sums + (int64_t)b * 3 * p.D + c;
                o[0] = s0;
                o[p.D] = s1;
                o[2 * (int64_t)p.D] = s2;
            }
        }
    }
}

// The weights' gradients from the samples' sums.
__global__ void __launch_bounds__(32) k_gated_norm_weights(const __grid_constant__ ReduceParams p) {
    const int c = blockIdx.x * 32 + threadIdx.x;
    grid_dep_launch();
    grid_dep_wait();
    if (c >= p.D) return;
    float dw = 0.0f, db = 0.0f, dwp = 0.0f;
#pragma unroll 4
    for (int b = 0; b < p.B; ++b) {
        const float* q = p.sums + (int64_t)b * 3 * p.D + c;
        const float a = p.scale ? 1.0f + load_param(p.scale, (int64_t)b * p.ld_scale + c, p.p32) : 1.0f;
        const float gate = p.gate ? load_param(p.gate, (int64_t)b * p.ld_gate + c, p.p32) : 1.0f;
        db = fmaf(a, q[0], db);
        dw = fmaf(a, q[p.D], dw);
        dwp = fmaf(p.alpha * gate, q[2 * (int64_t)p.D], dwp);
    }
    if (p.dw) p.dw[c] = dw;
    if (p.dbias) p.dbias[c] = db;
    if (p.dw_post) p.dw_post[c] = dwp;
}

}  // namespace norm
}  // namespace ft
