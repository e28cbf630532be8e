// k_rope.cuh -- rotary positions with several axes on the queries and keys
// of a QKV linear's output, with the RMS norm of each head before it, and
// their backward.
//
// A query or key head x [hd]:  n = x rstd w,  rstd = 1 / sqrt(mean(x^2) + eps),
// then its pairs (a, b) turn:  (a cos - b sin, b cos + a sin), pair j of row
// m by pos[m, axis(j)] freqs[j].  Backward: turn by the negative angle, then
//     dw = sum over rows and heads of d x rstd
//     dx = rstd (z - x rstd^2 mean(z x)),  z = d w
//
// The angle is formed in FP64 in turns and reduced by its nearest integer:
// p f / 2 pi carries 2^-53 of up to 2^31 turns, so what is left is exact to
// 2^-22 of a turn at the farthest position and to FP32 at a million.
//
// A warp takes a row, or a slice of its heads when there are few rows: it
// forms the cosines and sines of the row's pairs, a pair or more per lane,
// and then walks the heads, a power of two of lanes per head with eight
// values (four pairs) each, so a lane meets the same four pairs in every
// head.  The first and the second values of the pairs are held apart (for
// interleaved pairs by the way they are unpacked), which makes the turn
// two-lane arithmetic in either layout.  HBM bounds both directions, 4 B per
// element of qkv, 6 B per query and key element backward with a norm, as long
// as a head's values cost few instructions: an SM moves three elements a
// clock.  At 4608 rows of 3 x 24 heads of 128 with norms, replayed back to back:
// 36 us forward (0.73 of the measured HBM rate) and 52 us backward with the
// weights' sums (0.67); a table of turns in shared memory that a block shares,
// with a lookup per head, took 61 and 119 us.
#pragma once

#include <type_traits>

#include "../../include/ft.h"
#include "ft_ptx.cuh"
#include "ft_vec.cuh"

namespace ft {
namespace rope {

constexpr int kThreads = 128;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxPairs = 128;
template <bool kBwd, bool kNorm>
constexpr int kU = kBwd && kNorm ? 2 : 4;  // heads in flight per group of lanes
// Backward with a norm two operands per head are in flight: they come through
// a ring of kDepth batches in shared memory (cp.async, every thread its own
// slots), which holds more of them than registers could.
template <bool kBwd, bool kNorm>
constexpr bool kRing = kBwd && kNorm;
constexpr int kDepth = 2;
template <bool kBwd, bool kNorm>
constexpr int kRegs = kBwd && kNorm ? 96 : 64;
template <bool kBwd, bool kNorm>
constexpr int kRingBytes = kRing<kBwd, kNorm> ? kDepth * 2 * kU<kBwd, kNorm> * kThreads * 16 : 0;

struct Heads {
    __nv_bfloat16* p;
    int64_t sb, sh, st;
};

struct Params {
    int M, S, Hq, Hk, Hv, hd;  // Hv: 0 when the values are not copied
    int rot, halves, norm, pos_f32, p32, n_axes;
    int axis_end[4];  // pairs up to and including axis a
    int lanes;        // per head
    int whole;        // rows that one warp takes each
    int slices;       // of the heads of a row behind those
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

// Four pairs: their first values a, their second values b.
struct Quad {
    float2 a[2], b[2];
};
__device__ __forceinline__ Quad mul(const Quad& x, const Quad& y) {
    return {{mul2(x.a[0], y.a[0]), mul2(x.a[1], y.a[1])}, {mul2(x.b[0], y.b[0]), mul2(x.b[1], y.b[1])}};
}
__device__ __forceinline__ Quad mul(const Quad& x, float s) {
    const float2 c = both(s);
    return {{mul2(x.a[0], c), mul2(x.a[1], c)}, {mul2(x.b[0], c), mul2(x.b[1], c)}};
}
__device__ __forceinline__ Quad fma(const Quad& x, const Quad& y, const Quad& z) {
    return {{fma2(x.a[0], y.a[0], z.a[0]), fma2(x.a[1], y.a[1], z.a[1])},
            {fma2(x.b[0], y.b[0], z.b[0]), fma2(x.b[1], y.b[1], z.b[1])}};
}
__device__ __forceinline__ Quad fma(const Quad& x, float s, const Quad& z) {
    const float2 c = both(s);
    return {{fma2(x.a[0], c, z.a[0]), fma2(x.a[1], c, z.a[1])}, {fma2(x.b[0], c, z.b[0]), fma2(x.b[1], c, z.b[1])}};
}
__device__ __forceinline__ float dot(const Quad& x, const Quad& y) {
    const float2 s = fma2(x.b[1], y.b[1], fma2(x.b[0], y.b[0], fma2(x.a[1], y.a[1], mul2(x.a[0], y.a[0]))));
    return s.x + s.y;
}

// What a lane turns a head's pairs by: cosines and sines of its four pairs.
struct Turn {
    float2 c[2], s[2], n[2];  // n = -s
};
__device__ __forceinline__ Quad turn_by(const Quad& x, const Turn& t) {
    Quad y;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        y.a[i] = fma2(x.b[i], t.n[i], mul2(x.a[i], t.c[i]));
        y.b[i] = fma2(x.a[i], t.s[i], mul2(x.b[i], t.c[i]));
    }
    return y;
}

// Where a lane's eight values of a head are.  Split (halves, below rot / 8):
// firsts at 4 l, seconds at rot / 2 + 4 l.  Else 8 l .. 8 l + 7, pairs
// interleaved; of the halves' layout these are values that do not turn.  A
// lane behind the head's last value (hd / 8 not a power of two) has none.
template <bool kHalves>
struct Lane {
    int lo, hi;
    bool on;
    __device__ Lane(const Params& p, int l) {
        on = 8 * l < p.hd;
        const bool split = kHalves && on && 8 * l < p.rot;
        lo = split ? 4 * l : on ? 8 * l : 0;
        hi = split ? p.rot / 2 + 4 * l : lo + 4;
    }
    __device__ int value(int i) const { return i < 4 ? lo + i : hi + i - 4; }
    // at: the lane's first value
    __device__ __forceinline__ uint4 load(const __nv_bfloat16* at) const {
        if constexpr (!kHalves) return ld_stream_v4(at);
        const uint2 a = ld_stream_v2(at), b = ld_stream_v2(at + (hi - lo));
        return make_uint4(a.x, a.y, b.x, b.y);
    }
    __device__ __forceinline__ void copy(uint32_t dst, const __nv_bfloat16* at) const {
        if constexpr (!kHalves) {
            cp_async16(dst, at);
        } else {
            cp_async8(dst, at);
            cp_async8(dst + 8, at + (hi - lo));
        }
    }
    __device__ __forceinline__ void store(__nv_bfloat16* at, const uint4& v) const {
        if constexpr (!kHalves) {
            *reinterpret_cast<uint4*>(at) = v;
        } else {
            *reinterpret_cast<uint2*>(at) = make_uint2(v.x, v.y);
            *reinterpret_cast<uint2*>(at + (hi - lo)) = make_uint2(v.z, v.w);
        }
    }
};

template <bool kHalves>
__device__ __forceinline__ Quad quad_of(const uint4& v) {
    const float2 x0 = make_float2(bf16_lo(v.x), bf16_hi(v.x)), x1 = make_float2(bf16_lo(v.y), bf16_hi(v.y));
    const float2 x2 = make_float2(bf16_lo(v.z), bf16_hi(v.z)), x3 = make_float2(bf16_lo(v.w), bf16_hi(v.w));
    if (kHalves) return {{x0, x1}, {x2, x3}};  // a lane that does not turn may hold them in any order
    return {{make_float2(x0.x, x1.x), make_float2(x2.x, x3.x)}, {make_float2(x0.y, x1.y), make_float2(x2.y, x3.y)}};
}
template <bool kHalves>
__device__ __forceinline__ uint4 packed(const Quad& q) {
    if (kHalves)
        return make_uint4(pack_bf16(q.a[0].x, q.a[0].y), pack_bf16(q.a[1].x, q.a[1].y), pack_bf16(q.b[0].x, q.b[0].y),
                          pack_bf16(q.b[1].x, q.b[1].y));
    return make_uint4(pack_bf16(q.a[0].x, q.b[0].x), pack_bf16(q.a[0].y, q.b[0].y), pack_bf16(q.a[1].x, q.b[1].x),
                      pack_bf16(q.a[1].y, q.b[1].y));
}
// A vector of hd values in a lane's order (1 where there is none).
template <bool kHalves>
__device__ __forceinline__ Quad weights_of(const void* w, bool f32, const Lane<kHalves>& l) {
    float f[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] = w && l.on ? load_param(w, l.value(i), f32) : 1.0f;
    if (kHalves) return {{make_float2(f[0], f[1]), make_float2(f[2], f[3])}, {make_float2(f[4], f[5]), make_float2(f[6], f[7])}};
    return {{make_float2(f[0], f[2]), make_float2(f[4], f[6])}, {make_float2(f[1], f[3]), make_float2(f[5], f[7])}};
}

// Cosines and sines of row m's pairs, pair j at c[j], s[j]; pairs that are not
// rotated stay as they are (1, 0).
__device__ __forceinline__ void form_turns(const Params& p, int m, int lane_id, float* c, float* s, float sign) {
    const int pairs = p.lanes * 4;
    for (int j = lane_id; j < pairs; j += 32) {
        float cj = 1.0f, sj = 0.0f;
        if (j < p.rot / 2) {
            int a = 0;
            while (a + 1 < p.n_axes && j >= p.axis_end[a]) ++a;
            const uint32_t raw = __ldg(static_cast<const uint32_t*>(p.pos) + (int64_t)m * p.n_axes + a);
            const double pos = p.pos_f32 ? (double)__uint_as_float(raw) : (double)(int)raw;
            const double t = pos * __ldg(p.freqs + j) * 0.15915494309189533577;
            sincospif((float)(2.0 * (t - rint(t))), &sj, &cj);
        }
        c[j] = cj;
        s[j] = sign * sj;
    }
}

// Over the lanes of a head (a power of two).
__device__ __forceinline__ float head_sum(float v, int lanes) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        const float w = __shfl_xor_sync(0xFFFFFFFFu, v, o);
        if (o < lanes) v += w;
    }
    return v;
}

__device__ __forceinline__ float2 head_sum(float2 v, int lanes) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        const float2 w = make_float2(__shfl_xor_sync(0xFFFFFFFFu, v.x, o), __shfl_xor_sync(0xFFFFFFFFu, v.y, o));
        if (o < lanes) v = add2(v, w);
    }
    return v;
}

template <bool kBwd, bool kHalves, bool kNorm>
__global__ void __maxnreg__((kRegs<kBwd, kNorm>)) k_qk_rope(const __grid_constant__ Params p) {
    constexpr int U = kU<kBwd, kNorm>;
    extern __shared__ __align__(16) uint8_t ring_mem[];
    const uint32_t ring = smem_u32(ring_mem) + threadIdx.x * 16;  // + ((stage * U + u) * 2 + operand) * kThreads * 16
    __shared__ __align__(16) float cs[kWarps][2][kMaxPairs];
    __shared__ float red[32];
    __shared__ float4 dws[kBwd && kNorm ? 2 * 2 * kThreads : 1];  // a thread's sums for w_q and w_k
    __shared__ float sums[kBwd && kNorm ? 2 * 256 : 1];
    const int warp = threadIdx.x >> 5, lane_id = threadIdx.x & 31;
    const int lanes = p.lanes, groups = 32 / lanes, group = lane_id / lanes;
    const int l = lane_id - group * lanes;
    const Lane<kHalves> lane(p, l);
    if constexpr (kBwd && kNorm) {
#pragma unroll
        for (int i = 0; i < 4; ++i) dws[i * kThreads + threadIdx.x] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    }
    grid_dep_launch();
    grid_dep_wait();
    uint32_t amax = 0;
    const bool even = p.hd == 8 * lanes;  // every lane has values
    // A row's heads in turns of `groups`: queries, keys, values; a slice takes
    // its share of the turns.  32 bits hold tasks and turns times slices: only
    // the rows of the last round are sliced.
    const int nq = (p.Hq + groups - 1) / groups, nk = (p.Hk + groups - 1) / groups, nv = (p.Hv + groups - 1) / groups;
    const int total = nq + nk + nv;
    const uint32_t whole_rows = p.whole, slices = p.slices, stride = gridDim.x * kWarps;
    const uint32_t tasks = whole_rows + ((uint32_t)p.M - whole_rows) * slices;
    for (uint32_t task = blockIdx.x * kWarps + warp; task < tasks; task += stride) {
        int m = (int)task, from = 0, to = total;
        if (task >= whole_rows) {
            const uint32_t part = task - whole_rows, row = part / slices, slice = part - row * slices;
            m = (int)(whole_rows + row);
            from = (int)(total * slice / slices);
            to = (int)(total * (slice + 1) / slices);
        }
        const int b = m / p.S, s = m - b * p.S;
        // this lane's values of its group's first head
        const __nv_bfloat16* x = p.x + (int64_t)m * p.ld + group * p.hd + lane.lo;
        __nv_bfloat16* dx = kBwd ? p.dx + (int64_t)m * p.lddx + group * p.hd + lane.lo : nullptr;
        const int near_step = groups * p.hd;
        Turn t;
        bool formed = false;
        auto form = [&]() {
            form_turns(p, m, lane_id, cs[warp][0], cs[warp][1], kBwd ? -1.0f : 1.0f);
            __syncwarp();
            const float4 c = *reinterpret_cast<const float4*>(&cs[warp][0][4 * l]);
            const float4 n = *reinterpret_cast<const float4*>(&cs[warp][1][4 * l]);
            __syncwarp();
            t.c[0] = make_float2(c.x, c.y), t.c[1] = make_float2(c.z, c.w);
            t.s[0] = make_float2(n.x, n.y), t.s[1] = make_float2(n.z, n.w);
            t.n[0] = make_float2(-n.x, -n.y), t.n[1] = make_float2(-n.z, -n.w);
            formed = true;
        };
#pragma unroll
        for (int kind = 0; kind < 3; ++kind) {  // queries, keys, values (as they are)
            const int first = kind == 0 ? 0 : kind == 1 ? nq : nq + nk;
            const int heads = kind == 0 ? p.Hq : kind == 1 ? p.Hk : p.Hv;
            const int lo = max(from - first, 0);
            const int hi = min(to - first, kind == 0 ? nq : kind == 1 ? nk : nv);
            if (lo >= hi) continue;
            const int whole = even ? heads / groups : 0;  // turns without an idle lane
            const Heads& side = kind == 0 ? p.q : kind == 1 ? p.k : p.v;
            // the operand of the attention, and this row's part of qkv
            const int64_t far_step = groups * side.sh;
            __nv_bfloat16* far = side.p + b * side.sb + s * side.st + group * side.sh + lane.lo + lo * far_step;
            const int near = (kind == 0 ? 0 : kind == 1 ? p.Hq : p.Hq + p.Hk) * p.hd + lo * near_step;
            const __nv_bfloat16* xk = x + near;
            __nv_bfloat16* dxk = kBwd ? dx + near : nullptr;
            Quad w, dw = {};
            if (kNorm && kind < 2) w = weights_of<kHalves>(kind ? p.w_k : p.w_q, p.p32, lane);
            auto has = [&](int turn) { return turn < hi && turn * groups + group < heads && lane.on; };
            const int full_to = min(hi, whole);
            const __nv_bfloat16 *far_ahead = far, *x_ahead = xk;
            auto issue = [&](int turn, uint32_t slot) {  // a batch into the ring
                if (turn + U <= full_to) {
#pragma unroll
                    for (int u = 0; u < U; ++u) {
                        lane.copy(slot + 2 * u * kThreads * 16, far_ahead + u * far_step);
                        lane.copy(slot + (2 * u + 1) * kThreads * 16, x_ahead + u * near_step);
                    }
                } else {
#pragma unroll
                    for (int u = 0; u < U; ++u)
                        if (has(turn + u)) {
                            lane.copy(slot + 2 * u * kThreads * 16, far_ahead + u * far_step);
                            lane.copy(slot + (2 * u + 1) * kThreads * 16, x_ahead + u * near_step);
                        }
                }
                far_ahead += U * far_step;
                x_ahead += U * near_step;
                cp_async_commit();
            };
            auto batch = [&](int turn, auto full, uint32_t slot) {
                constexpr bool kFull = decltype(full)::value;
                uint4 in[U], ix[U];
                bool live[U];
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    live[u] = kFull || has(turn + u);
                    if (!kFull) in[u] = ix[u] = make_uint4(0, 0, 0, 0);
                    if (live[u]) {
                        if (kRing<kBwd, kNorm> && kind < 2) {
                            in[u] = ld_shared_v4(slot + 2 * u * kThreads * 16);
                            ix[u] = ld_shared_v4(slot + (2 * u + 1) * kThreads * 16);
                        } else {
                            in[u] = lane.load(kBwd ? far + u * far_step : xk + u * near_step);
                        }
                    }
                }
                if (kind < 2 && !formed) form();  // while the first heads arrive
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    uint4 v = in[u];
                    if (kind < 2) {
                        Quad f = quad_of<kHalves>(v);
                        if (!kBwd) {
                            if (kNorm) {
                                const float rstd = rsqrtf(fmaf(head_sum(dot(f, f), lanes), p.inv_hd, p.eps));
                                f = mul(mul(f, w), rstd);
                            }
                            f = turn_by(f, t);
                        } else {
                            f = turn_by(f, t);
                            if (kNorm) {
                                const Quad xq = quad_of<kHalves>(ix[u]);
                                // both sums over the head at once: z x, and x x
                                const Quad z = mul(f, w);
                                const float2 q = head_sum(make_float2(dot(xq, xq), dot(z, xq)), lanes);
                                const float rstd = rsqrtf(fmaf(q.x, p.inv_hd, p.eps));
                                const Quad g = mul(xq, rstd);
                                dw = fma(f, g, dw);
                                f = mul(fma(g, -q.y * rstd * p.inv_hd, z), rstd);
                            }
                        }
                        v = packed<kHalves>(f);
                    }
                    if (live[u]) {
                        lane.store(kBwd ? dxk + u * near_step : far + u * far_step, v);
                        if (kBwd) amax = max_mag8(amax, v);
                    }
                }
                far += U * far_step;
                xk += U * near_step;
                if (kBwd) dxk += U * near_step;
            };
            int turn = lo;
            if (kRing<kBwd, kNorm> && kind < 2) {
                constexpr uint32_t kStage = 2 * U * kThreads * 16;
#pragma unroll
                for (int k = 0; k < kDepth - 1; ++k) issue(lo + k * U, ring + k * kStage);
                uint32_t slot = ring, ahead = ring + (kDepth - 1) * kStage;
                for (; turn < hi; turn += U) {
                    issue(turn + (kDepth - 1) * U, ahead);
                    if (!formed) form();
                    cp_async_wait<kDepth - 1>();
                    if (turn + U <= full_to)
                        batch(turn, std::true_type(), slot);
                    else
                        batch(turn, std::false_type(), slot);
                    ahead = slot;
                    slot = slot == ring + (kDepth - 1) * kStage ? ring : slot + kStage;
                }
            } else {
                for (; turn + U <= full_to; turn += U) batch(turn, std::true_type(), 0u);
                for (; turn < hi; turn += U) batch(turn, std::false_type(), 0u);
            }
            if constexpr (kBwd && kNorm) {
                if (kind < 2 && p.partial) {
                    float4* at = dws + 2 * kind * kThreads + threadIdx.x;
                    float4 a = at[0], c = at[kThreads];
                    a = make_float4(a.x + dw.a[0].x, a.y + dw.a[0].y, a.z + dw.a[1].x, a.w + dw.a[1].y);
                    c = make_float4(c.x + dw.b[0].x, c.y + dw.b[0].y, c.z + dw.b[1].x, c.w + dw.b[1].y);
                    at[0] = a;
                    at[kThreads] = c;
                }
            }
        }
    }
    if constexpr (kBwd) {
        raise_amax(p.amax, amax_of(amax), red);
        if constexpr (kNorm) {
            if (p.partial) {
                // groups of a warp by shuffles, then the warps in turn
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    const float4 a = dws[2 * k * kThreads + threadIdx.x], c = dws[(2 * k + 1) * kThreads + threadIdx.x];
                    float f[8] = {a.x, a.y, a.z, a.w, c.x, c.y, c.z, c.w};
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        for (int o = p.lanes; o < 32; o <<= 1) f[i] += __shfl_xor_sync(0xFFFFFFFFu, f[i], o);
                    // f[i]: firsts 0..3, seconds 0..3 of the pairs
                    for (int w = 0; w < kWarps; ++w) {
                        if (w == warp && group == 0 && lane.on) {
#pragma unroll
                            for (int i = 0; i < 8; ++i) {
                                const int at = k * 256 + (kHalves ? lane.value(i) : lane.lo + 2 * (i & 3) + (i >> 2));
                                sums[at] = w == 0 ? f[i] : sums[at] + f[i];
                            }
                        }
                        __syncthreads();
                    }
                }
                float* out = p.partial + (int64_t)blockIdx.x * 2 * p.hd;
                for (int i = threadIdx.x; i < 2 * p.hd; i += kThreads)
                    out[i] = sums[i < p.hd ? i : 256 + i - p.hd];
            }
        }
    }
}

// dw_q, dw_k from the blocks' partial sums: 8 columns per block, a thread per
// column and every 128th partial row, so that few loads follow one another (32
// columns and every 32nd row: a backward call of 53.4 us instead of 51.6).
__global__ void __launch_bounds__(1024) k_qk_rope_reduce(const float* partial, int blocks, int hd, float* dw_q,
                                                         float* dw_k) {
    __shared__ float part[32][9];
    const int col = threadIdx.x & 7, warp = threadIdx.x >> 5, lane = threadIdx.x & 31, c = blockIdx.x * 8 + col;
    grid_dep_launch();
    grid_dep_wait();
    float s = 0.0f;  // 2 hd is a multiple of 8: every column is there
#pragma unroll 8
    for (int b = threadIdx.x >> 3; b < blocks; b += 128) s += __ldg(partial + (int64_t)b * 2 * hd + c);
    s += __shfl_xor_sync(0xFFFFFFFFu, s, 8);
    s += __shfl_xor_sync(0xFFFFFFFFu, s, 16);
    if (lane < 8) part[warp][col] = s;
    __syncthreads();
    if (warp == 0) {
        s = 0.0f;
#pragma unroll
        for (int i = 0; i < 8; ++i) s += part[4 * i + (lane >> 3)][col];
        s += __shfl_xor_sync(0xFFFFFFFFu, s, 8);
        s += __shfl_xor_sync(0xFFFFFFFFu, s, 16);
        float* out = c < hd ? dw_q : dw_k;
        if (lane < 8 && out) out[c < hd ? c : c - hd] = s;
    }
}

}  // namespace rope
}  // namespace ft
