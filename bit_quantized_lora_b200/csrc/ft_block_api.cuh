// ft_block_api.cuh -- the host side of the operators around the linears:
// argument checks, launch shapes, launches.  Part of ft_api.cu's translation
// unit (its launch helpers and timing).
#pragma once

namespace {

constexpr int64_t kMaxRows = int64_t(1) << 30;  // row counters are 32-bit and step past the end by a grid
constexpr int64_t kNormMaxD = 8192;

inline bool al4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }
inline bool al8(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 7u) == 0; }
inline bool dtype_ok(int t) { return t == FT_BF16 || t == FT_F32; }
// A row-major matrix whose rows start on 16-byte boundaries.
inline bool rows_al16(const void* p, int64_t ld, int elem) { return al16(p) && (ld * elem) % 16 == 0; }

// ------------------------------------------------------------ gated norm
// Threads of a row: below 33 vectors of eight a power of two of lanes, with
// several rows per block; above, a block of its own with `v` vectors per
// thread.
struct RowShape {
    bool wide;
    int v, tpr, threads;
};
RowShape row_shape(int64_t D, bool backward) {
    const int nvec = (int)(D / 8);
    if (nvec <= 32) {
        int t = 8;
        while (t < nvec) t *= 2;
        return {false, 1, t, 256};
    }
    const int v = backward ? (nvec > 512 ? 2 : 1) : nvec <= 128 ? 1 : nvec <= 256 ? 2 : 4;
    const int t = (cdiv(nvec, v) + 31) / 32 * 32;
    return {true, v, t, t};
}

// Rows of a block of the backward: as many blocks as the device holds at once
// (by registers and by the ring of an FP32 stream, the larger one), so that
// all start together and each writes one row of partial sums per sample.
constexpr int kBwdSms = 148;
int64_t norm_bwd_chunk(int64_t M, int64_t D, bool mod) {
    using namespace ft::norm;
    const RowShape s = row_shape(D, true);
    const int regs = !s.wide   ? kBwdRegs<1, false, false>
                     : s.v == 1 ? (mod ? kBwdRegs<1, true, true> : kBwdRegs<1, true, false>)
                                : (mod ? kBwdRegs<2, true, true> : kBwdRegs<2, true, false>);
    const int ring = kBwdStages * (s.v == 1 ? Ring<kBwdSlots<float>, 1>::bytes(s.threads)
                                            : Ring<kBwdSlots<float>, 2>::bytes(s.threads));
    // each of an SM's four schedulers has 16384 registers for its warps
    const int warps = 4 * (16384 / (32 * regs));
    const int64_t blocks =
        (int64_t)kBwdSms * std::max(1, std::min({warps / (s.threads / 32), 220 * 1024 / ring, 8}));
    const int64_t rows = s.wide ? 1 : s.threads / s.tpr;  // of a turn
    const int64_t c = (M + blocks - 1) / blocks;
    return std::max<int64_t>(1, (c + rows - 1) / rows) * rows;
}
size_t norm_bwd_partials(int64_t M, int64_t D, int64_t B) {
    const int64_t chunk = std::min(norm_bwd_chunk(M, D, false), norm_bwd_chunk(M, D, true));
    return (size_t)((M + chunk - 1) / chunk + B) * 3 * (size_t)D;
}
// The sums that a backward leaves in a workspace: behind the linears' words,
// which an FP32 sum over them would break for every later call of theirs, at a
// multiple of 4 KB (the rotation's rows of sums are 1 KB: from 512 bytes into
// one a backward call of 4608 rows took 51.9 us instead of 51.6).
constexpr size_t kWsSums = (kWsWords + 4095) / 4096 * 4096;
float* ws_sums(void* ws) { return ws ? reinterpret_cast<float*>(static_cast<uint8_t*>(ws) + kWsSums) : nullptr; }

ft_status check_norm(const ft_gated_norm* n) {
    if (!n || n->M < 0 || n->D < 0 || n->B < 1) return FT_ERR_INVALID_ARG;
    if (n->pre < FT_NORM_NONE || n->pre > FT_NORM_LAYER || n->post < FT_NORM_NONE || n->post > FT_NORM_LAYER)
        return FT_ERR_INVALID_ARG;
    if (!dtype_ok(n->xt) || !dtype_ok(n->pt)) return FT_ERR_INVALID_ARG;
    if (!(n->eps_pre >= 0.0f) || !(n->eps_post >= 0.0f)) return FT_ERR_INVALID_ARG;
    if (n->w_post && n->post == FT_NORM_NONE) return FT_ERR_INVALID_ARG;
    if (n->pre == FT_NORM_NONE && (n->scale || n->shift || n->w || n->bias)) return FT_ERR_INVALID_ARG;
    if (n->D < 8 || n->D % 8 || n->D > kNormMaxD || n->M > kMaxRows || n->B > kMaxRows) return FT_ERR_SHAPE;
    if (!n->offsets && n->M % n->B) return FT_ERR_SHAPE;
    const int ps = n->pt == FT_F32 ? 4 : 2;
    const void* mods[3] = {n->gate, n->scale, n->shift};
    const int64_t lds[3] = {n->ld_gate, n->ld_scale, n->ld_shift};
    for (int i = 0; i < 3; ++i) {
        if (!mods[i]) continue;
        if (n->B > 1 && lds[i] != 0 && lds[i] < n->D) return FT_ERR_SHAPE;
        if (!rows_al16(mods[i], n->B > 1 ? lds[i] : 0, ps)) return FT_ERR_ALIGN;
    }
    for (const void* q : {n->w_post, n->w, n->bias})
        if (q && !al16(q)) return FT_ERR_ALIGN;
    if (n->offsets && !al4(n->offsets)) return FT_ERR_ALIGN;
    return FT_OK;
}

uint32_t norm_has(const ft_gated_norm* n) {
    using namespace ft::norm;
    return (n->gate ? kGate : 0u) | (n->scale ? kScale : 0u) | (n->shift ? kShift : 0u) | (n->w ? kW : 0u) |
           (n->bias ? kBias : 0u) | (n->w_post ? kWPost : 0u) | (n->pre != FT_NORM_NONE ? kPre : 0u) |
           (n->pre == FT_NORM_LAYER ? kPreMean : 0u) | (n->post != FT_NORM_NONE ? kPost : 0u) |
           (n->post == FT_NORM_LAYER ? kPostMean : 0u);
}
// Blocks of `k` that an SM holds; lets the kernel take its shared memory
// first.  Asked once per kernel and launch shape in a context.  The limit is
// the kernel's, and one kernel serves many widths: it is only ever raised, so
// that a shape asked for before (or by another thread meanwhile) still fits.
ft_status blocks_per_sm(const void* k, int threads, size_t smem, DevInfo* d, int* out) {
    try {
        std::lock_guard<std::mutex> lk(g_mu);
        int& n = d->per_sm[std::make_tuple(k, threads, smem)];
        if (n == 0) {
            int got = 0;
            size_t& allowed = d->smem_allowed[k];
            // 32 KB and the static part are less than a launch may take unasked
            if (smem > std::max<size_t>(allowed, 32 * 1024)) {
                FT_TRY(cuda_ok(cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem)));
                allowed = smem;
            }
            FT_TRY(cuda_ok(cudaOccupancyMaxActiveBlocksPerMultiprocessor(&got, k, threads, smem)));
            n = std::max(1, got);
        }
        *out = n;
        return FT_OK;
    } catch (...) {  // no memory for the entry: nothing may leave a C entry point
        return FT_ERR_CUDA;
    }
}
// Launches `k` with `smem` bytes of dynamic shared memory per block, the grid
// cut to the blocks that the device holds at once when `resident` is set.
template <typename P>
ft_status launch_norm(void (*k)(P), const P& p, int grid, bool resident, int threads, size_t smem, DevInfo* d,
                      cudaStream_t st) {
    int per_sm = 1;
    FT_TRY(blocks_per_sm(reinterpret_cast<const void*>(k), threads, smem, d, &per_sm));
    if (resident && grid > d->sms) grid = cdiv(grid, cdiv(grid, per_sm * d->sms));  // the same number of turns each
    return launch_overlapped(k, grid, threads, smem, st, p);
}
template <typename XT, int V, bool kWide, bool k32>
ft_status launch_norm_fwd(const ft::norm::FwdParams& p, const RowShape& s, int grid, bool mod, DevInfo* d,
                          cudaStream_t st) {
    using namespace ft::norm;
    const size_t smem = kFwdStages * Ring<kFwdSlots<XT>, V>::bytes(s.threads);
    if constexpr (kWide)
        if (mod) return launch_norm(k_gated_norm_fwd<XT, V, kWide, k32, true>, p, grid, true, s.threads, smem, d, st);
    return launch_norm(k_gated_norm_fwd<XT, V, kWide, k32, false>, p, grid, true, s.threads, smem, d, st);
}
template <typename XT, int V, bool kWide, bool k32>
ft_status launch_norm_bwd(const ft::norm::BwdParams& p, const RowShape& s, int grid, bool mod, DevInfo* d,
                          cudaStream_t st) {
    using namespace ft::norm;
    const size_t smem = kBwdStages * Ring<kBwdSlots<XT>, V>::bytes(s.threads);
    if constexpr (kWide)
        if (mod) return launch_norm(k_gated_norm_bwd<XT, V, kWide, k32, true>, p, grid, false, s.threads, smem, d, st);
    return launch_norm(k_gated_norm_bwd<XT, V, kWide, k32, false>, p, grid, false, s.threads, smem, d, st);
}
constexpr uint32_t kFwdMod = ft::norm::kY | ft::norm::kGate | ft::norm::kScale | ft::norm::kShift | ft::norm::kPre;
constexpr uint32_t kBwdMod = ft::norm::kDh | ft::norm::kDr | ft::norm::kR | ft::norm::kY | ft::norm::kGate |
                             ft::norm::kScale | ft::norm::kDx | ft::norm::kDy | ft::norm::kPre | ft::norm::kStats;
constexpr uint32_t kNotMod = ft::norm::kW | ft::norm::kBias | ft::norm::kWPost | ft::norm::kPost;
template <typename XT, bool k32>
ft_status launch_norm(const ft::norm::FwdParams& p, const RowShape& s, int grid, DevInfo* d, cudaStream_t st) {
    const bool mod = (p.has & kFwdMod) == kFwdMod && !(p.has & kNotMod);
    if (!s.wide) return launch_norm_fwd<XT, 1, false, k32>(p, s, grid, false, d, st);
    if (s.v == 1) return launch_norm_fwd<XT, 1, true, k32>(p, s, grid, mod, d, st);
    if (s.v == 2) return launch_norm_fwd<XT, 2, true, k32>(p, s, grid, mod, d, st);
    return launch_norm_fwd<XT, 4, true, k32>(p, s, grid, mod, d, st);
}
bool norm_bwd_mod(const ft::norm::BwdParams& p) {
    return (p.has & kBwdMod) == kBwdMod && !(p.has & kNotMod);
}
template <typename XT, bool k32>
ft_status launch_norm(const ft::norm::BwdParams& p, const RowShape& s, int grid, DevInfo* d, cudaStream_t st) {
    const bool mod = norm_bwd_mod(p);
    if (!s.wide) return launch_norm_bwd<XT, 1, false, k32>(p, s, grid, false, d, st);
    if (s.v == 1) return launch_norm_bwd<XT, 1, true, k32>(p, s, grid, mod, d, st);
    return launch_norm_bwd<XT, 2, true, k32>(p, s, grid, mod, d, st);
}
template <typename P>
ft_status launch_norm(const P& p, int xt, const RowShape& s, int grid, DevInfo* d, cudaStream_t st) {
    if (xt == FT_F32) return p.p32 ? launch_norm<float, true>(p, s, grid, d, st) : launch_norm<float, false>(p, s, grid, d, st);
    return p.p32 ? launch_norm<__nv_bfloat16, true>(p, s, grid, d, st)
                 : launch_norm<__nv_bfloat16, false>(p, s, grid, d, st);
}

// ------------------------------------------------------------ rope
constexpr int kRopeSms = 148;
constexpr int kRopeMaxBlocks = kRopeSms * 8;

ft_status check_rope(const ft_rope* R) {
    if (!R || R->M < 0 || R->S < 0 || R->Hq < 0 || R->Hk < 0 || R->n_axes < 1 || R->n_axes > 4)
        return FT_ERR_INVALID_ARG;
    if (R->layout != FT_ROPE_PAIRS && R->layout != FT_ROPE_HALVES) return FT_ERR_INVALID_ARG;
    if (R->norm != FT_NORM_NONE && R->norm != FT_NORM_RMS) return FT_ERR_INVALID_ARG;
    if (R->pos_t != FT_POS_I32 && R->pos_t != FT_POS_F32) return FT_ERR_INVALID_ARG;
    if (!dtype_ok(R->pt) || !(R->eps >= 0.0f)) return FT_ERR_INVALID_ARG;
    if ((R->w_q || R->w_k) && R->norm == FT_NORM_NONE) return FT_ERR_INVALID_ARG;
    if (R->hd < 8 || R->hd % 8 || R->hd > 256 || R->Hq > 65536 || R->Hk > 65536) return FT_ERR_SHAPE;
    int64_t rot = 0;
    for (int a = 0; a < R->n_axes; ++a) {
        if (R->axis_dims[a] < 0 || R->axis_dims[a] > R->hd || R->axis_dims[a] % 2) return FT_ERR_SHAPE;
        rot += R->axis_dims[a];
    }
    if (rot > R->hd || (R->layout == FT_ROPE_HALVES && rot % 8)) return FT_ERR_SHAPE;
    if (R->M > kMaxRows) return FT_ERR_SHAPE;
    if (R->M > 0 && (R->S < 1 || R->M % R->S)) return FT_ERR_SHAPE;
    if (R->M > 0 && rot > 0 && (!R->pos || !R->freqs)) return FT_ERR_INVALID_ARG;
    if (!al4(R->pos) || !al8(R->freqs)) return FT_ERR_ALIGN;
    const uintptr_t wmask = R->pt == FT_F32 ? 3u : 1u;
    if (((uintptr_t)R->w_q | (uintptr_t)R->w_k) & wmask) return FT_ERR_ALIGN;
    return FT_OK;
}
ft_status check_heads(const ft_heads* h, int heads, bool needed) {
    if (!h) return FT_ERR_INVALID_ARG;
    if (heads == 0 || (!needed && !h->p)) return FT_OK;
    if (!h->p) return FT_ERR_INVALID_ARG;
    if (!al16(h->p) || h->sb % 8 || h->sh % 8 || h->st % 8) return FT_ERR_ALIGN;
    return FT_OK;
}
ft::rope::Heads to_heads(const ft_heads* h) {
    return {static_cast<__nv_bfloat16*>(h->p), h->sb, h->sh, h->st};
}
ft::rope::Params rope_params(const ft_rope* R, const ft_heads* q, const ft_heads* k, const ft_heads* v) {
    ft::rope::Params p = {};
    p.M = (int)R->M;
    p.S = (int)std::max<int64_t>(1, R->S);
    p.Hq = R->Hq;
    p.Hk = R->Hk;
    p.hd = R->hd;
    p.Hv = v->p ? R->Hk : 0;
    p.halves = R->layout == FT_ROPE_HALVES;
    p.norm = R->norm != FT_NORM_NONE;
    p.pos_f32 = R->pos_t == FT_POS_F32;
    p.p32 = R->pt == FT_F32;
    p.n_axes = R->n_axes;
    for (int a = 0, end = 0; a < R->n_axes; ++a) {
        p.rot += R->axis_dims[a];
        p.axis_end[a] = end += R->axis_dims[a] / 2;
    }
    p.lanes = 1;
    while (8 * p.lanes < p.hd) p.lanes *= 2;
    p.eps = R->eps;
    p.inv_hd = 1.0f / (float)R->hd;
    p.pos = R->pos;
    p.freqs = R->freqs;
    p.w_q = R->w_q;
    p.w_k = R->w_k;
    p.q = to_heads(q);
    p.k = to_heads(k);
    p.v = to_heads(v);
    return p;
}
// Warps over rows, as many as the device holds, in rounds.  The rows of the
// last round, fewer than there are warps, are cut into slices of whole turns:
// into as many as there are warps for when that is two or more (few rows), else
// into up to six where rounding up the slices' rounds costs less than rounding
// up the rows' (forming a row's turns again is about a fourteenth of its work).
// 4608 rows of 24 heads backward: 2960 whole and 1648 in three, 50.5 us a
// launch against 51.8 us with whole rows only.
template <bool kBwd>
int rope_grid(ft::rope::Params* p) {
    using namespace ft::rope;
    const int groups = 32 / p->lanes;
    const int turns = cdiv(p->Hq, groups) + cdiv(p->Hk, groups) + cdiv(p->Hv, groups);
    const int regs = p->norm ? kRegs<kBwd, true> : kRegs<kBwd, false>;
    const int blocks = std::min(kRopeMaxBlocks, kRopeSms * (4 * (16384 / (32 * regs)) / kWarps));
    const int64_t warps = (int64_t)blocks * kWarps, rest = p->M % warps;
    p->whole = (int)(p->M - rest);
    p->slices = 1;
    if (rest > 0 && rest * 2 <= warps) {
        p->slices = (int)std::min<int64_t>(turns, warps / rest);
    } else if (rest > 0) {
        double best = 1.0;
        for (int s = 2; s <= std::min(6, turns); ++s) {
            const double cost = (double)((rest * s + warps - 1) / warps) / s * (1.0 + 0.07 * (s - 1));
            if (cost < best) best = cost, p->slices = s;
        }
    }
    return (int)std::min<int64_t>((p->whole + rest * p->slices + kWarps - 1) / kWarps, blocks);
}
template <bool kBwd>
ft_status launch_rope(const ft::rope::Params& p, int grid, DevInfo* d, cudaStream_t st) {
    using namespace ft::rope;
    auto* k = p.halves ? (p.norm ? k_qk_rope<kBwd, true, true> : k_qk_rope<kBwd, true, false>)
                       : (p.norm ? k_qk_rope<kBwd, false, true> : k_qk_rope<kBwd, false, false>);
    const size_t smem = p.norm ? kRingBytes<kBwd, true> : kRingBytes<kBwd, false>;
    int per_sm = 1;
    if (smem) FT_TRY(blocks_per_sm(reinterpret_cast<const void*>(k), kThreads, smem, d, &per_sm));
    return launch_overlapped(k, grid, kThreads, smem, st, p);
}

// ------------------------------------------------------------ adamw
// Tensors of one launch: the list rides in the launch's parameters (4 KB for
// the small form; 32 KB is the most a launch takes).
constexpr int kAdamFew = 40, kAdamMany = 340;

template <bool k8, int kMax>
ft_status launch_adamw(const ft::adamw::Params<kMax>& p, DevInfo* d, cudaStream_t st) {
    const int grid = (int)std::max<int64_t>(1, std::min<int64_t>(p.units, (int64_t)d->sms * ft::adamw::kPerSm));
    LaunchTimer lt(KID_ADAMW, st);
    const ft_status s = launch_overlapped(ft::adamw::k_adamw<k8, kMax>, grid, 32 * ft::adamw::kWarps, 0, st, p);
    lt.stop();
    return s;
}

template <int kMax>
ft_status adamw_group(const ft_adamw_tensor* t, int64_t begin, int64_t end, const ft_adamw_hyper* h, bool k8, bool last,
                      int64_t* step, const float* lr_dev, const float* grad_scale, DevInfo* d, cudaStream_t st) {
    ft::adamw::Params<kMax> p = {};
    p.b1 = (float)h->beta1;
    p.c1 = (float)(1.0 - h->beta1);
    p.b2 = (float)h->beta2;
    p.c2 = (float)(1.0 - h->beta2);
    p.eps = (float)h->eps;
    p.lr = h->lr;
    p.log_b1 = std::log(h->beta1);
    p.log_b2 = std::log(h->beta2);
    p.lr_dev = lr_dev;
    p.grad_scale = grad_scale;
    p.step = reinterpret_cast<long long*>(step);
    p.last = last;
    // The fast root leaves out what a subnormal v adds to eps, at most
    // 1.1e-19 / sqrt(1 - beta2): below 2^-21 of eps it does not count.
    p.exact = !(h->eps * std::sqrt(1.0 - h->beta2) >= 2.5e-13);
    for (int64_t i = begin; i < end; ++i) {
        const ft_adamw_tensor& a = t[i];
        if (a.n == 0) continue;
        ft::adamw::Tensor& q = p.t[p.count++];
        q.p = a.p;
        q.p16 = static_cast<__nv_bfloat16*>(a.p16);
        q.g = a.grad;
        q.m = a.m;
        q.v = a.v;
        q.ms = a.m_scale;
        q.vs = a.v_scale;
        q.n = a.n;
        q.wd = a.weight_decay;
        q.g16 = a.gt == FT_BF16;
        q.vec = al16(a.p) && al8(a.p16) && (q.g16 ? al8(a.grad) : al16(a.grad)) &&
                (k8 ? al4(a.m) && al4(a.v) : al16(a.m) && al16(a.v));
        q.usual = q.vec && !q.g16 && a.p && a.p16;
        q.first = p.units;
        p.units += (unsigned)((a.n + ft::adamw::kUnit - 1) / ft::adamw::kUnit);
    }
    return k8 ? launch_adamw<true, kMax>(p, d, st) : launch_adamw<false, kMax>(p, d, st);
}

}  // namespace

extern "C" {

size_t ft_gated_norm_workspace_bytes(int64_t M, int64_t D, int64_t B) {
    if (M < 0 || M > kMaxRows || D < 8 || D % 8 || D > kNormMaxD || B < 1 || B > kMaxRows) return 0;
    return kWsSums + (norm_bwd_partials(M, D, B) + (size_t)B * 3 * (size_t)D) * sizeof(float);
}

ft_status ft_gated_norm_fwd(const ft_gated_norm* n, const void* x, int64_t ldx, const void* y, int64_t ldy, void* r,
                            int64_t ldr, void* h, int64_t ldh, float* stats, float* amax_h, void* stream) {
    FT_TRY(check_norm(n));
    const bool rows = n->M > 0;
    if (rows) {
        if (!x || (n->pre == FT_NORM_NONE) != (h == nullptr)) return FT_ERR_INVALID_ARG;
        if (!y && (r || n->gate || n->post != FT_NORM_NONE)) return FT_ERR_INVALID_ARG;
        if ((y && !r) || (amax_h && !h)) return FT_ERR_INVALID_ARG;
    }
    const int xs = n->xt == FT_F32 ? 4 : 2;
    if (ldx < n->D || (y && (ldy < n->D || ldr < n->D)) || (h && ldh < n->D)) return FT_ERR_SHAPE;
    if (!rows_al16(x, ldx, xs) || (y && (!rows_al16(y, ldy, 2) || !rows_al16(r, ldr, xs))) ||
        (h && !rows_al16(h, ldh, 2)) || !al16(stats) || !al4(amax_h))
        return FT_ERR_ALIGN;
    if (!rows || (!y && !h && !stats)) return FT_OK;
    DevInfo* d;
    FT_TRY(device_info(&d));
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    const RowShape s = row_shape(n->D, false);
    ft::norm::FwdParams p = {};
    p.M = (int)n->M;
    p.D = (int)n->D;
    p.B = (int)n->B;
    p.S = (int)(n->M / n->B);
    p.offsets = n->offsets;
    p.eps_pre = n->eps_pre;
    p.eps_post = n->eps_post;
    p.alpha = n->alpha;
    p.inv_d = 1.0f / (float)n->D;
    p.p32 = n->pt == FT_F32;
    p.ld_gate = n->B > 1 ? n->ld_gate : 0;
    p.ld_scale = n->B > 1 ? n->ld_scale : 0;
    p.ld_shift = n->B > 1 ? n->ld_shift : 0;
    p.gate = n->gate;
    p.scale = n->scale;
    p.shift = n->shift;
    p.w_post = n->w_post;
    p.w = n->w;
    p.bias = n->bias;
    p.x = x;
    p.ldx = ldx;
    p.y = static_cast<const __nv_bfloat16*>(y);
    p.ldy = ldy;
    p.r = r;
    p.ldr = ldr;
    p.h = static_cast<__nv_bfloat16*>(h);
    p.ldh = ldh;
    p.stats = reinterpret_cast<float4*>(stats);
    p.amax = amax_h;
    p.tpr = s.tpr;
    p.has = norm_has(n) | (y ? ft::norm::kY : 0u) | (stats ? ft::norm::kStats : 0u);
    const int per = s.wide ? 1 : s.threads / s.tpr;
    const int grid = cdiv(n->M, per);
    LaunchTimer lt(KID_NORM_FWD, st);
    const ft_status e = launch_norm(p, n->xt, s, grid, d, st);
    lt.stop();
    return e;
}

ft_status ft_gated_norm_bwd(const ft_gated_norm* n, const void* dh, int64_t lddh, const void* dr, int64_t lddr,
                            const void* r, int64_t ldr, const void* y, int64_t ldy, const float* stats,
                            const ft_gated_norm_grads* g, void* ws, size_t ws_bytes, void* stream) {
    FT_TRY(check_norm(n));
    if (!g) return FT_ERR_INVALID_ARG;
    const bool rows = n->M > 0, pre = n->pre != FT_NORM_NONE, post = n->post != FT_NORM_NONE;
    const bool need_s = g->dscale || g->dshift || g->dw || g->dbias, need_t = g->dgate || g->dw_post;
    if ((need_s && !pre) || (g->dscale && !n->scale) || (g->dgate && !n->gate) || (g->dw && !n->w) ||
        (g->dw_post && !n->w_post))
        return FT_ERR_INVALID_ARG;
    const bool use_y = post || need_t;
    if (rows) {
        if ((!pre && dh) || (g->amax_dy && !g->dy)) return FT_ERR_INVALID_ARG;
        if (!dh && !dr) return FT_ERR_INVALID_ARG;
        if (pre && (!dh || !r)) return FT_ERR_INVALID_ARG;
        if (use_y && !y) return FT_ERR_INVALID_ARG;
        if ((pre || post) && !stats) return FT_ERR_INVALID_ARG;
    }
    const int xs = n->xt == FT_F32 ? 4 : 2;
    if ((dh && lddh < n->D) || (dr && lddr < n->D) || (r && ldr < n->D) || (y && ldy < n->D) ||
        (g->dx && g->lddx < n->D) || (g->dy && g->lddy < n->D))
        return FT_ERR_SHAPE;
    if ((dh && !rows_al16(dh, lddh, 2)) || (dr && !rows_al16(dr, lddr, xs)) || (r && !rows_al16(r, ldr, xs)) ||
        (y && !rows_al16(y, ldy, 2)) || (g->dx && !rows_al16(g->dx, g->lddx, xs)) ||
        (g->dy && !rows_al16(g->dy, g->lddy, 2)) || !al16(stats) || !al4(g->amax_dy) || !al4(g->dgate) ||
        !al4(g->dscale) || !al4(g->dshift) || !al4(g->dw_post) || !al4(g->dw) || !al4(g->dbias))
        return FT_ERR_ALIGN;
    const bool acc = need_s || need_t;
    if (acc) {
        if (!ws || ws_bytes < ft_gated_norm_workspace_bytes(n->M, n->D, n->B)) return FT_ERR_WORKSPACE;
        if (!al16(ws)) return FT_ERR_ALIGN;
    }
    if ((!rows || (!g->dx && !g->dy)) && !acc) return FT_OK;
    DevInfo* d;
    FT_TRY(device_info(&d));
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    const RowShape s = row_shape(n->D, true);
    int64_t chunk = 1;
    if (rows) {
        ft::norm::BwdParams p = {};
        p.M = (int)n->M;
        p.D = (int)n->D;
        p.B = (int)n->B;
        p.S = (int)(n->M / n->B);
        p.offsets = n->offsets;
        p.alpha = n->alpha;
        p.inv_d = 1.0f / (float)n->D;
        p.p32 = n->pt == FT_F32;
        p.ld_gate = n->B > 1 ? n->ld_gate : 0;
        p.ld_scale = n->B > 1 ? n->ld_scale : 0;
        p.gate = n->gate;
        p.scale = n->scale;
        p.w_post = n->w_post;
        p.w = n->w;
        p.dh = static_cast<const __nv_bfloat16*>(dh);
        p.lddh = lddh;
        p.dr = dr;
        p.lddr = lddr;
        p.r = pre ? r : nullptr;
        p.ldr = ldr;
        p.y = use_y && (g->dy || need_t) ? static_cast<const __nv_bfloat16*>(y) : nullptr;
        p.ldy = ldy;
        p.stats = pre || post ? reinterpret_cast<const float4*>(stats) : nullptr;
        p.dx = g->dx;
        p.lddx = g->lddx;
        p.dy = static_cast<__nv_bfloat16*>(g->dy);
        p.lddy = g->lddy;
        p.amax = g->amax_dy;
        p.partial = ws_sums(ws);
        p.need_s = need_s;
        p.need_t = need_t;
        p.has = norm_has(n) | (dh ? ft::norm::kDh : 0u) | (dr ? ft::norm::kDr : 0u) | (p.r ? ft::norm::kR : 0u) |
                (p.y ? ft::norm::kY : 0u) | (g->dx ? ft::norm::kDx : 0u) | (g->dy ? ft::norm::kDy : 0u) |
                (p.stats ? ft::norm::kStats : 0u);
        chunk = norm_bwd_chunk(n->M, n->D, norm_bwd_mod(p));
        p.chunk = (int)chunk;
        p.tpr = s.tpr;
        const int chunks = (int)((n->M + chunk - 1) / chunk);
        LaunchTimer lt(KID_NORM_BWD, st);
        const ft_status e = launch_norm(p, n->xt, s, chunks, d, st);
        lt.stop();
        FT_TRY(e);
    }
    if (!acc) return FT_OK;
    ft::norm::ReduceParams q = {};
    q.M = (int)n->M;
    q.D = (int)n->D;
    q.B = (int)n->B;
    q.S = (int)(n->M / n->B);
    q.chunk = (int)chunk;
    q.offsets = n->offsets;
    q.alpha = n->alpha;
    q.p32 = n->pt == FT_F32;
    q.ld_gate = n->B > 1 ? n->ld_gate : 0;
    q.ld_scale = n->B > 1 ? n->ld_scale : 0;
    q.gate = n->gate;
    q.scale = n->scale;
    q.w_post = n->w_post;
    q.w = n->w;
    q.bias = n->bias;
    q.partial = ws_sums(ws);
    q.dgate = g->dgate;
    q.dscale = g->dscale;
    q.dshift = g->dshift;
    q.dw_post = g->dw_post;
    q.dw = g->dw;
    q.dbias = g->dbias;
    q.need_s = need_s;
    q.need_t = need_t;
    if (g->dw_post || g->dw || g->dbias) q.sums = ws_sums(ws) + norm_bwd_partials(n->M, n->D, n->B);
    LaunchTimer lt(KID_NORM_REDUCE, st);
    // partial rows of a sample of average length
    const bool few = n->M / chunk / n->B < 8;
    const dim3 grid(cdiv(n->D, 32), (unsigned)std::min<int64_t>(n->B, 32768));
    ft_status e = few ? launch_overlapped(ft::norm::k_gated_norm_reduce<4>, grid, 128, 0, st, q)
                      : launch_overlapped(ft::norm::k_gated_norm_reduce<32>, grid, 1024, 0, st, q);
    lt.stop();
    if (e != FT_OK || !q.sums) return e;
    LaunchTimer lt2(KID_NORM_WEIGHTS, st);
    e = launch_overlapped(ft::norm::k_gated_norm_weights, cdiv(n->D, 32), 32, 0, st, q);
    lt2.stop();
    return e;
}

ft_status ft_gelu_bwd_bf16(const void* y, const void* dh, void* dy, int64_t n, float* amax_dy, void* stream) {
    if (n < 0 || (n > 0 && (!y || !dh || !dy))) return FT_ERR_INVALID_ARG;
    if (n % 8) return FT_ERR_SHAPE;
    if (!al16(y) || !al16(dh) || !al16(dy) || !al4(amax_dy)) return FT_ERR_ALIGN;
    if (n == 0) return FT_OK;
    DevInfo* d;
    FT_TRY(device_info(&d));
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    // a table pays once a block looks up more slopes than its 4096 entries
    const bool table = n >= (int64_t)d->sms * ft::gelub::kTab;
    const int threads = table ? ft::gelub::kThreads : 128;
    const int grid = (int)std::min<int64_t>((n / 8 + threads - 1) / threads, (int64_t)d->sms * (table ? 1 : 16));
    LaunchTimer lt(KID_GELU_BWD, st);
    const ft_status e = launch_overlapped_args(
        table ? ft::gelub::k_gelu_bwd_bf16<true> : ft::gelub::k_gelu_bwd_bf16<false>, grid, threads, 0, st,
        static_cast<const __nv_bfloat16*>(y), static_cast<const __nv_bfloat16*>(dh), static_cast<__nv_bfloat16*>(dy), n,
        amax_dy);
    lt.stop();
    return e;
}

ft_status ft_qk_rope_fwd(const ft_rope* R, const void* qkv, int64_t ld, const ft_heads* q, const ft_heads* k,
                         const ft_heads* v, void* stream) {
    FT_TRY(check_rope(R));
    FT_TRY(check_heads(q, R->Hq, R->M > 0));
    FT_TRY(check_heads(k, R->Hk, R->M > 0));
    FT_TRY(check_heads(v, R->Hk, false));
    if (R->M > 0 && !qkv) return FT_ERR_INVALID_ARG;
    if (ld < ((int64_t)R->Hq + 2 * (int64_t)R->Hk) * R->hd) return FT_ERR_SHAPE;
    if (!rows_al16(qkv, ld, 2)) return FT_ERR_ALIGN;
    ft::rope::Params p = rope_params(R, q, k, v);
    if (R->M == 0 || p.Hq + p.Hk + p.Hv == 0) return FT_OK;
    DevInfo* d;
    FT_TRY(device_info(&d));
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    p.x = static_cast<const __nv_bfloat16*>(qkv);
    p.ld = ld;
    LaunchTimer lt(KID_ROPE_FWD, st);
    const int grid = rope_grid<false>(&p);
    const ft_status e = launch_rope<false>(p, grid, d, st);
    lt.stop();
    return e;
}

size_t ft_qk_rope_workspace_bytes(int64_t M, int64_t hd) {
    if (M < 0 || hd < 0) return 0;
    return kWsSums + (size_t)kRopeMaxBlocks * 2 * (size_t)hd * sizeof(float);
}

ft_status ft_qk_rope_bwd(const ft_rope* R, const ft_heads* dq, const ft_heads* dk, const ft_heads* dv,
                         const void* qkv, int64_t ld, void* dqkv, int64_t lddqkv, float* dw_q, float* dw_k,
                         float* amax, void* ws, size_t ws_bytes, void* stream) {
    FT_TRY(check_rope(R));
    FT_TRY(check_heads(dq, R->Hq, R->M > 0));
    FT_TRY(check_heads(dk, R->Hk, R->M > 0));
    FT_TRY(check_heads(dv, R->Hk, false));
    const bool norm = R->norm != FT_NORM_NONE, dw = dw_q || dw_k;
    if ((dw && !norm) || (R->M > 0 && (!dqkv || (norm && !qkv)))) return FT_ERR_INVALID_ARG;
    const int64_t width = ((int64_t)R->Hq + 2 * (int64_t)R->Hk) * R->hd;
    if ((qkv && ld < width) || lddqkv < width) return FT_ERR_SHAPE;
    if ((qkv && !rows_al16(qkv, ld, 2)) || !rows_al16(dqkv, lddqkv, 2) || !al4(dw_q) || !al4(dw_k) || !al4(amax))
        return FT_ERR_ALIGN;
    if (dw && (!ws || ws_bytes < ft_qk_rope_workspace_bytes(R->M, R->hd))) return FT_ERR_WORKSPACE;
    if (dw && !al4(ws)) return FT_ERR_ALIGN;
    ft::rope::Params p = rope_params(R, dq, dk, dv);
    const bool work = R->M > 0 && p.Hq + p.Hk + p.Hv > 0;
    if (!work && !dw) return FT_OK;
    DevInfo* d;
    FT_TRY(device_info(&d));
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    int blocks = 0;
    if (work) {
        p.x = static_cast<const __nv_bfloat16*>(qkv);
        p.ld = ld;
        p.dx = static_cast<__nv_bfloat16*>(dqkv);
        p.lddx = lddqkv;
        p.amax = amax;
        p.partial = dw ? ws_sums(ws) : nullptr;
        blocks = rope_grid<true>(&p);
        LaunchTimer lt(KID_ROPE_BWD, st);
        const ft_status e = launch_rope<true>(p, blocks, d, st);
        lt.stop();
        FT_TRY(e);
    }
    if (!dw) return FT_OK;
    LaunchTimer lt(KID_ROPE_REDUCE, st);
    const ft_status e = launch_overlapped_args(ft::rope::k_qk_rope_reduce, 2 * R->hd / 8, 1024, 0, st,
                                               static_cast<const float*>(ws_sums(ws)), blocks, (int)R->hd, dw_q, dw_k);
    lt.stop();
    return e;
}

ft_status ft_adamw_step(const ft_adamw_tensor* t, int64_t count, const ft_adamw_hyper* h, int state_bits,
                        int64_t* step, const float* lr_dev, const float* grad_scale, void* stream) {
    if (count < 0 || (count > 0 && !t) || !h || !step) return FT_ERR_INVALID_ARG;
    if (state_bits != 32 && state_bits != 8) return FT_ERR_INVALID_ARG;
    if (!(h->beta1 >= 0.0 && h->beta1 < 1.0) || !(h->beta2 >= 0.0 && h->beta2 < 1.0) || !(h->eps >= 0.0) ||
        !(h->lr == h->lr))
        return FT_ERR_INVALID_ARG;
    const bool k8 = state_bits == 8;
    if (!al8(step) || !al4(lr_dev) || !al4(grad_scale)) return FT_ERR_ALIGN;
    for (int64_t i = 0; i < count; ++i) {
        const ft_adamw_tensor& a = t[i];
        if (a.n < 0 || !dtype_ok(a.gt)) return FT_ERR_INVALID_ARG;
        if (a.n == 0) continue;
        if ((!a.p && !a.p16) || !a.grad || !a.m || !a.v || (k8 && (!a.m_scale || !a.v_scale)))
            return FT_ERR_INVALID_ARG;
        if (a.n > (int64_t(1) << 36)) return FT_ERR_SHAPE;
        const uintptr_t p16 = reinterpret_cast<uintptr_t>(a.p16), g = reinterpret_cast<uintptr_t>(a.grad);
        if (!al4(a.p) || (p16 & 1u) || (g & (a.gt == FT_F32 ? 3u : 1u)) || (!k8 && (!al4(a.m) || !al4(a.v))) ||
            !al4(a.m_scale) || !al4(a.v_scale))
            return FT_ERR_ALIGN;
    }
    DevInfo* d;
    FT_TRY(device_info(&d));
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (count <= kAdamFew)
        return adamw_group<kAdamFew>(t, 0, count, h, k8, true, step, lr_dev, grad_scale, d, st);
    for (int64_t i = 0; i < count; i += kAdamMany) {
        const int64_t end = std::min<int64_t>(count, i + kAdamMany);
        FT_TRY(adamw_group<kAdamMany>(t, i, end, h, k8, end == count, step, lr_dev, grad_scale, d, st));
    }
    return FT_OK;
}

ft_status ft_adamw_decode(const void* codes, const float* scales, int64_t n, int second, float* out, void* stream) {
    if (n < 0 || (n > 0 && (!codes || !scales || !out)) || (second != 0 && second != 1)) return FT_ERR_INVALID_ARG;
    if (!al4(scales) || !al4(out)) return FT_ERR_ALIGN;
    if (n == 0) return FT_OK;
    DevInfo* d;
    FT_TRY(device_info(&d));
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    const int vec = al4(codes) && al16(out);
    const int64_t blocks = (n + ft::adamw::kBlock - 1) / ft::adamw::kBlock;
    const int grid = (int)std::min<int64_t>((blocks + 7) / 8, (int64_t)d->sms * 6);
    LaunchTimer lt(KID_ADAMW_DECODE, st);
    const ft_status e = launch_overlapped_args(ft::adamw::k_adamw_decode, grid, 256, 0, st,
                                               static_cast<const uint8_t*>(codes), scales, (long long)n, second, out,
                                               vec);
    lt.stop();
    return e;
}

}  // extern "C"
