// ft_torch.cpp -- the torch side of the operators around the linears: checks
// of tensors, allocation of the outputs that a call was not given, and the
// calls of the C ABI (include/ft.h); for the optimizer, the look at its
// tensors before a step.  Marshalling only, in C++ because a small
// call's host time is what its user waits for: the same checks took 15 to 45
// us per call in Python, more than the kernels.  The Python functions
// (blockops.py) document the arguments, and put the tensors' device and stream
// in place first.
#include <c10/cuda/CUDAGraphsC10Utils.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/extension.h>

#include "../../include/ft.h"

namespace {

namespace py = pybind11;
using at::Tensor;
using Opt = std::optional<Tensor>;

[[noreturn]] void type_error(const std::string& what) { throw py::type_error(what); }
[[noreturn]] void value_error(const std::string& what) { throw py::value_error(what); }

std::string str(at::IntArrayRef sizes) {
    std::string s = "[";
    for (size_t i = 0; i < sizes.size(); ++i) s += (i ? ", " : "") + std::to_string(sizes[i]);
    return s + "]";
}
std::string str(at::ScalarType t) { return std::string("torch.") + at::toString(t); }

void* ptr(const Opt& t) { return t ? t->data_ptr() : nullptr; }

// Raises the package's error for a status of the C ABI.
void check(const char* name, ft_status s) {
    if (s != FT_OK) py::module_::import("bit_quantized_lora_b200._lib").attr("check")(name, (int)s);
}

void* stream_of(const Tensor& t) { return c10::cuda::getCurrentCUDAStream(t.get_device()).stream(); }

void same_device(const Tensor& t, const char* name, int64_t dev) {
    if (!t.is_cuda() || t.get_device() != dev)
        value_error(std::string(name) + " is on " + t.device().str() + ", the call is on cuda:" + std::to_string(dev));
}

// A row-major matrix: its leading dimension.
int64_t matrix(const Tensor& t, const char* name, at::ScalarType dtype, int64_t rows, int64_t cols, int64_t dev) {
    if (t.scalar_type() != dtype) type_error(std::string(name) + " must be " + str(dtype) + ", not " + str(t.scalar_type()));
    same_device(t, name, dev);
    if (t.dim() != 2 || t.size(0) != rows || t.size(1) != cols)
        value_error(std::string(name) + " must be [" + std::to_string(rows) + ", " + std::to_string(cols) + "], not " +
                    str(t.sizes()));
    if (cols > 1 && t.stride(1) != 1) value_error(std::string(name) + " must have unit column stride");
    return rows > 1 ? t.stride(0) : cols;
}
int64_t matrix(const Opt& t, const char* name, at::ScalarType dtype, int64_t rows, int64_t cols, int64_t dev) {
    return t ? matrix(*t, name, dtype, rows, cols, dev) : 0;
}

float* floats(const Opt& t, const char* name, int64_t n, int64_t dev) {
    if (!t) return nullptr;
    if (t->scalar_type() != at::kFloat || t->numel() < n || !t->is_contiguous())
        type_error(std::string(name) + " must be a contiguous float32 tensor of " + std::to_string(n));
    same_device(*t, name, dev);
    return static_cast<float*>(t->data_ptr());
}

int dtype_of(at::ScalarType t, const char* what) {
    if (t == at::kBFloat16) return FT_BF16;
    if (t == at::kFloat) return FT_F32;
    type_error(std::string(what) + " must be bfloat16 or float32, not " + str(t));
}

// Scratch of one call: the caller's workspace, or memory of the current
// stream.  A captured call always takes the latter, which its graph owns: a
// workspace gives its memory back when a later call needs more, and the graph
// would go on writing there.
Tensor scratch(const py::object& ws, size_t bytes, const Tensor& like) {
    if (!ws.is_none() && c10::cuda::currentStreamCaptureStatusMayInitCtx() == c10::cuda::CaptureStatus::None)
        return ws.attr("get")(bytes, py::cast(like).attr("device")).cast<Tensor>();
    return at::empty({(int64_t)bytes}, like.options().dtype(at::kByte));
}

// ---------------------------------------------------------------- gated norm
struct Norm {
    ft_gated_norm n = {};
    Opt gate, scale, shift, weight, bias, w_post;
    std::optional<at::ScalarType> pt;

    void param(const Tensor& t, int64_t dev) {
        same_device(t, "a parameter vector", dev);
        const auto dt = t.scalar_type();
        if ((dt != at::kBFloat16 && dt != at::kFloat) || (pt && *pt != dt))
            type_error("gate, scale, shift and the norms' weights must all be bfloat16 or all float32");
        pt = dt;
    }
    const void* mod(const Opt& t, const char* name, int64_t* ld, int64_t dev) {
        *ld = 0;
        if (!t) return nullptr;
        const bool rows = t->dim() == 2;
        if ((t->dim() != 1 && !rows) || t->size(-1) != n.D || (rows && t->size(0) != n.B && t->size(0) != 1))
            value_error(std::string(name) + " must be [" + std::to_string(n.B) + ", " + std::to_string(n.D) + "] or [" +
                        std::to_string(n.D) + "], not " + str(t->sizes()));
        if (t->stride(-1) != 1) value_error(std::string(name) + " must have unit column stride");
        if (rows && t->size(0) > 1) *ld = t->stride(0);
        param(*t, dev);
        return t->data_ptr();
    }
    const void* vec(const Opt& t, const char* name, int64_t dev) {
        if (!t) return nullptr;
        if (t->dim() != 1 || t->size(0) != n.D || !t->is_contiguous())
            value_error(std::string(name) + " must be contiguous [" + std::to_string(n.D) + "], not " + str(t->sizes()));
        param(*t, dev);
        return t->data_ptr();
    }

    Norm(const py::object& norm, int64_t M, int64_t D, at::ScalarType xt, const Opt& g, const Opt& sc, const Opt& sh,
         const Opt& offsets, int64_t dev)
        : gate(g), scale(sc), shift(sh) {
        weight = norm.attr("weight").cast<Opt>();
        bias = norm.attr("bias").cast<Opt>();
        w_post = norm.attr("w_post").cast<Opt>();
        n.M = M;
        n.D = D;
        n.B = 1;
        n.xt = dtype_of(xt, "the residual stream");
        n.pre = norm.attr("pre").cast<int>();
        n.post = norm.attr("post").cast<int>();
        n.alpha = norm.attr("alpha").cast<float>();
        n.eps_pre = norm.attr("eps").cast<float>();
        const py::object eps_post = norm.attr("eps_post");
        n.eps_post = eps_post.is_none() ? n.eps_pre : eps_post.cast<float>();
        if (offsets) {
            if (offsets->scalar_type() != at::kInt || offsets->dim() != 1 || offsets->size(0) < 2 ||
                !offsets->is_contiguous())
                type_error("offsets must be a contiguous int32 tensor [samples + 1]");
            same_device(*offsets, "offsets", dev);
            n.B = offsets->size(0) - 1;
            n.offsets = static_cast<const int32_t*>(offsets->data_ptr());
        } else {
            for (const Opt* t : {&gate, &scale, &shift})
                if (*t && (*t)->dim() == 2 && (*t)->size(0) != 1) {
                    n.B = (*t)->size(0);
                    break;
                }
        }
        n.gate = mod(gate, "gate", &n.ld_gate, dev);
        n.scale = mod(scale, "scale", &n.ld_scale, dev);
        n.shift = mod(shift, "shift", &n.ld_shift, dev);
        n.w = vec(weight, "weight", dev);
        n.bias = vec(bias, "bias", dev);
        n.w_post = vec(w_post, "w_post", dev);
        n.pt = pt == at::kBFloat16 ? FT_BF16 : FT_F32;
    }
};

py::tuple gated_norm_fwd(const py::object& norm, const Tensor& x, const Opt& y, const Opt& gate, const Opt& scale,
                         const Opt& shift, const Opt& offsets, Opt r, Opt h, const py::object& want_stats,
                         const Opt& amax_h) {
    if (x.dim() != 2) value_error("x must be [rows, channels]");
    const int64_t M = x.size(0), D = x.size(1), dev = x.get_device();
    const auto xt = x.scalar_type();
    const Norm nv(norm, M, D, xt, gate, scale, shift, offsets, dev);
    const int64_t ldx = matrix(x, "x", xt, M, D, dev), ldy = matrix(y, "y", at::kBFloat16, M, D, dev);
    if (!y && r) value_error("r is written only with y");
    if (y && !r) r = at::empty({M, D}, x.options());
    const bool pre = nv.n.pre != FT_NORM_NONE;
    if (!pre && h) value_error("h is written only with a pre norm");
    if (pre && !h) h = at::empty({M, D}, x.options().dtype(at::kBFloat16));
    const int64_t ldr = matrix(r, "r", xt, M, D, dev), ldh = matrix(h, "h", at::kBFloat16, M, D, dev);
    Opt stats;
    if (py::isinstance<py::bool_>(want_stats)) {
        if (want_stats.cast<bool>()) stats = at::empty({M, 4}, x.options().dtype(at::kFloat));
    } else {
        stats = want_stats.cast<Opt>();
    }
    check("ft_gated_norm_fwd",
          ft_gated_norm_fwd(&nv.n, x.data_ptr(), ldx, ptr(y), ldy, ptr(r), ldr, ptr(h), ldh,
                            floats(stats, "stats", 4 * M, dev), floats(amax_h, "amax_h", 1, dev), stream_of(x)));
    return py::make_tuple(y ? *r : x, h, stats);
}

// wanted: of gate, scale, shift, weight, bias, w_post, or None for all given.
// Returns dx, dy and the six gradients.
py::tuple gated_norm_bwd(const Tensor& some, const py::object& norm, const Opt& dh, const Opt& r, const Opt& stats,
                         const Opt& dr, const Opt& y, const Opt& gate, const Opt& scale, const Opt& shift,
                         const Opt& offsets, std::optional<bool> residual, bool need_dx, Opt dx, Opt dy,
                         const std::optional<std::array<bool, 6>>& names, const Opt& amax_dy, const py::object& ws) {
    if (some.dim() != 2) value_error("gradients must be [rows, channels]");
    const int64_t M = some.size(0), D = some.size(1), dev = some.get_device();
    const auto bf = at::kBFloat16;
    const auto xt = r ? r->scalar_type() : dr ? dr->scalar_type() : dx ? dx->scalar_type() : bf;
    const Norm nv(norm, M, D, xt, gate, scale, shift, offsets, dev);
    const int64_t B = nv.n.B;
    const Opt* given[6] = {&nv.gate, &nv.scale, &nv.shift, &nv.weight, &nv.bias, &nv.w_post};
    bool wanted[6];
    int mods = 0, weights = 0;
    for (int i = 0; i < 6; ++i) {
        wanted[i] = names ? (*names)[i] : given[i]->has_value();
        if (wanted[i] && !given[i]->has_value()) value_error("no gradient for a parameter that is not given");
        (i < 3 ? mods : weights) += wanted[i];
    }
    const bool post = nv.n.post != FT_NORM_NONE;
    if (!residual) residual = y || gate || dy || post;
    if (!y && (post || wanted[0] || wanted[5])) value_error("the post norm and the gradient of the gate need y");
    const int64_t lddh = matrix(dh, "dh", bf, M, D, dev), lddr = matrix(dr, "dr", xt, M, D, dev);
    const int64_t ldr = matrix(r, "r", xt, M, D, dev), ldy = matrix(y, "y", bf, M, D, dev);
    if (!need_dx)
        dx.reset();
    else if (!dx)
        dx = at::empty({M, D}, some.options().dtype(xt));
    if (*residual && !dy) dy = at::empty({M, D}, some.options().dtype(bf));
    ft_gated_norm_grads g = {};
    g.dx = ptr(dx);
    g.lddx = matrix(dx, "dx", xt, M, D, dev);
    g.dy = ptr(dy);
    g.lddy = matrix(dy, "dy", bf, M, D, dev);
    g.amax_dy = floats(amax_dy, "amax_dy", 1, dev);
    // the gradients of modulation vectors share one allocation, those of weights another
    Opt out[6];
    float** to[6] = {&g.dgate, &g.dscale, &g.dshift, &g.dw, &g.dbias, &g.dw_post};
    const auto f32 = some.options().dtype(at::kFloat);
    Tensor all = mods ? at::empty({mods, B, D}, f32) : Tensor(), flat = weights ? at::empty({weights, D}, f32) : Tensor();
    int64_t a = 0, b = 0;
    for (int i = 0; i < 6; ++i) {
        if (!wanted[i]) continue;
        out[i] = i < 3 ? all.select(0, a++) : flat.select(0, b++);
        *to[i] = static_cast<float*>(out[i]->data_ptr());
    }
    Tensor buf;
    size_t bytes = 0;
    if (mods || weights) {
        bytes = ft_gated_norm_workspace_bytes(M, D, B);
        buf = scratch(ws, bytes, some);
    }
    check("ft_gated_norm_bwd",
          ft_gated_norm_bwd(&nv.n, ptr(dh), lddh, ptr(dr), lddr, ptr(r), ldr, ptr(y), ldy,
                            floats(stats, "stats", 4 * M, dev), &g, buf.defined() ? buf.data_ptr() : nullptr, bytes,
                            stream_of(some)));
    for (int i = 0; i < 3; ++i)  // one for all samples
        if (wanted[i] && ((*given[i])->dim() == 1 || (*given[i])->size(0) != B))
            out[i] = (B > 1 ? out[i]->sum(0) : *out[i]).view((*given[i])->sizes());
    return py::make_tuple(dx, dy, out[0], out[1], out[2], out[3], out[4], out[5]);
}

// ---------------------------------------------------------------- GELU backward
Tensor gelu_bwd(const Tensor& y, const Tensor& dh, const Opt& given, const Opt& amax_dy) {
    const int64_t dev = y.get_device();
    const Tensor out = given ? *given : at::empty_like(y);
    const std::pair<const char*, const Tensor*> all[] = {{"y", &y}, {"dh", &dh}, {"out", &out}};
    for (const auto& [name, t] : all) {
        if (t->scalar_type() != at::kBFloat16) type_error(std::string(name) + " must be a CUDA bfloat16 tensor");
        same_device(*t, name, dev);
        if (!t->is_contiguous() || t->sizes() != y.sizes())
            value_error(std::string(name) + " must be contiguous and of y's shape");
    }
    check("ft_gelu_bwd_bf16", ft_gelu_bwd_bf16(y.data_ptr(), dh.data_ptr(), out.data_ptr(), y.numel(),
                                               floats(amax_dy, "amax_dy", 1, dev), stream_of(y)));
    return out;
}

// ---------------------------------------------------------------- rotary positions
struct RopeView {
    ft_rope R = {};
    Tensor freqs;
    Opt w_q, w_k;
    int64_t width = 0;

    RopeView(const py::object& rope, const Tensor& pos, int64_t dev) : freqs(rope.attr("freqs").cast<Tensor>()) {
        R.Hq = rope.attr("heads").cast<int>();
        R.Hk = rope.attr("kv_heads").cast<int>();
        R.hd = rope.attr("head_dim").cast<int>();
        width = ((int64_t)R.Hq + 2 * (int64_t)R.Hk) * R.hd;
        const py::tuple axes(rope.attr("axes"));
        if (axes.size() < 1 || axes.size() > 4) value_error("rotary positions have one to four axes");
        R.n_axes = (int)axes.size();
        int64_t rot = 0;
        for (int a = 0; a < R.n_axes; ++a) rot += R.axis_dims[a] = axes[a].cast<int>();
        R.layout = rope.attr("layout").cast<int>();
        R.norm = rope.attr("norm").cast<bool>() ? FT_NORM_RMS : FT_NORM_NONE;
        R.eps = rope.attr("eps").cast<float>();
        if (pos.scalar_type() != at::kInt && pos.scalar_type() != at::kFloat)
            type_error("pos must be int32 or float32, not " + str(pos.scalar_type()));
        R.pos_t = pos.scalar_type() == at::kInt ? FT_POS_I32 : FT_POS_F32;
        if (freqs.scalar_type() != at::kDouble || freqs.numel() != rot / 2 || !freqs.is_contiguous())
            type_error("freqs must be a contiguous float64 tensor of " + std::to_string(rot / 2));
        same_device(pos, "pos", dev);
        same_device(freqs, "freqs", dev);
        w_q = rope.attr("w_q").cast<Opt>();
        w_k = rope.attr("w_k").cast<Opt>();
        R.pt = FT_F32;
        std::optional<at::ScalarType> pt;
        for (const Opt* w : {&w_q, &w_k}) {
            if (!*w) continue;
            const auto dt = (*w)->scalar_type();
            if ((dt != at::kBFloat16 && dt != at::kFloat) || (pt && *pt != dt))
                type_error("w_q and w_k must both be bfloat16 or both float32");
            if ((*w)->dim() != 1 || (*w)->size(0) != R.hd || !(*w)->is_contiguous())
                value_error("w_q and w_k must be contiguous [" + std::to_string(R.hd) + "]");
            same_device(**w, "a head's weight", dev);
            pt = dt;
            R.pt = dt == at::kBFloat16 ? FT_BF16 : FT_F32;
        }
        R.pos = pos.data_ptr();
        R.freqs = static_cast<const double*>(freqs.data_ptr());
        R.w_q = ptr(w_q);
        R.w_k = ptr(w_k);
    }
    void rows(const Tensor& pos, int64_t M, int64_t S) {
        R.M = M;
        R.S = S;
        const bool flat = R.n_axes == 1 && pos.dim() == 1 && pos.size(0) == M;
        if ((!flat && (pos.dim() != 2 || pos.size(0) != M || pos.size(1) != R.n_axes)) || !pos.is_contiguous())
            value_error("pos must be contiguous [" + std::to_string(M) + ", " + std::to_string(R.n_axes) + "], not " +
                        str(pos.sizes()));
    }
};

ft_heads heads_of(const Opt& t, const char* name, int64_t B, int64_t H, int64_t S, int64_t hd, int64_t dev, bool out) {
    ft_heads h = {};
    if (!t) return h;
    if (t->scalar_type() != at::kBFloat16) type_error(std::string(name) + " must be a CUDA bfloat16 tensor");
    same_device(*t, name, dev);
    if (t->dim() != 4 || t->size(0) != B || t->size(1) != H || t->size(2) != S || t->size(3) != hd)
        value_error(std::string(name) + " must be " + str(std::vector<int64_t>{B, H, S, hd}) + ", not " +
                    str(t->sizes()));
    if (t->stride(3) != 1) value_error(std::string(name) + " must have unit stride along a head");
    // the stride of an axis of one element says nothing
    h.p = t->data_ptr();
    h.sb = B > 1 ? t->stride(0) : 0;
    h.sh = H > 1 ? t->stride(1) : 0;
    h.st = S > 1 ? t->stride(2) : 0;
    if (out && ((B > 1 && !h.sb) || (H > 1 && !h.sh) || (S > 1 && !h.st)))
        value_error(std::string(name) + " is written: its elements must be apart");
    return h;
}

py::tuple qk_rope_fwd(const py::object& rope, const Tensor& qkv, const Tensor& pos, std::optional<int64_t> tokens,
                      bool head_major, Opt q, Opt k, Opt v, bool copy_v) {
    if (qkv.dim() != 2) value_error("qkv must be [rows, width]");
    const int64_t M = qkv.size(0), dev = qkv.get_device(), S = tokens ? *tokens : M;
    if (S < 0 || (M > 0 && (S < 1 || M % S)))
        value_error(std::to_string(M) + " rows are no samples of " + std::to_string(S) + " tokens");
    const int64_t B = S ? M / S : 0;
    RopeView rv(rope, pos, dev);
    const int64_t Hq = rv.R.Hq, Hk = rv.R.Hk, hd = rv.R.hd;
    const int64_t ld = matrix(qkv, "qkv", at::kBFloat16, M, rv.width, dev);
    rv.rows(pos, M, S);
    auto make = [&](int64_t H) {
        return head_major ? at::empty({B, H, S, hd}, qkv.options()) : at::empty({B, S, H, hd}, qkv.options()).transpose(1, 2);
    };
    if (!q) q = make(Hq);
    if (!k) k = make(Hk);
    if (!v && copy_v) v = make(Hk);
    const ft_heads hq = heads_of(q, "q", B, Hq, S, hd, dev, true), hk = heads_of(k, "k", B, Hk, S, hd, dev, true),
                   hv = heads_of(v, "v", B, Hk, S, hd, dev, true);
    check("ft_qk_rope_fwd", ft_qk_rope_fwd(&rv.R, qkv.data_ptr(), ld, &hq, &hk, &hv, stream_of(qkv)));
    if (!v) v = qkv.narrow(1, (Hq + Hk) * hd, Hk * hd).unflatten(1, {Hk, hd}).unflatten(0, {B, S}).transpose(1, 2);
    return py::make_tuple(q, k, v);
}

py::tuple qk_rope_bwd(const py::object& rope, const Tensor& dq, const Tensor& dk, const Opt& dv, const Tensor& pos,
                      const Opt& qkv, Opt dqkv, bool weight_grads, const Opt& amax, const py::object& ws) {
    if (dq.dim() != 4) value_error("dq must be [samples, heads, tokens, head_dim]");
    const int64_t B = dq.size(0), S = dq.size(2), M = B * S, dev = dq.get_device();
    RopeView rv(rope, pos, dev);
    const int64_t Hq = rv.R.Hq, Hk = rv.R.Hk, hd = rv.R.hd;
    const bool norm = rv.R.norm != FT_NORM_NONE;
    if (norm && !qkv) value_error("the gradient through the norm needs qkv");
    rv.rows(pos, M, S);
    const auto bf = dq.options().dtype(at::kBFloat16);
    if (!dqkv) dqkv = dv ? at::empty({M, rv.width}, bf) : at::zeros({M, rv.width}, bf);
    const int64_t ld = matrix(qkv, "qkv", at::kBFloat16, M, rv.width, dev),
                  ldd = matrix(*dqkv, "dqkv", at::kBFloat16, M, rv.width, dev);
    const ft_heads hq = heads_of(dq, "dq", B, Hq, S, hd, dev, false), hk = heads_of(dk, "dk", B, Hk, S, hd, dev, false),
                   hv = heads_of(dv, "dv", B, Hk, S, hd, dev, false);
    Opt dw_q, dw_k;
    Tensor buf;
    size_t bytes = 0;
    if (weight_grads && norm && (rv.w_q || rv.w_k)) {
        const auto f32 = dq.options().dtype(at::kFloat);
        if (rv.w_q) dw_q = at::empty({hd}, f32);
        if (rv.w_k) dw_k = at::empty({hd}, f32);
        bytes = ft_qk_rope_workspace_bytes(M, hd);
        buf = scratch(ws, bytes, dq);
    }
    check("ft_qk_rope_bwd",
          ft_qk_rope_bwd(&rv.R, &hq, &hk, &hv, ptr(qkv), ld, dqkv->data_ptr(), ldd, static_cast<float*>(ptr(dw_q)),
                         static_cast<float*>(ptr(dw_k)), floats(amax, "amax", 1, dev),
                         buf.defined() ? buf.data_ptr() : nullptr, bytes, stream_of(dq)));
    return py::make_tuple(dqkv, dw_q, dw_k);
}

// ---------------------------------------------------------------- optimizer
// What a step takes for granted of its tensors, as bytes to compare with those
// of the step before: where each lies, its type, sizes and strides.
py::bytes layout_of(const py::sequence& tensors) {
    std::string key;
    key.reserve(64 * py::len(tensors));
    auto put = [&](int64_t v) { key.append(reinterpret_cast<const char*>(&v), sizeof(v)); };
    for (const py::handle& h : tensors) {
        if (!THPVariable_Check(h.ptr())) type_error("parameters and gradients must be tensors");
        const Tensor& t = THPVariable_Unpack(h.ptr());
        put(reinterpret_cast<int64_t>(t.data_ptr()));
        put((int64_t)t.scalar_type() << 32 | t.dim());
        for (int64_t n : t.sizes()) put(n);
        for (int64_t n : t.strides()) put(n);
    }
    return py::bytes(key);
}

}  // namespace

PYBIND11_MODULE(_ft_torch, m) {
    m.def("gated_norm_fwd", &gated_norm_fwd);
    m.def("gated_norm_bwd", &gated_norm_bwd);
    m.def("gelu_bwd", &gelu_bwd);
    m.def("qk_rope_fwd", &qk_rope_fwd);
    m.def("qk_rope_bwd", &qk_rope_bwd);
    m.def("layout_of", &layout_of);
}
