"""Operators of a DiT block between its linears, over the C ABI: the gated
norm (residual with gate, norm with modulation), the rotary positions of
queries and keys, and GELU's backward.  Each hands the next linear the tensor
amax of what it writes (amax_h, amax_dy, amax), so that ft_linear_fwd and
ft_linear_bwd quantize in a single pass.

Calls run on `stream`, or on the current stream of their tensors' device;
what they allocate (outputs that are not given, scratch) belongs to that
stream.  They may be captured in a CUDA graph.
"""
from __future__ import annotations

import functools
import struct
from dataclasses import dataclass

import torch

from ._lib import check, load

NORM_NONE, NORM_RMS, NORM_LAYER = 0, 1, 2
ROPE_PAIRS, ROPE_HALVES = 0, 1
_BF16, _F32 = torch.bfloat16, torch.float32
_DTYPE = {_BF16: 0, _F32: 1}
# the C structs (ft_gated_norm, ft_gated_norm_grads, ft_rope, ft_heads) as bytes: a call fills its own
_NORM = struct.Struct("@3qP2i3f2i3q6P")
_NORM_GRADS = struct.Struct("@PqPq7P")
_ROPE = struct.Struct("@2q4i4i2if2i4P")
_HEADS = struct.Struct("@P3q")
_raw_stream = torch._C._cuda_getCurrentRawStream


def _on_device(at: int):
    """Runs a call with its tensors' device and the stream it was given (or
    that device's current one) current; argument `at` is such a tensor."""
    def wrap(fn):
        @functools.wraps(fn)
        def call(*args, stream=None, **kw):
            dev = args[at].get_device()
            if dev < 0:
                raise TypeError(f"{fn.__name__} needs CUDA tensors")
            if stream is None and dev == torch._C._cuda_getDevice():
                return fn(*args, **kw)
            stream = torch.cuda.current_stream(dev) if stream is None else stream
            if stream.device.index != dev:
                raise ValueError(f"the stream is on {stream.device}, the tensors are on cuda:{dev}")
            with torch.cuda.stream(stream):
                return fn(*args, **kw)
        return call
    return wrap


def _ptr(t) -> int:
    return 0 if t is None else t.data_ptr()


def _same_device(t: torch.Tensor, dev: int, name: str) -> None:
    if t.get_device() != dev:
        raise ValueError(f"{name} is on {t.device}, the call is on cuda:{dev}")


def _matrix(t: torch.Tensor, name: str, dtype, rows: int, cols: int, dev: int) -> int:
    """Checks a row-major matrix and returns its leading dimension."""
    if t.dtype is not dtype:
        raise TypeError(f"{name} must be {dtype}, not {t.dtype}")
    if t.get_device() != dev:
        _same_device(t, dev, name)
    if t.shape != (rows, cols):
        raise ValueError(f"{name} must be [{rows}, {cols}], not {list(t.shape)}")
    ld, unit = t.stride()
    if unit != 1 and cols > 1:
        raise ValueError(f"{name} must have unit column stride")
    return ld if rows > 1 else cols


def _f32(t, name: str, n: int, dev: int) -> int:
    if t is None:
        return 0
    if t.dtype is not _F32 or t.numel() < n or not t.is_contiguous():
        raise TypeError(f"{name} must be a contiguous float32 tensor of {n}")
    if t.get_device() != dev:
        _same_device(t, dev, name)
    return t.data_ptr()


def _scratch(ws, nbytes: int, like: torch.Tensor):
    """Scratch of one call: the caller's workspace, or memory of the current
    stream (an allocation that a captured graph owns with the call)."""
    return ws.get(nbytes, like.device) if ws is not None else like.new_empty(nbytes, dtype=torch.uint8)


# ---------------------------------------------------------------- gated norm
@dataclass
class GatedNorm:
    """The fixed part of a block's boundary: the norm of the block behind
    (pre) with its weight and bias [D], the norm of the block before (post)
    with its weight, the residual scale alpha.  Weights are bf16 or float32."""
    pre: int = NORM_LAYER
    post: int = NORM_NONE
    alpha: float = 1.0
    eps: float = 1e-6
    weight: torch.Tensor | None = None
    bias: torch.Tensor | None = None
    w_post: torch.Tensor | None = None
    eps_post: float | None = None  # eps where it is not given


@dataclass
class GatedNormGrads:
    """What ft_gated_norm_bwd returns; float32 gradients of parameters in
    their parameters' shapes, None where there is none."""
    dx: torch.Tensor | None
    dy: torch.Tensor | None
    dgate: torch.Tensor | None = None
    dscale: torch.Tensor | None = None
    dshift: torch.Tensor | None = None
    dweight: torch.Tensor | None = None
    dbias: torch.Tensor | None = None
    dw_post: torch.Tensor | None = None


def _norm_view(norm: GatedNorm, M: int, D: int, xt, gate, scale, shift, offsets, dev: int):
    """The C struct of a call, and its number of samples."""
    if xt not in _DTYPE:
        raise TypeError(f"the residual stream must be bfloat16 or float32, not {xt}")
    B, pt = 1, None
    mods = (("gate", gate), ("scale", scale), ("shift", shift))
    if offsets is not None:
        if offsets.dtype is not torch.int32 or offsets.dim() != 1 or len(offsets) < 2 or not offsets.is_contiguous():
            raise TypeError("offsets must be a contiguous int32 tensor [samples + 1]")
        _same_device(offsets, dev, "offsets")
        B = len(offsets) - 1
    else:
        for _, t in mods:
            if t is not None and t.dim() == 2 and len(t) != 1:
                B = len(t)
                break
    ld = []
    for name, t in mods:
        if t is None:
            ld.append(0)
            continue
        shape, stride = t.shape, t.stride()
        if shape != (B, D) and shape != (D,) and shape != (1, D):
            raise ValueError(f"{name} must be [{B}, {D}] or [{D}], not {list(shape)}")
        if stride[-1] != 1:
            raise ValueError(f"{name} must have unit column stride")
        ld.append(stride[0] if len(shape) == 2 and shape[0] > 1 else 0)
        pt = _param_type(t, pt, dev)
    for name, t in (("weight", norm.weight), ("bias", norm.bias), ("w_post", norm.w_post)):
        if t is not None:
            if t.shape != (D,) or not t.is_contiguous():
                raise ValueError(f"{name} must be contiguous [{D}], not {list(t.shape)}")
            pt = _param_type(t, pt, dev)
    eps = norm.eps
    return _NORM.pack(M, D, B, _ptr(offsets), norm.pre, norm.post, eps, eps if norm.eps_post is None else norm.eps_post,
                      norm.alpha, _DTYPE[xt], 0 if pt is _BF16 else 1, *ld, _ptr(gate), _ptr(scale), _ptr(shift),
                      _ptr(norm.w_post), _ptr(norm.weight), _ptr(norm.bias)), B


def _param_type(t: torch.Tensor, pt, dev: int):
    if t.get_device() != dev:
        _same_device(t, dev, "a parameter vector")
    if t.dtype not in _DTYPE or (pt is not None and t.dtype is not pt):
        raise TypeError("gate, scale, shift and the norms' weights must all be bfloat16 or all float32")
    return t.dtype


@_on_device(1)
def ft_gated_norm_fwd(norm: GatedNorm, x: torch.Tensor, y: torch.Tensor | None = None, gate=None, scale=None,
                      shift=None, *, offsets: torch.Tensor | None = None, r: torch.Tensor | None = None,
                      h: torch.Tensor | None = None, stats: torch.Tensor | bool = True,
                      amax_h: torch.Tensor | None = None):
    """r = x + alpha gate (y, or N_post(y) w_post) and h = (N_pre(r) weight +
    bias)(1 + scale) + shift on x [M, D] (bf16 or float32) and y (bf16).
    gate, scale, shift: [samples, D], or [D] / [1, D] for all samples; rows
    belong to samples evenly, or by offsets (int32 [samples + 1]; rows from
    offsets[-1] on are not written).  amax_h: an optional float32 device
    scalar (>= 0) raised to max|h|.  Returns (r, h, stats): r is x without y,
    h is None without a pre norm; stats float32 [M, 4] (None with
    stats=False) is for the backward."""
    if x.dim() != 2:
        raise ValueError("x must be [rows, channels]")
    M, D = x.shape
    dev, xt = x.get_device(), x.dtype
    n, _ = _norm_view(norm, M, D, xt, gate, scale, shift, offsets, dev)
    ldx = _matrix(x, "x", xt, M, D, dev)
    ldy = ldr = ldh = 0
    if y is not None:
        ldy = _matrix(y, "y", _BF16, M, D, dev)
        r = x.new_empty((M, D)) if r is None else r
        ldr = _matrix(r, "r", xt, M, D, dev)
    elif r is not None:
        raise ValueError("r is written only with y")
    if norm.pre != NORM_NONE:
        h = x.new_empty((M, D), dtype=_BF16) if h is None else h
        ldh = _matrix(h, "h", _BF16, M, D, dev)
    elif h is not None:
        raise ValueError("h is written only with a pre norm")
    if stats is True:
        stats = x.new_empty((M, 4), dtype=_F32)
    elif stats is False:
        stats = None
    check("ft_gated_norm_fwd", load().ft_gated_norm_fwd(
        n, x.data_ptr(), ldx, _ptr(y), ldy, _ptr(r), ldr, _ptr(h), ldh, _f32(stats, "stats", 4 * M, dev),
        _f32(amax_h, "amax_h", 1, dev), _raw_stream(dev)))
    return (x if y is None else r), h, stats


_PARAMS = ("gate", "scale", "shift", "weight", "bias", "w_post")


def ft_gated_norm_bwd(norm: GatedNorm, dh: torch.Tensor | None, r: torch.Tensor | None,
                      stats: torch.Tensor | None, *, dr: torch.Tensor | None = None,
                      y: torch.Tensor | None = None, gate=None, scale=None, shift=None,
                      offsets: torch.Tensor | None = None, residual: bool | None = None,
                      need_dx: bool = True, dx: torch.Tensor | None = None, dy: torch.Tensor | None = None,
                      param_grads=True, amax_dy: torch.Tensor | None = None, ws=None,
                      stream=None) -> GatedNormGrads:
    """Gradients of ft_gated_norm_fwd from dh (bf16, None without a pre norm)
    and dr, the gradient of r from the blocks above (None: zero).  r, stats:
    the forward's.  y: the forward's, needed with a post norm and for the
    gate's gradient.  residual: whether there is a y to give a gradient (by
    default when y, gate or dy is given or there is a post norm).
    param_grads: True for the gradient of every parameter given, or the names
    wanted out of 'gate', 'scale', 'shift', 'weight', 'bias', 'w_post'; a
    gate, scale or shift that all samples share gets the sum over them.
    amax_dy: an optional float32 device scalar (>= 0) raised to max|dy|."""
    some = dh if dh is not None else dr
    if some is None:
        raise ValueError("one of dh and dr must be given")
    return _gated_norm_bwd(some, norm, dh, r, stats, dr, y, gate, scale, shift, offsets, residual, need_dx, dx, dy,
                           param_grads, amax_dy, ws, stream=stream)


@_on_device(0)
def _gated_norm_bwd(some, norm, dh, r, stats, dr, y, gate, scale, shift, offsets, residual, need_dx, dx, dy,
                    param_grads, amax_dy, ws) -> GatedNormGrads:
    if some.dim() != 2:
        raise ValueError("gradients must be [rows, channels]")
    M, D = some.shape
    dev = some.get_device()
    xt = r.dtype if r is not None else dr.dtype if dr is not None else dx.dtype if dx is not None else _BF16
    n, B = _norm_view(norm, M, D, xt, gate, scale, shift, offsets, dev)
    weight, bias, w_post = norm.weight, norm.bias, norm.w_post
    given = (gate, scale, shift, weight, bias, w_post)
    if param_grads is True:
        wanted = [v is not None for v in given]
    else:
        names = set(param_grads or ())
        wanted = [k in names for k in _PARAMS]
        unknown = names.difference(k for k, v in zip(_PARAMS, given) if v is not None)
        if unknown:
            raise ValueError(f"no gradient for {sorted(unknown)}: not among the parameters given")
    if residual is None:
        residual = y is not None or gate is not None or dy is not None or norm.post != NORM_NONE
    if y is None and (norm.post != NORM_NONE or wanted[0] or wanted[5]):
        raise ValueError("the post norm and the gradient of the gate need y")
    lddh = 0 if dh is None else _matrix(dh, "dh", _BF16, M, D, dev)
    lddr = 0 if dr is None else _matrix(dr, "dr", xt, M, D, dev)
    ldr = 0 if r is None else _matrix(r, "r", xt, M, D, dev)
    ldy = 0 if y is None else _matrix(y, "y", _BF16, M, D, dev)
    if not need_dx:
        dx = None
    elif dx is None:
        dx = some.new_empty((M, D), dtype=xt)
    if residual and dy is None:
        dy = some.new_empty((M, D), dtype=_BF16)
    lddx = 0 if dx is None else _matrix(dx, "dx", xt, M, D, dev)
    lddy = 0 if dy is None else _matrix(dy, "dy", _BF16, M, D, dev)
    # the gradients of modulation vectors share one allocation, those of weights another
    out, buf, nws = [None] * 6, None, 0
    mods, weights = sum(wanted[:3]), sum(wanted[3:])
    if mods:
        parts = iter(some.new_empty((mods, B, D), dtype=_F32).unbind(0))
        out[:3] = [next(parts) if w else None for w in wanted[:3]]
    if weights:
        parts = iter(some.new_empty((weights, D), dtype=_F32).unbind(0))
        out[3:] = [next(parts) if w else None for w in wanted[3:]]
    if mods or weights:
        nws = load().ft_gated_norm_workspace_bytes(M, D, B)
        buf = _scratch(ws, nws, some)
    dgate, dscale, dshift, dw, db, dwp = out
    g = _NORM_GRADS.pack(_ptr(dx), lddx, _ptr(dy), lddy, _ptr(dgate), _ptr(dscale), _ptr(dshift), _ptr(dwp), _ptr(dw),
                         _ptr(db), _f32(amax_dy, "amax_dy", 1, dev))
    check("ft_gated_norm_bwd", load().ft_gated_norm_bwd(
        n, _ptr(dh), lddh, _ptr(dr), lddr, _ptr(r), ldr, _ptr(y), ldy, _f32(stats, "stats", 4 * M, dev), g,
        _ptr(buf), nws, _raw_stream(dev)))
    for i in range(3):
        if wanted[i] and given[i].shape != (B, D):  # one for all samples
            out[i] = (out[i].sum(0) if B > 1 else out[i]).view(given[i].shape)
    return GatedNormGrads(dx, dy, *out)


# ---------------------------------------------------------------- GELU backward
@_on_device(0)
def ft_gelu_bwd_bf16(y: torch.Tensor, dh: torch.Tensor, out: torch.Tensor | None = None,
                     amax_dy: torch.Tensor | None = None) -> torch.Tensor:
    """dy = dh GELU'(y) on bf16, the backward of ft_gelu_bf16.  amax_dy: an
    optional float32 device scalar (>= 0) raised to max|dy|."""
    out = torch.empty_like(y) if out is None else out
    dev, shape = y.get_device(), y.shape
    for name, t in (("y", y), ("dh", dh), ("out", out)):
        if t.dtype is not _BF16:
            raise TypeError(f"{name} must be a CUDA bfloat16 tensor")
        if t.get_device() != dev:
            _same_device(t, dev, name)
        if not t.is_contiguous() or t.shape != shape:
            raise ValueError(f"{name} must be contiguous and of y's shape")
    check("ft_gelu_bwd_bf16", load().ft_gelu_bwd_bf16(
        y.data_ptr(), dh.data_ptr(), out.data_ptr(), y.numel(), _f32(amax_dy, "amax_dy", 1, dev), _raw_stream(dev)))
    return out


# ---------------------------------------------------------------- rotary positions
@dataclass
class Rope:
    """The rotation of a QKV linear's queries and keys: `heads` query heads
    and `kv_heads` key and value heads of head_dim; axes: how many of a
    head's values each position axis turns (their sum may leave a rest that
    passes through); freqs: float64 [sum(axes) / 2] radians per position
    (rope_freqs); an optional RMS norm of each head first, with weights
    [head_dim] (bf16 or float32)."""
    heads: int
    kv_heads: int
    head_dim: int
    axes: tuple
    freqs: torch.Tensor
    layout: int = ROPE_PAIRS
    norm: bool = False
    w_q: torch.Tensor | None = None
    w_k: torch.Tensor | None = None
    eps: float = 1e-6

    @property
    def width(self) -> int:
        return (self.heads + 2 * self.kv_heads) * self.head_dim


def rope_freqs(axes, theta: float = 10000.0, shared: bool = False, device="cuda") -> torch.Tensor:
    """Frequencies of the pairs of each axis: theta^(-2 i / d) with i counted
    and d taken within the axis, or with `shared` over all rotated values."""
    if shared:
        d = sum(axes)
        return theta ** (-2.0 * torch.arange(d // 2, dtype=torch.float64, device=device) / d)
    return torch.cat([theta ** (-2.0 * torch.arange(a // 2, dtype=torch.float64, device=device) / a) for a in axes])


def _rope_view(rope: Rope, pos: torch.Tensor, M: int, S: int, dev: int) -> bytes:
    axes = rope.axes
    na, rot = len(axes), sum(axes)
    if not 1 <= na <= 4:
        raise ValueError("rotary positions have one to four axes")
    if pos.dtype is not torch.int32 and pos.dtype is not _F32:
        raise TypeError(f"pos must be int32 or float32, not {pos.dtype}")
    if (pos.shape != (M, na) and not (na == 1 and pos.shape == (M,))) or not pos.is_contiguous():
        raise ValueError(f"pos must be contiguous [{M}, {na}], not {list(pos.shape)}")
    f, wq, wk, hd = rope.freqs, rope.w_q, rope.w_k, rope.head_dim
    if f.dtype is not torch.float64 or f.numel() != rot // 2 or not f.is_contiguous():
        raise TypeError(f"freqs must be a contiguous float64 tensor of {rot // 2}")
    pt = None
    for name, w in (("w_q", wq), ("w_k", wk)):
        if w is not None:
            if w.dtype not in _DTYPE or (pt is not None and w.dtype is not pt):
                raise TypeError("w_q and w_k must both be bfloat16 or both float32")
            if w.shape != (hd,) or not w.is_contiguous():
                raise ValueError(f"{name} must be contiguous [{hd}]")
            _same_device(w, dev, name)
            pt = w.dtype
    _same_device(pos, dev, "pos")
    _same_device(f, dev, "freqs")
    return _ROPE.pack(M, S, rope.heads, rope.kv_heads, hd, na, *axes, *(0,) * (4 - na), rope.layout,
                      NORM_RMS if rope.norm else NORM_NONE, rope.eps, 0 if pos.dtype is torch.int32 else 1,
                      0 if pt is _BF16 else 1, pos.data_ptr(), f.data_ptr(), _ptr(wq), _ptr(wk))


_NO_HEADS = _HEADS.pack(0, 0, 0, 0)


def _heads(t, name: str, shape: tuple, dev: int, out: bool) -> bytes:
    if t is None:
        return _NO_HEADS
    if t.dtype is not _BF16:
        raise TypeError(f"{name} must be a CUDA bfloat16 tensor")
    if t.get_device() != dev:
        _same_device(t, dev, name)
    if t.shape != shape:
        raise ValueError(f"{name} must be {list(shape)}, not {list(t.shape)}")
    sb, sh, st, unit = t.stride()
    if unit != 1:
        raise ValueError(f"{name} must have unit stride along a head")
    B, H, S, _ = shape
    # the stride of an axis of one element says nothing
    sb, sh, st = sb if B > 1 else 0, sh if H > 1 else 0, st if S > 1 else 0
    if out and ((B > 1 and sb == 0) or (H > 1 and sh == 0) or (S > 1 and st == 0)):
        raise ValueError(f"{name} is written: its elements must be apart")
    return _HEADS.pack(t.data_ptr(), sb, sh, st)


@_on_device(1)
def ft_qk_rope_fwd(rope: Rope, qkv: torch.Tensor, pos: torch.Tensor, *, tokens: int | None = None,
                   head_major: bool = True, q: torch.Tensor | None = None, k: torch.Tensor | None = None,
                   v: torch.Tensor | None = None, copy_v: bool = True):
    """Splits qkv (bf16 [M, rope.width]) into q, k, v as [samples, heads,
    tokens, head_dim], queries and keys normed and rotated by pos (int32 or
    float32 [M, axes]).  tokens: rows per sample (M: one sample).  Outputs
    that are not given are allocated head by head (head_major) or token by
    token in memory; given ones may have any strides, views of qkv itself
    among them (in place).  copy_v=False: v is returned as a view of qkv."""
    if qkv.dim() != 2:
        raise ValueError("qkv must be [rows, width]")
    M, dev = len(qkv), qkv.get_device()
    S = M if tokens is None else tokens
    if S < 0 or (M > 0 and (S < 1 or M % S)):
        raise ValueError(f"{M} rows are no samples of {S} tokens")
    B = M // S if S else 0
    Hq, Hk, hd = rope.heads, rope.kv_heads, rope.head_dim
    ld = _matrix(qkv, "qkv", _BF16, M, rope.width, dev)

    def new(H):
        return qkv.new_empty((B, H, S, hd)) if head_major else qkv.new_empty((B, S, H, hd)).transpose(1, 2)

    view = _rope_view(rope, pos, M, S, dev)
    q = new(Hq) if q is None else q
    k = new(Hk) if k is None else k
    if v is None and copy_v:
        v = new(Hk)
    hq = _heads(q, "q", (B, Hq, S, hd), dev, True)
    hk = _heads(k, "k", (B, Hk, S, hd), dev, True)
    hv = _heads(v, "v", (B, Hk, S, hd), dev, True)
    check("ft_qk_rope_fwd", load().ft_qk_rope_fwd(view, qkv.data_ptr(), ld, hq, hk, hv, _raw_stream(dev)))
    if v is None:
        v = qkv[:, (Hq + Hk) * hd:].unflatten(1, (Hk, hd)).unflatten(0, (B, S)).transpose(1, 2)
    return q, k, v


@_on_device(1)
def ft_qk_rope_bwd(rope: Rope, dq: torch.Tensor, dk: torch.Tensor, dv: torch.Tensor | None, pos: torch.Tensor, *,
                   qkv: torch.Tensor | None = None, dqkv: torch.Tensor | None = None, weight_grads: bool = True,
                   amax: torch.Tensor | None = None, ws=None):
    """The gradient of qkv from those of q, k and v ([samples, heads, tokens,
    head_dim], any strides).  qkv: the forward's input, needed with the norm
    (not after a forward in place).  dv=None leaves dqkv's value columns as
    they are (zero where dqkv is not given).  amax: an optional float32 device
    scalar (>= 0) raised to max|dqkv|.  Returns (dqkv, dw_q, dw_k)."""
    if dq.dim() != 4:
        raise ValueError("dq must be [samples, heads, tokens, head_dim]")
    B, _, S, _ = dq.shape
    M, dev = B * S, dq.get_device()
    Hq, Hk, hd = rope.heads, rope.kv_heads, rope.head_dim
    if rope.norm and qkv is None:
        raise ValueError("the gradient through the norm needs qkv")
    view = _rope_view(rope, pos, M, S, dev)
    ld = 0 if qkv is None else _matrix(qkv, "qkv", _BF16, M, rope.width, dev)
    if dqkv is None:
        dqkv = (dq.new_zeros if dv is None else dq.new_empty)((M, rope.width))
    ldd = _matrix(dqkv, "dqkv", _BF16, M, rope.width, dev)
    hq = _heads(dq, "dq", (B, Hq, S, hd), dev, False)
    hk = _heads(dk, "dk", (B, Hk, S, hd), dev, False)
    hv = _heads(dv, "dv", (B, Hk, S, hd), dev, False)
    dw_q = dw_k = buf = None
    nws = 0
    if weight_grads and rope.norm:
        dw_q = None if rope.w_q is None else dq.new_empty(hd, dtype=_F32)
        dw_k = None if rope.w_k is None else dq.new_empty(hd, dtype=_F32)
        if dw_q is not None or dw_k is not None:
            nws = load().ft_qk_rope_workspace_bytes(M, hd)
            buf = _scratch(ws, nws, dq)
    check("ft_qk_rope_bwd", load().ft_qk_rope_bwd(
        view, hq, hk, hv, _ptr(qkv), ld, dqkv.data_ptr(), ldd, _ptr(dw_q), _ptr(dw_k), _f32(amax, "amax", 1, dev),
        _ptr(buf), nws, _raw_stream(dev)))
    return dqkv, dw_q, dw_k
