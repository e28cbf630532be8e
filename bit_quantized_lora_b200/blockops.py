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

import ctypes
import functools
from dataclasses import dataclass

import torch

from ._lib import FtGatedNorm, FtGatedNormGrads, FtHeads, FtRope, check, load

NORM_NONE, NORM_RMS, NORM_LAYER = 0, 1, 2
ROPE_PAIRS, ROPE_HALVES = 0, 1
_DTYPE = {torch.bfloat16: 0, torch.float32: 1}


def _on_device(at: int):
    """Runs a call with its tensors' device and the stream it was given (or
    that device's current one) current; argument `at` is such a tensor."""
    def wrap(fn):
        @functools.wraps(fn)
        def call(*args, stream=None, **kw):
            dev = args[at].device
            if dev.type != "cuda":
                raise TypeError(f"{fn.__name__} needs CUDA tensors")
            if stream is None and dev.index == torch.cuda.current_device():
                return fn(*args, **kw)
            stream = torch.cuda.current_stream(dev) if stream is None else stream
            if stream.device != dev:
                raise ValueError(f"the stream is on {stream.device}, the tensors are on {dev}")
            with torch.cuda.stream(stream):
                return fn(*args, **kw)
        return call
    return wrap


def _raw_stream(t: torch.Tensor) -> int:
    return torch.cuda.current_stream(t.device).cuda_stream


def _ptr(t):
    return None if t is None else t.data_ptr()


def _same_device(t: torch.Tensor, dev, name: str) -> None:
    if t.device != dev:
        raise ValueError(f"{name} is on {t.device}, the call is on {dev}")


def _matrix(t: torch.Tensor, name: str, dtype, rows: int, cols: int, dev) -> int:
    """Checks a row-major matrix and returns its leading dimension."""
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, not {t.dtype}")
    _same_device(t, dev, name)
    if tuple(t.shape) != (rows, cols):
        raise ValueError(f"{name} must be [{rows}, {cols}], not {list(t.shape)}")
    if t.stride(1) != 1 and cols > 1:
        raise ValueError(f"{name} must have unit column stride")
    return t.stride(0) if rows > 1 else cols


def _f32(t, name: str, n: int, dev):
    if t is None:
        return None
    if t.dtype != torch.float32 or t.numel() < n or not t.is_contiguous():
        raise TypeError(f"{name} must be a contiguous float32 tensor of {n}")
    _same_device(t, dev, name)
    return t.data_ptr()


def _scratch(ws, nbytes: int, dev):
    """Scratch of one call: the caller's workspace, or memory of the current
    stream (an allocation that a captured graph owns with the call)."""
    return ws.get(nbytes, dev) if ws is not None else torch.empty(nbytes, dtype=torch.uint8, device=dev)


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


def _norm_view(norm: GatedNorm, M: int, D: int, xt, mods, offsets, dev):
    """FtGatedNorm of a call, and its number of samples."""
    rows = {m.shape[0] if m.dim() == 2 else 1 for m in mods if m is not None} - {1}
    if offsets is not None:
        if offsets.dtype != torch.int32 or offsets.dim() != 1 or offsets.numel() < 2 or not offsets.is_contiguous():
            raise TypeError("offsets must be a contiguous int32 tensor [samples + 1]")
        _same_device(offsets, dev, "offsets")
        rows.add(offsets.numel() - 1)
    rows = rows - {1} if len(rows) > 1 else rows
    if len(rows) > 1:
        raise ValueError(f"gate, scale, shift and offsets disagree on the samples: {sorted(rows)}")
    B = rows.pop() if rows else 1
    pt, ld = None, []
    for name, t in zip(("gate", "scale", "shift"), mods):
        if t is None:
            ld.append(0)
            continue
        if t.dim() not in (1, 2) or t.shape[-1] != D or (t.dim() == 2 and t.shape[0] not in (1, B)):
            raise ValueError(f"{name} must be [{B}, {D}] or [{D}], not {list(t.shape)}")
        if t.stride(-1) != 1:
            raise ValueError(f"{name} must have unit column stride")
        ld.append(t.stride(0) if t.dim() == 2 and t.shape[0] > 1 else 0)
    for name, t in (("weight", norm.weight), ("bias", norm.bias), ("w_post", norm.w_post)):
        if t is not None and (tuple(t.shape) != (D,) or not t.is_contiguous()):
            raise ValueError(f"{name} must be contiguous [{D}], not {list(t.shape)}")
    for t in (*mods, norm.weight, norm.bias, norm.w_post):
        if t is None:
            continue
        _same_device(t, dev, "a parameter vector")
        if t.dtype not in _DTYPE or (pt is not None and t.dtype != pt):
            raise TypeError("gate, scale, shift and the norms' weights must all be bfloat16 or all float32")
        pt = t.dtype
    if xt not in _DTYPE:
        raise TypeError(f"the residual stream must be bfloat16 or float32, not {xt}")
    eps_post = norm.eps if norm.eps_post is None else norm.eps_post
    return FtGatedNorm(M, D, B, _ptr(offsets), norm.pre, norm.post, norm.eps, eps_post, norm.alpha, _DTYPE[xt],
                       _DTYPE[pt or torch.float32], *ld, *map(_ptr, mods), _ptr(norm.w_post), _ptr(norm.weight),
                       _ptr(norm.bias)), B


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
    dev = x.device
    n, _ = _norm_view(norm, M, D, x.dtype, (gate, scale, shift), offsets, dev)
    ldx = _matrix(x, "x", x.dtype, M, D, dev)
    ldy = ldr = ldh = 0
    if y is not None:
        ldy = _matrix(y, "y", torch.bfloat16, M, D, dev)
        r = torch.empty(M, D, dtype=x.dtype, device=dev) if r is None else r
        ldr = _matrix(r, "r", x.dtype, M, D, dev)
    elif r is not None:
        raise ValueError("r is written only with y")
    if norm.pre != NORM_NONE:
        h = torch.empty(M, D, dtype=torch.bfloat16, device=dev) if h is None else h
        ldh = _matrix(h, "h", torch.bfloat16, M, D, dev)
    elif h is not None:
        raise ValueError("h is written only with a pre norm")
    if stats is True:
        stats = torch.empty(M, 4, dtype=torch.float32, device=dev)
    elif stats is False:
        stats = None
    check("ft_gated_norm_fwd", load().ft_gated_norm_fwd(
        ctypes.byref(n), x.data_ptr(), ldx, _ptr(y), ldy, _ptr(r), ldr, _ptr(h), ldh,
        _f32(stats, "stats", 4 * M, dev), _f32(amax_h, "amax_h", 1, dev), _raw_stream(x)))
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
    dev = some.device
    xt = r.dtype if r is not None else dr.dtype if dr is not None else dx.dtype if dx is not None else torch.bfloat16
    n, B = _norm_view(norm, M, D, xt, (gate, scale, shift), offsets, dev)
    given = dict(gate=gate, scale=scale, shift=shift, weight=norm.weight, bias=norm.bias, w_post=norm.w_post)
    if param_grads is True:
        wanted = {k for k, v in given.items() if v is not None}
    else:
        wanted = set(param_grads or ())
        unknown = {k for k in wanted if k not in _PARAMS or given[k] is None}
        if unknown:
            raise ValueError(f"no gradient for {sorted(unknown)}: not among the parameters given")
    if residual is None:
        residual = y is not None or gate is not None or dy is not None or norm.post != NORM_NONE
    if y is None and (norm.post != NORM_NONE or wanted & {"gate", "w_post"}):
        raise ValueError("the post norm and the gradient of the gate need y")
    lds = {}
    for name, t, dtype in (("dh", dh, torch.bfloat16), ("dr", dr, xt), ("r", r, xt), ("y", y, torch.bfloat16)):
        lds[name] = 0 if t is None else _matrix(t, name, dtype, M, D, dev)
    if need_dx and dx is None:
        dx = torch.empty(M, D, dtype=xt, device=dev)
    if not need_dx:
        dx = None
    if residual and dy is None:
        dy = torch.empty(M, D, dtype=torch.bfloat16, device=dev)
    lddx = 0 if dx is None else _matrix(dx, "dx", xt, M, D, dev)
    lddy = 0 if dy is None else _matrix(dy, "dy", torch.bfloat16, M, D, dev)
    out = {k: torch.empty((B, D) if k in ("gate", "scale", "shift") else (D,), dtype=torch.float32, device=dev)
           for k in _PARAMS if k in wanted}
    nws = load().ft_gated_norm_workspace_bytes(M, D, B) if wanted else 0
    buf = _scratch(ws, nws, dev) if nws else None
    g = FtGatedNormGrads(_ptr(dx), lddx, _ptr(dy), lddy, *(_ptr(out.get(k)) for k in ("gate", "scale", "shift")),
                         *(_ptr(out.get(k)) for k in ("w_post", "weight", "bias")), _f32(amax_dy, "amax_dy", 1, dev))
    check("ft_gated_norm_bwd", load().ft_gated_norm_bwd(
        ctypes.byref(n), _ptr(dh), lds["dh"], _ptr(dr), lds["dr"], _ptr(r), lds["r"], _ptr(y), lds["y"],
        _f32(stats, "stats", 4 * M, dev), ctypes.byref(g), _ptr(buf), 0 if buf is None else buf.numel(),
        _raw_stream(some)))
    for k in ("gate", "scale", "shift"):
        if k in out and tuple(given[k].shape) != (B, D):
            out[k] = out[k].sum(0).view(given[k].shape)
    return GatedNormGrads(dx, dy, **{("dw_post" if k == "w_post" else "d" + k): v for k, v in out.items()})


# ---------------------------------------------------------------- GELU backward
@_on_device(0)
def ft_gelu_bwd_bf16(y: torch.Tensor, dh: torch.Tensor, out: torch.Tensor | None = None,
                     amax_dy: torch.Tensor | None = None) -> torch.Tensor:
    """dy = dh GELU'(y) on bf16, the backward of ft_gelu_bf16.  amax_dy: an
    optional float32 device scalar (>= 0) raised to max|dy|."""
    out = torch.empty_like(y) if out is None else out
    for name, t in (("y", y), ("dh", dh), ("out", out)):
        if t.dtype != torch.bfloat16:
            raise TypeError(f"{name} must be a CUDA bfloat16 tensor")
        _same_device(t, y.device, name)
        if not t.is_contiguous() or t.shape != y.shape:
            raise ValueError(f"{name} must be contiguous and of y's shape")
    check("ft_gelu_bwd_bf16", load().ft_gelu_bwd_bf16(
        y.data_ptr(), dh.data_ptr(), out.data_ptr(), y.numel(), _f32(amax_dy, "amax_dy", 1, y.device),
        _raw_stream(y)))
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


def _rope_view(rope: Rope, pos: torch.Tensor, M: int, S: int, dev) -> FtRope:
    axes = tuple(rope.axes)
    if not 1 <= len(axes) <= 4:
        raise ValueError("rotary positions have one to four axes")
    if pos.dtype not in (torch.int32, torch.float32):
        raise TypeError(f"pos must be int32 or float32, not {pos.dtype}")
    if tuple(pos.shape) not in ((M, len(axes)),) + (((M,),) if len(axes) == 1 else ()) or not pos.is_contiguous():
        raise ValueError(f"pos must be contiguous [{M}, {len(axes)}], not {list(pos.shape)}")
    f = rope.freqs
    if f.dtype != torch.float64 or f.numel() != sum(axes) // 2 or not f.is_contiguous():
        raise TypeError(f"freqs must be a contiguous float64 tensor of {sum(axes) // 2}")
    pt = None
    for name, w in (("w_q", rope.w_q), ("w_k", rope.w_k)):
        if w is None:
            continue
        if w.dtype not in _DTYPE or (pt is not None and w.dtype != pt):
            raise TypeError("w_q and w_k must both be bfloat16 or both float32")
        if tuple(w.shape) != (rope.head_dim,) or not w.is_contiguous():
            raise ValueError(f"{name} must be contiguous [{rope.head_dim}]")
        _same_device(w, dev, name)
        pt = w.dtype
    _same_device(pos, dev, "pos")
    _same_device(f, dev, "freqs")
    return FtRope(M, S, rope.heads, rope.kv_heads, rope.head_dim, len(axes),
                  (ctypes.c_int32 * 4)(*axes), rope.layout, NORM_RMS if rope.norm else NORM_NONE, rope.eps,
                  0 if pos.dtype == torch.int32 else 1, _DTYPE[pt or torch.float32], pos.data_ptr(), f.data_ptr(),
                  _ptr(rope.w_q), _ptr(rope.w_k))


def _heads(t, name: str, B: int, H: int, S: int, hd: int, dev, out: bool) -> FtHeads:
    if t is None:
        return FtHeads(None, 0, 0, 0)
    if t.dtype != torch.bfloat16:
        raise TypeError(f"{name} must be a CUDA bfloat16 tensor")
    _same_device(t, dev, name)
    if tuple(t.shape) != (B, H, S, hd):
        raise ValueError(f"{name} must be [{B}, {H}, {S}, {hd}], not {list(t.shape)}")
    if t.stride(3) != 1:
        raise ValueError(f"{name} must have unit stride along a head")
    # the stride of an axis of one element says nothing
    st = [t.stride(i) if t.shape[i] > 1 else 0 for i in range(3)]
    if out and any(t.shape[i] > 1 and st[i] == 0 for i in range(3)):
        raise ValueError(f"{name} is written: its elements must be apart")
    return FtHeads(t.data_ptr(), *st)


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
    M, dev = qkv.shape[0], qkv.device
    S = M if tokens is None else tokens
    if S < 0 or (M > 0 and (S < 1 or M % S)):
        raise ValueError(f"{M} rows are no samples of {S} tokens")
    B = M // S if S else 0
    ld = _matrix(qkv, "qkv", torch.bfloat16, M, rope.width, dev)

    def new(H):
        if head_major:
            return torch.empty(B, H, S, rope.head_dim, dtype=torch.bfloat16, device=dev)
        return torch.empty(B, S, H, rope.head_dim, dtype=torch.bfloat16, device=dev).transpose(1, 2)

    view = _rope_view(rope, pos, M, S, dev)
    q = new(rope.heads) if q is None else q
    k = new(rope.kv_heads) if k is None else k
    if v is None and copy_v:
        v = new(rope.kv_heads)
    hq = _heads(q, "q", B, rope.heads, S, rope.head_dim, dev, True)
    hk = _heads(k, "k", B, rope.kv_heads, S, rope.head_dim, dev, True)
    hv = _heads(v, "v", B, rope.kv_heads, S, rope.head_dim, dev, True)
    check("ft_qk_rope_fwd", load().ft_qk_rope_fwd(ctypes.byref(view), qkv.data_ptr(), ld, ctypes.byref(hq),
                                                  ctypes.byref(hk), ctypes.byref(hv), _raw_stream(qkv)))
    if v is None:
        v = qkv[:, (rope.heads + rope.kv_heads) * rope.head_dim:].unflatten(1, (rope.kv_heads, rope.head_dim))
        v = v.unflatten(0, (B, S)).transpose(1, 2)
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
    M, dev = B * S, dq.device
    if rope.norm and qkv is None:
        raise ValueError("the gradient through the norm needs qkv")
    view = _rope_view(rope, pos, M, S, dev)
    ld = 0 if qkv is None else _matrix(qkv, "qkv", torch.bfloat16, M, rope.width, dev)
    if dqkv is None:
        new = torch.zeros if dv is None else torch.empty
        dqkv = new(M, rope.width, dtype=torch.bfloat16, device=dev)
    ldd = _matrix(dqkv, "dqkv", torch.bfloat16, M, rope.width, dev)
    hq = _heads(dq, "dq", B, rope.heads, S, rope.head_dim, dev, False)
    hk = _heads(dk, "dk", B, rope.kv_heads, S, rope.head_dim, dev, False)
    hv = _heads(dv, "dv", B, rope.kv_heads, S, rope.head_dim, dev, False)
    dw = [torch.empty(rope.head_dim, dtype=torch.float32, device=dev)
          if weight_grads and rope.norm and w is not None else None for w in (rope.w_q, rope.w_k)]
    buf = None
    if dw[0] is not None or dw[1] is not None:
        buf = _scratch(ws, load().ft_qk_rope_workspace_bytes(M, rope.head_dim), dev)
    check("ft_qk_rope_bwd", load().ft_qk_rope_bwd(
        ctypes.byref(view), ctypes.byref(hq), ctypes.byref(hk), ctypes.byref(hv), _ptr(qkv), ld, dqkv.data_ptr(), ldd,
        _ptr(dw[0]), _ptr(dw[1]), _f32(amax, "amax", 1, dev), _ptr(buf), 0 if buf is None else buf.numel(),
        _raw_stream(dq)))
    return dqkv, dw[0], dw[1]
