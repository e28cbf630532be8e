"""Operators of a DiT block between its linears, over the C ABI: the gated
norm (residual with gate, norm with modulation), the rotary positions of
queries and keys, and GELU's backward.  Each hands the next linear the tensor
amax of what it writes (amax_h, amax_dy, amax), so that ft_linear_fwd and
ft_linear_bwd quantize in a single pass.

Calls run on `stream`, or on the current stream of their tensors' device;
what they allocate (outputs that are not given, scratch) belongs to that
stream.  They may be captured in a CUDA graph, which then owns their scratch
(a Workspace that the call is given is not used in a capture).
"""
from __future__ import annotations

import functools
from dataclasses import dataclass

import torch

from ._lib import load_torch

NORM_NONE, NORM_RMS, NORM_LAYER = 0, 1, 2
ROPE_PAIRS, ROPE_HALVES = 0, 1


def _on_device(at: int):
    """Runs a call with its tensors' device and the stream it was given (or
    that device's current one) current; argument `at` is such a tensor."""
    def wrap(fn):
        name = fn.__code__.co_varnames[at]

        @functools.wraps(fn)
        def call(*args, stream=None, **kw):
            some = args[at] if len(args) > at else kw.get(name)
            if not isinstance(some, torch.Tensor):
                raise TypeError(f"{fn.__name__} needs CUDA tensors")
            dev = some.get_device()
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
    return load_torch().gated_norm_fwd(norm, x, y, gate, scale, shift, offsets, r, h, stats, amax_h)


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
    amax_dy: an optional float32 device scalar (>= 0) raised to max|dy|.  ws:
    a Workspace for the parameters' sums in place of scratch of the call's own
    (it may be the linears', in turn)."""
    some = dh if dh is not None else dr
    if some is None:
        raise ValueError("one of dh and dr must be given")
    if param_grads is True:
        wanted = None
    else:
        names = set(param_grads or ())
        if not names.issubset(_PARAMS):
            raise ValueError(f"no gradient for {sorted(names.difference(_PARAMS))}")
        wanted = [k in names for k in _PARAMS]
    return GatedNormGrads(*_gated_norm_bwd(some, norm, dh, r, stats, dr, y, gate, scale, shift, offsets, residual,
                                           need_dx, dx, dy, wanted, amax_dy, ws, stream=stream))


@_on_device(0)
def _gated_norm_bwd(*args):
    return load_torch().gated_norm_bwd(*args)


# ---------------------------------------------------------------- GELU backward
@_on_device(0)
def ft_gelu_bwd_bf16(y: torch.Tensor, dh: torch.Tensor, out: torch.Tensor | None = None,
                     amax_dy: torch.Tensor | None = None) -> torch.Tensor:
    """dy = dh GELU'(y) on bf16, the backward of ft_gelu_bf16.  amax_dy: an
    optional float32 device scalar (>= 0) raised to max|dy|."""
    return load_torch().gelu_bwd(y, dh, out, amax_dy)


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
    return load_torch().qk_rope_fwd(rope, qkv, pos, tokens, head_major, q, k, v, copy_v)


@_on_device(1)
def ft_qk_rope_bwd(rope: Rope, dq: torch.Tensor, dk: torch.Tensor, dv: torch.Tensor | None, pos: torch.Tensor, *,
                   qkv: torch.Tensor | None = None, dqkv: torch.Tensor | None = None, weight_grads: bool = True,
                   amax: torch.Tensor | None = None, ws=None):
    """The gradient of qkv from those of q, k and v ([samples, heads, tokens,
    head_dim], any strides).  qkv: the forward's input, needed with the norm
    (not after a forward in place).  dv=None leaves dqkv's value columns as
    they are (zero where dqkv is not given).  amax: an optional float32 device
    scalar (>= 0) raised to max|dqkv| over the columns written: with dv=None
    it does not see a given dqkv's value columns, so raise it to max|dv| too
    before ft_linear_bwd takes it.  ws: a Workspace for the weights' sums in
    place of scratch of the call's own (it may be the linears', in turn).
    Returns (dqkv, dw_q, dw_k)."""
    return load_torch().qk_rope_bwd(rope, dq, dk, dv, pos, qkv, dqkv, weight_grads, amax, ws)
