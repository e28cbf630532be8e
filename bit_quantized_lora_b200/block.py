"""A DiT block's training step around its four triple-branch linears.

FourTune replaces the linears of a diffusion transformer's blocks and reports
the DiT training step as a whole (section 4.2); the block around them is the
usual one: each half reads a norm modulated by the sample's conditioning and
returns through a gate,

    h1 = N(x) (1 + scale1) + shift1        q, k, v = rope(norm(QKV(h1)))
    r  = x + gate1 Out(attention(q, k, v))
    h2 = N(r) (1 + scale2) + shift2        x' = r + gate2 Down(GELU(Up(h2)))

`DitBlock` runs its forward and its backward over the C ABI: the residual of
one half and the norm of the next are one kernel.  The norms find the tensor
amax of QKV's and Up's inputs on the way, and the kernel before each linear's
backward that of its output gradient, so that these are quantized in a single
pass; Out and Down look for their inputs' themselves (they follow the
attention and GELU).  The attention itself is the caller's.
"""
from __future__ import annotations

from dataclasses import dataclass

import torch

from . import (Layer, Workspace, ft_gelu_bf16, ft_linear_bwd, ft_linear_fwd, ft_workspace_bytes)
from .blockops import (NORM_LAYER, NORM_NONE, GatedNorm, Rope, ft_gated_norm_bwd, ft_gated_norm_fwd,
                       ft_gelu_bwd_bf16, ft_qk_rope_bwd, ft_qk_rope_fwd)

# rows of a block's modulation [samples, 6, D]
SHIFT1, SCALE1, GATE1, SHIFT2, SCALE2, GATE2 = range(6)


@dataclass
class BlockGrads:
    """What a block's backward returns: the gradients of x, of the
    modulation (float32 [samples, 6, D]), of the adapters (dA, dB) of the
    four linears in the order qkv, out, up, down, and of the query and key
    norms' weights."""
    dx: torch.Tensor
    dmod: torch.Tensor
    adapters: list
    dw_q: torch.Tensor | None
    dw_k: torch.Tensor | None


class DitBlock:
    """One block: the layers qkv [(heads + 2 kv_heads) head_dim, D], out
    [D, heads head_dim], up [F, D] and down [D, F], the rotation of its
    queries and keys, and the kind of its two norms.

    forward(x, mod, pos, attention): x bf16 or float32 [M, D] of `samples`
    times M / samples tokens (the rows of mod), mod [samples, 6, D], pos
    [M, axes].  attention.forward(q, k, v) takes [samples, heads, tokens,
    head_dim] and returns (o of q's shape, what its backward needs);
    attention.backward(do, saved) returns (dq, dk, dv).  Returns (x', saved).
    backward(dx', saved, attention) returns BlockGrads.  A block's calls share
    its workspace and go to one stream at a time."""

    def __init__(self, qkv: Layer, out: Layer, up: Layer, down: Layer, rope: Rope, norm: int = NORM_LAYER,
                 eps: float = 1e-6):
        D = qkv.K
        if qkv.N != rope.width or out.K != rope.heads * rope.head_dim or out.N != D:
            raise ValueError("the attention's linears and its heads do not fit together")
        if up.K != D or down.N != D or down.K != up.N:
            raise ValueError("the MLP's linears do not fit together")
        self.qkv, self.out, self.up, self.down, self.rope, self.D = qkv, out, up, down, rope, D
        self.norm = GatedNorm(pre=norm, eps=eps)
        self.end = GatedNorm(pre=NORM_NONE)
        self.ws = Workspace()

    @property
    def layers(self) -> list[Layer]:
        return [self.qkv, self.out, self.up, self.down]

    def _workspace(self, M: int, device) -> Workspace:
        self.ws.get(max(ft_workspace_bytes(M, L.N, L.K, L.r_s, L.r_l) for L in self.layers), device)
        return self.ws

    def forward(self, x: torch.Tensor, mod: torch.Tensor, pos: torch.Tensor, attention):
        M, D = x.shape
        B = len(mod)
        if mod.shape != (B, 6, D) or B < 1 or M < 1 or M % B:
            raise ValueError(f"mod must be [samples, 6, {D}] with samples that divide the {M} rows of x")
        ws = self._workspace(M, x.device)
        amax = x.new_zeros(2, dtype=torch.float32)
        h1, st1 = ft_gated_norm_fwd(self.norm, x, scale=mod[:, SCALE1], shift=mod[:, SHIFT1], amax_h=amax[:1])[1:]
        y_qkv, p_qkv = ft_linear_fwd(self.qkv, h1, amax_x=amax[:1], ws=ws)
        q, k, v = ft_qk_rope_fwd(self.rope, y_qkv, pos, tokens=M // B)
        o, saved_attn = attention.forward(q, k, v)
        o = o.transpose(1, 2).reshape(M, self.out.K)
        y_out, p_out = ft_linear_fwd(self.out, o, ws=ws)
        r, h2, st2 = ft_gated_norm_fwd(self.norm, x, y_out, mod[:, GATE1], mod[:, SCALE2], mod[:, SHIFT2],
                                       amax_h=amax[1:])
        y_up, p_up = ft_linear_fwd(self.up, h2, amax_x=amax[1:], ws=ws)
        h = ft_gelu_bf16(y_up)
        y_down, p_down = ft_linear_fwd(self.down, h, ws=ws)
        x2 = ft_gated_norm_fwd(self.end, r, y_down, mod[:, GATE2], stats=False)[0]
        saved = (x, mod, pos, h1, st1, y_qkv, p_qkv, saved_attn, o, p_out, y_out, r, h2, st2, y_up, p_up, h, p_down,
                 y_down)
        return x2, saved

    def backward(self, dx2: torch.Tensor, saved, attention) -> BlockGrads:
        (x, mod, pos, h1, st1, y_qkv, p_qkv, saved_attn, o, p_out, y_out, r, h2, st2, y_up, p_up, h, p_down,
         y_down) = saved
        M, D = x.shape
        B = len(mod)
        ws = self._workspace(M, x.device)
        amax = x.new_zeros(4, dtype=torch.float32)
        dmod = x.new_empty((B, 6, D), dtype=torch.float32)
        # x' = r + gate2 y_down
        g = ft_gated_norm_bwd(self.end, None, None, None, dr=dx2, y=y_down, gate=mod[:, GATE2], need_dx=False,
                              amax_dy=amax[:1])
        dmod[:, GATE2] = g.dgate
        dh, *g_down = ft_linear_bwd(self.down, g.dy, h, p_down, amax_dy=amax[:1], ws=ws)
        dy = ft_gelu_bwd_bf16(y_up, dh, out=dh, amax_dy=amax[1:2])
        dh2, *g_up = ft_linear_bwd(self.up, dy, h2, p_up, amax_dy=amax[1:2], ws=ws)
        # r = x + gate1 y_out, h2 = N(r)
        g = ft_gated_norm_bwd(self.norm, dh2, r, st2, dr=dx2, y=y_out, gate=mod[:, GATE1], scale=mod[:, SCALE2],
                              shift=mod[:, SHIFT2], amax_dy=amax[2:3])
        dmod[:, GATE1], dmod[:, SCALE2], dmod[:, SHIFT2] = g.dgate, g.dscale, g.dshift
        do, *g_out = ft_linear_bwd(self.out, g.dy, o, p_out, amax_dy=amax[2:3], ws=ws)
        do = do.view(B, M // B, self.rope.heads, self.rope.head_dim).transpose(1, 2)
        # autograd may hand back gradients that lie the other way round
        dq, dk, dv = (t if t.stride(-1) == 1 else t.contiguous() for t in attention.backward(do, saved_attn))
        dqkv, dw_q, dw_k = ft_qk_rope_bwd(self.rope, dq, dk, dv, pos, qkv=y_qkv, amax=amax[3:])
        dh1, *g_qkv = ft_linear_bwd(self.qkv, dqkv, h1, p_qkv, amax_dy=amax[3:], ws=ws)
        # h1 = N(x)
        g = ft_gated_norm_bwd(self.norm, dh1, x, st1, dr=g.dx, scale=mod[:, SCALE1], shift=mod[:, SHIFT1])
        dmod[:, SCALE1], dmod[:, SHIFT1] = g.dscale, g.dshift
        return BlockGrads(g.dx, dmod, [tuple(p) for p in (g_qkv, g_out, g_up, g_down)], dw_q, dw_k)
