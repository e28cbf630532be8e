"""64-bit formulas of the operators around the linears, for the tests: plain
torch on float64 tensors, differentiable, and the roundings a kernel is
allowed."""
import math

import torch

EPS = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24, torch.float16: 2.0 ** -11}
U32 = 2.0 ** -24


def check_rounded(got, ref, slack):
    """got = ref + at most `slack` (the FP32 steps' error, elementwise or a
    number), rounded once to its type: half a step of the value before the
    rounding, or of the subnormals' spacing."""
    u = EPS[got.dtype]
    g, ref = got.double(), ref.double()
    slack = torch.as_tensor(slack, dtype=torch.float64, device=g.device)
    tiny = 2.0 ** -134 if got.dtype == torch.bfloat16 else 2.0 ** -150
    bound = slack + u * (ref.abs() + slack) + tiny
    excess = (g - ref).abs() - bound
    assert torch.isfinite(g).all()
    assert bool((excess <= 0).all()), (float(excess.max()), int(excess.argmax()), float((g - ref).abs().max()))


def norm64(x, kind, eps):
    """(normalised, mean, 1 / deviation)"""
    mean = x.mean(1, keepdim=True) if kind == 2 else torch.zeros_like(x[:, :1])
    if kind == 0:
        return x, mean, torch.ones_like(mean)
    rstd = 1 / ((x - mean).square().mean(1, keepdim=True) + eps).sqrt()
    return (x - mean) * rstd, mean, rstd


def rows_of(vec, sample):
    """A gate, scale or shift ([B, D], [1, D] or [D]) row by row."""
    if vec is None or vec.dim() == 1 or vec.shape[0] == 1:
        return vec
    return vec[sample]


def gated_norm64(x, y, gate, scale, shift, w, bias, w_post, pre, post, alpha, eps, sample, r_stored=None):
    """(r, h): float64; h from `r_stored` where it is given."""
    r = x
    if y is not None:
        u = norm64(y, post, eps)[0]
        u = u if w_post is None else u * w_post
        u = u if gate is None else u * rows_of(gate, sample)
        r = x + alpha * u
    if pre == 0:
        return r, None
    n = norm64(r if r_stored is None else r_stored, pre, eps)[0]
    n = n if w is None else n * w
    n = n if bias is None else n + bias
    n = n if scale is None else n * (1 + rows_of(scale, sample))
    return r, n if shift is None else n + rows_of(shift, sample)


def rope64(x, ang, rot, halves):
    """x [M, heads, hd] float64, ang [M, rot / 2]."""
    cos, sin = ang.cos()[:, None], ang.sin()[:, None]
    if halves:
        a, b = x[..., :rot // 2], x[..., rot // 2:rot]
        return torch.cat([a * cos - b * sin, b * cos + a * sin, x[..., rot:]], -1)
    a, b = x[..., 0:rot:2], x[..., 1:rot:2]
    return torch.cat([torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2), x[..., rot:]], -1)


def gelu_slope64(y):
    return 0.5 * torch.special.erfc(-y / math.sqrt(2)) + y * torch.exp(-0.5 * y * y) / math.sqrt(2 * math.pi)


def differences(f, x, direction, step):
    """Central difference of f at x along direction, and a bound on its own
    error from halving the step."""
    d1 = (f(x + step * direction) - f(x - step * direction)) / (2 * step)
    d2 = (f(x + step / 2 * direction) - f(x - step / 2 * direction)) / step
    return d2, (d2 - d1).abs()
