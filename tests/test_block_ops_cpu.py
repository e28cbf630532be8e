"""The operators around the linears on a host without a GPU: every refusal
of their C entry points happens before anything touches a device, and the
64-bit formulas that the GPU tests compare with have the right gradients."""
import ctypes

import pytest
import torch

import block_ref as R
import bit_quantized_lora_b200 as ft
from bit_quantized_lora_b200 import _lib
from bit_quantized_lora_b200._lib import (FtAdamwHyper, FtAdamwTensor, FtGatedNorm, FtGatedNormGrads, FtHeads, FtRope)

OK, ARG, SHAPE, ALIGN, WORKSPACE = 0, 1, 2, 3, 6
P = 0x100000  # a pointer that is never followed


@pytest.fixture(scope="module")
def L():
    return _lib.load(build_if_missing=True)


def test_struct_sizes():
    assert ctypes.sizeof(FtGatedNorm) == 4 * 8 + 7 * 4 + 4 + 9 * 8
    assert ctypes.sizeof(FtGatedNormGrads) == 11 * 8
    assert ctypes.sizeof(FtRope) == 2 * 8 + 13 * 4 + 4 + 4 * 8
    assert ctypes.sizeof(FtHeads) == 32
    assert ctypes.sizeof(FtAdamwTensor) == 72
    assert ctypes.sizeof(FtAdamwHyper) == 32


def test_the_torch_side_loads():
    m = _lib.load_torch()
    for name in ("gated_norm_fwd", "gated_norm_bwd", "gelu_bwd", "qk_rope_fwd", "qk_rope_bwd"):
        assert callable(getattr(m, name))
    from bit_quantized_lora_b200 import optim
    assert optim._HYPER.size == ctypes.sizeof(FtAdamwHyper)


def test_the_torch_side_says_what_is_wrong():
    """Refusals that name shapes and types, before any device is asked."""
    import bit_quantized_lora_b200 as ft
    m, x, z = _lib.load_torch(), torch.zeros(4, 64), torch.zeros

    def call(norm=ft.GatedNorm(), x=x, gate=None, scale=None, offsets=None):
        return m.gated_norm_fwd(norm, x, None, gate, scale, None, offsets, None, None, True, None)

    for error, text, kw in ((ValueError, r"gate must be \[3, 64\] or \[64\], not \[3, 5\]", dict(gate=z(3, 5))),
                            (ValueError, r"not \[2, 2, 2\]", dict(scale=z(2, 2, 2))),
                            (ValueError, r"weight must be contiguous \[64\], not \[3\]",
                             dict(norm=ft.GatedNorm(weight=z(3)))),
                            (ValueError, r"x must be \[rows, channels\]", dict(x=x[0])),
                            (TypeError, "bfloat16 or float32", dict(x=x.half())),
                            (TypeError, "int32", dict(offsets=z(2))),
                            (ValueError, "cpu", dict())):
        with pytest.raises(error, match=text):
            call(**kw)


def norm(**kw):
    d = dict(M=8, D=64, B=2, offsets=None, pre=2, post=0, eps_pre=1e-6, eps_post=1e-6, alpha=1.0, xt=0, pt=1,
             ld_gate=64, ld_scale=64, ld_shift=64, gate=P, scale=P, shift=P, w_post=None, w=None, bias=None)
    d.update(kw)
    return FtGatedNorm(**d)


def fwd(L, n, x=P, ldx=64, y=P, ldy=64, r=P, ldr=64, h=P, ldh=64, stats=P, amax=P):
    return L.ft_gated_norm_fwd(ctypes.byref(n), x, ldx, y, ldy, r, ldr, h, ldh, stats, amax, None)


def test_gated_norm_forward_refusals(L):
    assert L.ft_gated_norm_fwd(None, P, 64, P, 64, P, 64, P, 64, P, P, None) == ARG
    for bad in (dict(pre=3), dict(post=-1), dict(xt=2), dict(pt=-1), dict(B=0), dict(M=-1), dict(eps_pre=-1.0),
                dict(eps_pre=float("nan")), dict(w_post=P), dict(pre=0)):
        assert fwd(L, norm(**bad)) == ARG, bad
    for bad in (dict(D=60), dict(D=0), dict(D=8200), dict(M=7), dict(M=(1 << 30) + 2), dict(ld_gate=32),
                dict(ld_scale=-64)):
        assert fwd(L, norm(**bad), ldx=9000, ldy=9000, ldr=9000, ldh=9000) == SHAPE, bad
    for bad in (dict(gate=P + 4), dict(ld_shift=66), dict(w=P + 8), dict(offsets=P + 2)):
        assert fwd(L, norm(**bad)) == ALIGN, bad
    n = norm()
    assert fwd(L, n, x=None) == ARG
    assert fwd(L, n, h=None) == ARG          # a pre norm and nowhere to put it
    assert fwd(L, n, r=None) == ARG          # a residual and nowhere to put it
    assert fwd(L, n, y=None) == ARG          # r and a gate without y
    assert fwd(L, norm(gate=None), y=None) == ARG
    assert fwd(L, n, ldx=56) == SHAPE
    assert fwd(L, n, ldh=32) == SHAPE
    assert fwd(L, n, ldx=68) == ALIGN
    assert fwd(L, n, x=P + 8) == ALIGN
    assert fwd(L, n, stats=P + 8) == ALIGN
    assert fwd(L, n, amax=P + 1) == ALIGN
    assert fwd(L, norm(M=0)) == OK
    none = norm(pre=0, scale=None, shift=None)
    assert fwd(L, none) == ARG               # h without a pre norm
    assert fwd(L, none, h=None) == ARG       # an amax of nothing
    assert fwd(L, norm(pre=0, scale=None, shift=None, M=0), h=None, amax=None) == OK


def bwd(L, n, g, dh=P, dr=P, r=P, y=P, stats=P, ws=P, nws=1 << 30, ld=64):
    return L.ft_gated_norm_bwd(ctypes.byref(n), dh, ld, dr, ld, r, ld, y, ld, stats,
                               None if g is None else ctypes.byref(g), ws, nws, None)


def grads(**kw):
    d = dict(dx=P, lddx=64, dy=P, lddy=64, dgate=P, dscale=P, dshift=P)
    d.update(kw)
    return FtGatedNormGrads(**d)


def test_gated_norm_backward_refusals(L):
    n = norm()
    assert bwd(L, n, None) == ARG
    assert bwd(L, n, grads(), dh=None, dr=None) == ARG
    assert bwd(L, n, grads(), dh=None) == ARG
    assert bwd(L, n, grads(), r=None) == ARG
    assert bwd(L, n, grads(), y=None) == ARG       # the gate's gradient reads y
    assert bwd(L, n, grads(), stats=None) == ARG
    assert bwd(L, norm(gate=None), grads()) == ARG  # a gradient of nothing
    assert bwd(L, n, grads(dw=P)) == ARG
    assert bwd(L, n, grads(dw_post=P)) == ARG
    assert bwd(L, n, grads(dy=None, amax_dy=P)) == ARG
    assert bwd(L, n, grads(), ld=56) == SHAPE
    assert bwd(L, n, grads(lddx=8)) == SHAPE
    assert bwd(L, n, grads(), ld=68) == ALIGN
    assert bwd(L, n, grads(dx=P + 2)) == ALIGN
    assert bwd(L, n, grads(dgate=P + 2)) == ALIGN
    need = L.ft_gated_norm_workspace_bytes(8, 64, 2)
    assert bwd(L, n, grads(), nws=need - 1) == WORKSPACE
    assert bwd(L, n, grads(), ws=None) == WORKSPACE
    assert bwd(L, n, grads(), ws=P + 4) == ALIGN
    assert bwd(L, norm(M=0), grads(dgate=None, dscale=None, dshift=None)) == OK
    assert L.ft_gated_norm_workspace_bytes(-1, 64, 1) == 0
    assert L.ft_gated_norm_workspace_bytes(8, 60, 1) == 0
    assert L.ft_gated_norm_workspace_bytes(8, 64, 0) == 0
    a = [L.ft_gated_norm_workspace_bytes(m, 1024, 3) for m in (0, 1, 100, 10000, 1 << 30)]
    assert a == sorted(a) and a[0] > 0


def test_gelu_backward_refusals(L):
    assert L.ft_gelu_bwd_bf16(None, P, P, 8, None, None) == ARG
    assert L.ft_gelu_bwd_bf16(P, P, P, -8, None, None) == ARG
    assert L.ft_gelu_bwd_bf16(P, P, P, 12, None, None) == SHAPE
    assert L.ft_gelu_bwd_bf16(P, P + 8, P, 8, None, None) == ALIGN
    assert L.ft_gelu_bwd_bf16(P, P, P, 8, P + 2, None) == ALIGN
    assert L.ft_gelu_bwd_bf16(P, P, P, 0, None, None) == OK


def rope(**kw):
    d = dict(M=4, S=2, Hq=4, Hk=2, hd=64, n_axes=2, axis_dims=(ctypes.c_int32 * 4)(16, 32, 0, 0), layout=0, norm=1,
             eps=1e-6, pos_t=0, pt=1, pos=P, freqs=P, w_q=P, w_k=P)
    if "axis_dims" in kw:
        kw["axis_dims"] = (ctypes.c_int32 * 4)(*kw["axis_dims"])
    d.update(kw)
    return FtRope(**d)


def heads(**kw):
    d = dict(p=P, sb=512, sh=64, st=256)
    d.update(kw)
    return FtHeads(**d)


def rope_fwd(L, r, x=P, ld=512, q=None, k=None, v=None):
    q, k, v = (heads() if t is None else t for t in (q, k, v))
    return L.ft_qk_rope_fwd(ctypes.byref(r), x, ld, ctypes.byref(q), ctypes.byref(k), ctypes.byref(v), None)


def test_rope_refusals(L):
    h = heads()
    assert L.ft_qk_rope_fwd(None, P, 512, ctypes.byref(h), ctypes.byref(h), ctypes.byref(h), None) == ARG
    for bad in (dict(M=-1), dict(Hq=-1), dict(n_axes=0), dict(n_axes=5), dict(layout=2), dict(norm=2), dict(pos_t=2),
                dict(pt=3), dict(eps=-1.0), dict(norm=0), dict(pos=None), dict(freqs=None)):
        assert rope_fwd(L, rope(**bad)) == ARG, bad
    for bad in (dict(hd=60), dict(hd=264), dict(hd=0), dict(axis_dims=(15, 32, 0, 0)), dict(axis_dims=(64, 32, 0, 0)),
                dict(axis_dims=(-16, 32, 0, 0)), dict(axis_dims=(16, 20, 0, 0), layout=1), dict(S=0), dict(S=3),
                dict(M=1 << 31, S=1)):
        assert rope_fwd(L, rope(**bad), ld=1 << 20) == SHAPE, bad
    for bad in (dict(pos=P + 2), dict(freqs=P + 4), dict(w_q=P + 2), dict(pt=0, w_k=P + 1)):
        assert rope_fwd(L, rope(**bad)) == ALIGN, bad
    r = rope()
    assert rope_fwd(L, r, x=None) == ARG
    assert rope_fwd(L, r, q=heads(p=None)) == ARG
    assert rope_fwd(L, r, ld=504) == SHAPE
    assert rope_fwd(L, r, ld=516) == ALIGN
    assert rope_fwd(L, r, k=heads(p=P + 8)) == ALIGN
    assert rope_fwd(L, r, v=heads(st=260)) == ALIGN
    assert rope_fwd(L, rope(M=0, S=0)) == OK

    def back(r, dw=P, ws=P, nws=1 << 30, x=P, dx=P, ldd=512):
        return L.ft_qk_rope_bwd(ctypes.byref(r), ctypes.byref(h), ctypes.byref(h), ctypes.byref(h), x, 512, dx, ldd, dw,
                                dw, None, ws, nws, None)

    assert back(r, x=None) == ARG                 # the norm's gradient reads qkv
    assert back(r, dx=None) == ARG
    assert back(rope(norm=0, w_q=None, w_k=None)) == ARG  # a gradient of absent weights
    assert back(r, ldd=504) == SHAPE
    assert back(r, dx=P + 8) == ALIGN
    assert back(r, nws=L.ft_qk_rope_workspace_bytes(4, 64) - 1) == WORKSPACE
    assert back(r, ws=None) == WORKSPACE
    assert L.ft_qk_rope_workspace_bytes(-1, 64) == 0


def adam(**kw):
    d = dict(p=P, p16=P, grad=P, m=P, v=P, m_scale=P, v_scale=P, n=100, weight_decay=0.0, gt=1)
    d.update(kw)
    return FtAdamwTensor(**d)


def test_adamw_refusals(L):
    h = FtAdamwHyper(1e-3, 0.9, 0.999, 1e-8)

    def step(t, bits=32, hyper=h, steps=P, count=1, lr=None, gs=None):
        return L.ft_adamw_step(None if t is None else ctypes.addressof(t), count,
                               None if hyper is None else ctypes.byref(hyper), bits, steps, lr, gs, None)

    t = adam()
    assert step(None) == ARG
    assert step(t, count=-1) == ARG
    assert step(t, hyper=None) == ARG
    assert step(t, steps=None) == ARG
    assert step(t, bits=16) == ARG
    for bad in (FtAdamwHyper(1e-3, 1.0, 0.999, 1e-8), FtAdamwHyper(1e-3, 0.9, -0.1, 1e-8),
                FtAdamwHyper(1e-3, 0.9, 0.999, -1.0), FtAdamwHyper(float("nan"), 0.9, 0.999, 1e-8)):
        assert step(t, hyper=bad) == ARG
    for bad in (dict(p=None, p16=None), dict(grad=None), dict(m=None), dict(v=None), dict(n=-1), dict(gt=2)):
        assert step(adam(**bad)) == ARG, bad
    assert step(adam(m_scale=None), bits=8) == ARG
    assert step(adam(n=1 << 40)) == SHAPE
    for bad in (dict(p=P + 2), dict(p16=P + 1), dict(grad=P + 2), dict(m=P + 2), dict(v_scale=P + 1)):
        assert step(adam(**bad)) == ALIGN, bad
    assert step(t, steps=P + 4) == ALIGN
    assert step(t, lr=P + 2) == ALIGN
    assert step(t, gs=P + 1) == ALIGN
    assert L.ft_adamw_decode(None, P, 5, 0, P, None) == ARG
    assert L.ft_adamw_decode(P, P, 5, 2, P, None) == ARG
    assert L.ft_adamw_decode(P, P + 1, 5, 0, P, None) == ALIGN
    assert L.ft_adamw_decode(P, P, 0, 0, P, None) == OK


@pytest.mark.parametrize("pre,post", [(1, 0), (2, 0), (2, 1), (1, 2), (0, 1), (0, 0)])
def test_reference_gated_norm_gradient_matches_differences(pre, post):
    """The 64-bit formula's autograd along random directions against central
    differences; their own truncation error is read off by halving the step
    (the error falls fourfold, so it is below the change itself)."""
    g = torch.Generator().manual_seed(pre * 3 + post)
    M, D, B = 5, 24, 2
    sample = torch.tensor([0, 0, 1, 1, 1])
    rnd = lambda *s: torch.randn(*s, generator=g, dtype=torch.float64)  # noqa: E731
    leaves = dict(x=rnd(M, D), y=rnd(M, D), gate=rnd(B, D), w_post=rnd(D) if post else None,
                  scale=rnd(B, D) if pre else None, shift=rnd(B, D) if pre else None, w=rnd(D) if pre else None,
                  bias=rnd(D) if pre else None)
    cr, ch = rnd(M, D), rnd(M, D)

    def loss(**lv):
        r, h = R.gated_norm64(lv["x"], lv["y"], lv["gate"], lv["scale"], lv["shift"], lv["w"], lv["bias"], lv["w_post"],
                              pre, post, 0.7, 1e-6, sample)
        return (r * cr).sum() + (0 if h is None else (h * ch).sum())

    for name, v in leaves.items():
        if v is None:
            continue
        leaf = v.clone().requires_grad_()
        grad, = torch.autograd.grad(loss(**{**leaves, name: leaf}), leaf)
        d = rnd(*v.shape)
        num, err = R.differences(lambda t: loss(**{**leaves, name: t}), v, d, 1e-4)
        want = (grad * d).sum()
        # truncation below `err`; rounding 2^-53 |loss terms| / step < 1e-9
        assert abs(num - want) <= err + 1e-8 * (1 + abs(want)), name


def test_reference_gelu_slope_matches_differences():
    y = torch.linspace(-9, 9, 181, dtype=torch.float64)
    f = lambda t: t * 0.5 * torch.special.erfc(-t / 2 ** 0.5)  # noqa: E731
    num, err = R.differences(f, y, torch.ones_like(y), 1e-4)
    assert bool(((num - R.gelu_slope64(y)).abs() <= err + 1e-10).all())


def test_python_side_refuses_cpu_tensors():
    import bit_quantized_lora_b200 as ft
    x = torch.zeros(4, 64, dtype=torch.bfloat16)
    with pytest.raises(TypeError):
        ft.ft_gated_norm_fwd(ft.GatedNorm(), x)
    with pytest.raises(TypeError):
        ft.ft_gelu_bwd_bf16(x, x)
    with pytest.raises(TypeError):
        ft.AdamW([x])
    with pytest.raises(ValueError):
        ft.AdamW([])


class _Tensor:
    """Stands in for a CUDA tensor where only its bookkeeping is looked at."""
    is_cuda = True

    def __init__(self, at, n, dtype=torch.float32, device="cuda:0", contiguous=True):
        self.at, self.n, self.dtype, self.device, self.contiguous = at, n, dtype, device, contiguous
        self.nbytes = n * dtype.itemsize

    def data_ptr(self):
        return self.at

    def numel(self):
        return self.n

    def is_contiguous(self):
        return self.contiguous


def test_parameters_of_an_optimizer_are_apart_and_stay_what_they_were():
    from bit_quantized_lora_b200.optim import _check_params
    F, H = torch.float32, torch.bfloat16
    ok = [_Tensor(4096, 64), _Tensor(4096 + 256, 64, H), _Tensor(0, 0)]
    _check_params(ok, "cuda:0")
    _check_params(ok, "cuda:0", [F, H, F], [64, 64, 0])
    _check_params([_Tensor(9000, 64), _Tensor(0, 0), _Tensor(0, 0)], "cuda:0")  # empty ones lie nowhere
    for bad, text in (
            ([_Tensor(4096, 64), _Tensor(4096, 64)], "twice"),
            ([_Tensor(4096, 64), _Tensor(4096 + 252, 64)], "share"),
            ([_Tensor(8192, 64), _Tensor(8192 - 4, 2)], "share"),
            ([_Tensor(4096, 64, device="cuda:1")], "one device"),
            ([_Tensor(4096, 64, contiguous=False)], "contiguous")):
        with pytest.raises(ValueError, match=text):
            _check_params(bad, "cuda:0")
    with pytest.raises(TypeError):
        _check_params([_Tensor(4096, 64, torch.float16)], "cuda:0")
    for now in (_Tensor(4096, 63), _Tensor(0, 0), _Tensor(4096, 64, H)):
        with pytest.raises(ValueError, match="another type or size"):
            _check_params([now], "cuda:0", [F], [64])


def test_calls_by_position_and_by_name_refuse_alike():
    x, n = torch.zeros(2, 16, dtype=torch.bfloat16), ft.GatedNorm()
    rope = ft.Rope(heads=1, kv_heads=0, head_dim=16, axes=(16,), freqs=torch.zeros(8, dtype=torch.float64))
    pos = torch.zeros(2, dtype=torch.int32)
    for call in (lambda: ft.ft_gated_norm_fwd(n, x), lambda: ft.ft_gated_norm_fwd(norm=n, x=x),
                 lambda: ft.ft_gated_norm_fwd(n), lambda: ft.ft_gated_norm_fwd(n, None),
                 lambda: ft.ft_gated_norm_bwd(norm=n, dh=x, r=x, stats=x),
                 lambda: ft.ft_gelu_bwd_bf16(x, x), lambda: ft.ft_gelu_bwd_bf16(y=x, dh=x),
                 lambda: ft.ft_qk_rope_fwd(rope, x, pos), lambda: ft.ft_qk_rope_fwd(rope=rope, qkv=x, pos=pos),
                 lambda: ft.ft_adamw_decode(x, x), lambda: ft.ft_adamw_decode(codes=x, scales=x)):
        with pytest.raises(TypeError, match="CUDA"):
            call()


def test_the_layout_of_an_optimizers_tensors():
    """What a step compares with the step before: memory, type, sizes and
    strides of every tensor, in order."""
    layout = _lib.load_torch().layout_of
    a, b = torch.zeros(16, 16), torch.zeros(64, dtype=torch.bfloat16)
    key = layout([a, b])
    assert key == layout((a, b)) == layout([a.view(16, 16), b.detach()])
    for other in ([b, a], [a], [a.t(), b], [a.view(8, 32), b], [a.clone(), b], [a[:8], b], [a.view(torch.int32), b],
                  [a, b.view(torch.float16)], [a, b.view(torch.int8)], [a, b[1:]], [a, b[::2]], [a, b, b], []):
        assert layout(other) != key
    assert layout([]) == layout(())
    assert layout([torch.zeros(0)]) == layout([torch.zeros(0)]) != layout([torch.zeros(0, dtype=torch.int32)])
    for bad in ([None], [a, 3]):
        with pytest.raises(TypeError):
            layout(bad)
