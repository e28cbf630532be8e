"""A DiT block's training step: the gated norms, the rotation, GELU's backward
and the triple-branch linears in one forward and backward, and the AdamW step
of the adapters behind it.

Against 64 bits (autograd of the whole block) with 16-bit activations and
gradients, where the linears' weights are exactly Q(W_res) + V U^T + s B A^T.
Each tensor that a kernel hands on is rounded to bf16 once, a relative error
of at most 2^-8 of its norm; a path through the block passes 12 such tensors
forward (h1, P, y, q or v, o, P, y, h2, P, y, h, P, y) and as many again
backward, and to first order the errors add: 13 * 2^-8 = 5.1 % forward, 26 *
2^-8 = 10.2 % backward at the very most, were they all at half a step and all
aligned.  Rounding errors are neither: their root mean square is 2^-8 / sqrt 3
of half-step bounds over a binade less, and independent ones add as squares,
so sqrt(26) 2^-8 / sqrt 3 = 1.2 %; the limits below are twice that, 2.5 %.
"""
import pytest
import torch

import bit_quantized_lora_b200 as ft
from bit_quantized_lora_b200.stack import LinearStack
from block_ref import gelu_slope64  # noqa: F401  (the reference's GELU is torch's, checked against its slope)

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16
FWD, BWD = 0.025, 0.025


class Softmax:
    """Plain attention in FP32 for the tests."""

    def forward(self, q, k, v):
        saved = [t.float().requires_grad_() for t in (q, k, v)]
        with torch.enable_grad():
            k2, v2 = (t.repeat_interleave(q.shape[1] // t.shape[1], 1) for t in saved[1:])
            o = torch.softmax(saved[0] @ k2.transpose(-1, -2) / q.shape[-1] ** 0.5, -1) @ v2
        return o.detach().to(BF16), (saved, o)

    def backward(self, do, saved):
        leaves, o = saved
        return [g.to(BF16) for g in torch.autograd.grad(o, leaves, do.float(), retain_graph=True)]


def layer(g, N, K, precision, r=16):
    rnd = lambda *s, std: (torch.randn(*s, generator=g, device="cuda") * std).to(BF16)  # noqa: E731
    return ft.prepare_layer(W_res=rnd(N, K, std=K ** -0.5), U=rnd(K, r, std=0.1), V=rnd(N, r, std=0.1),
                            A=rnd(K, r, std=0.1), B=rnd(N, r, std=0.1), s=0.5, precision=precision)


def make(seed=0, precision="W4A16G16", D=256, F=512, heads=4, kv=4, hd=64, axes=(16, 24, 24), B=2, S=48, xt=BF16,
         norm=ft.NORM_LAYER):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    rnd = lambda *s, std=1.0, mean=0.0: torch.randn(*s, generator=g, device="cuda") * std + mean  # noqa: E731
    rope = ft.Rope(heads, kv, hd, axes, ft.rope_freqs(axes), norm=True, w_q=rnd(hd, std=0.1, mean=1.0),
                   w_k=rnd(hd, std=0.1, mean=1.0))
    blk = ft.DitBlock(layer(g, rope.width, D, precision), layer(g, D, heads * hd, precision),
                      layer(g, F, D, precision), layer(g, D, F, precision), rope, norm=norm)
    x = rnd(B * S, D).to(xt)
    mod = rnd(B, 6, D, std=0.5)
    pos = torch.randint(0, 40, (B * S, len(axes)), generator=g, device="cuda", dtype=torch.int32)
    dx2 = rnd(B * S, D, std=0.1).to(xt)
    return blk, x, mod, pos, dx2


def weight64(L):
    """Q(W_res) + V U^T, with the adapter's factors as leaves."""
    w = L.wd_k.double() * L.w_k.tscale.double() + L.V.double() @ L.U.double().T
    A, B = L.A.double().requires_grad_(), L.B.double().requires_grad_()
    return w + L.s * B @ A.T, A, B


def reference(blk, x, mod, pos, dx2):
    """x' and all gradients of the block in 64 bits."""
    rope, (M, D) = blk.rope, x.shape
    B, H, K, hd = len(mod), rope.heads, rope.kv_heads, rope.head_dim
    x, mod = x.double().requires_grad_(), mod.double().requires_grad_()
    wq, wk = rope.w_q.double().requires_grad_(), rope.w_k.double().requires_grad_()
    W, As, Bs = zip(*(weight64(L) for L in blk.layers))
    rows = torch.arange(M, device="cuda") * B // M

    def norm(t):
        t = t - t.mean(1, keepdim=True) if blk.norm.pre == ft.NORM_LAYER else t
        return t / (t.square().mean(1, keepdim=True) + blk.norm.eps).sqrt()

    m = mod[rows]
    which = sum(([a] * (w // 2) for a, w in enumerate(rope.axes)), [])
    ang = (pos.double()[:, which] * rope.freqs)[:, None]

    def heads(t, n, w):
        t = t.view(M, n, hd)
        if w is not None:
            t = t / (t.square().mean(-1, keepdim=True) + rope.eps).sqrt() * w
            a, b = t[..., 0::2], t[..., 1::2]
            t = torch.stack([a * ang.cos() - b * ang.sin(), b * ang.cos() + a * ang.sin()], -1).flatten(-2)
        return t.view(B, M // B, n, hd).transpose(1, 2)

    qkv = (norm(x) * (1 + m[:, 1]) + m[:, 0]) @ W[0].T
    q, k, v = heads(qkv[:, :H * hd], H, wq), heads(qkv[:, H * hd:(H + K) * hd], K, wk), \
        heads(qkv[:, (H + K) * hd:], K, None)
    k, v = (t.repeat_interleave(H // K, 1) for t in (k, v))
    o = torch.softmax(q @ k.transpose(-1, -2) / hd ** 0.5, -1) @ v
    r = x + m[:, 2] * (o.transpose(1, 2).reshape(M, -1) @ W[1].T)
    h = torch.nn.functional.gelu((norm(r) * (1 + m[:, 4]) + m[:, 3]) @ W[2].T)
    x2 = r + m[:, 5] * (h @ W[3].T)
    names = [x, mod, wq, wk, *As, *Bs]
    return x2.detach(), torch.autograd.grad(x2, names, dx2.double())


def off(got, want):
    return float((got.double() - want).norm() / want.norm())


@pytest.mark.parametrize("kw", [dict(), dict(xt=torch.float32, B=3, S=25, norm=ft.NORM_RMS),
                                dict(heads=8, kv=4, hd=32, axes=(8, 12, 12), B=1, S=70, seed=4)], ids=str)
def test_block_against_64_bits(kw):
    blk, x, mod, pos, dx2 = make(**kw)
    attn = Softmax()
    x2, saved = blk.forward(x, mod, pos, attn)
    g = blk.backward(dx2, saved, attn)
    torch.cuda.synchronize()
    assert ft.ft_device_error() == 0
    want, (dx, dmod, dwq, dwk, *ab) = reference(blk, x, mod, pos, dx2)
    # the block's own contribution, the residual taken off
    assert off(x2.double() - x.double(), want - x.double()) <= FWD
    assert off(g.dx, dx) <= BWD
    for i in range(6):
        assert off(g.dmod[:, i], dmod[:, i]) <= BWD, i
    assert off(g.dw_q, dwq) <= BWD and off(g.dw_k, dwk) <= BWD
    for i, (dA, dB) in enumerate(g.adapters):
        assert off(dA, ab[i]) <= BWD and off(dB, ab[4 + i]) <= BWD, i


def test_the_norms_amax_is_the_linears():
    """4-bit activations and gradients: the linears that get their tensor amax
    from the kernel before them give the bits of those that look for it."""
    blk, x, mod, pos, dx2 = make(precision="W4A4G4", seed=2)
    attn = Softmax()
    x2, saved = blk.forward(x, mod, pos, attn)
    h1, y_qkv, h2, y_up = saved[3], saved[5], saved[12], saved[14]
    assert torch.equal(ft.ft_linear_fwd(blk.qkv, h1)[0], y_qkv)
    assert torch.equal(ft.ft_linear_fwd(blk.up, h2)[0], y_up)
    g = blk.backward(dx2, saved, attn)
    # the down layer's gradients from a gate's backward of our own
    gate = ft.ft_gated_norm_bwd(ft.GatedNorm(pre=ft.NORM_NONE), None, None, None, dr=dx2, y=saved[18],
                                gate=mod[:, 5], need_dx=False)
    _, dA, dB = ft.ft_linear_bwd(blk.down, gate.dy, saved[16], saved[17])
    assert torch.equal(dA, g.adapters[3][0]) and torch.equal(dB, g.adapters[3][1])
    # again, the same bits
    x3, saved = blk.forward(x, mod, pos, attn)
    g3 = blk.backward(dx2, saved, attn)
    assert torch.equal(x2, x3) and torch.equal(g.dx, g3.dx) and torch.equal(g.dmod, g3.dmod)
    assert torch.isfinite(g.dx).all() and torch.isfinite(g.dmod).all()


def test_a_block_of_zeros():
    """No activation at all: every amax is zero, every output the residual."""
    blk, x, mod, pos, dx2 = make(precision="W4A4G4")
    x.zero_(), mod.zero_()
    attn = Softmax()
    x2, saved = blk.forward(x, mod, pos, attn)
    g = blk.backward(dx2, saved, attn)
    torch.cuda.synchronize()
    assert not x2.any() and torch.equal(g.dx, dx2)
    for dA, dB in g.adapters:
        assert not dA.any() and not dB.any()


@pytest.mark.parametrize("bits", [32, 8])
def test_training_steps(bits):
    """Three steps of a block's adapters: they move, by at most the rate times
    Adam's largest step (1 + weight decay's share), and stay finite."""
    blk, x, mod, pos, dx2 = make(precision="W4A4G4", seed=3)
    attn = Softmax()
    params = [p for L in blk.layers for p in (L.A, L.B)]
    before = [p.clone() for p in params]
    opt = ft.AdamW(params, lr=2.0 ** -8, state_bits=bits, weight_decay=0.0)
    for _ in range(3):
        x2, saved = blk.forward(x, mod, pos, attn)
        g = blk.backward(dx2, saved, attn)
        opt.step([t for pair in g.adapters for t in pair])
    torch.cuda.synchronize()
    assert int(opt.step_count) == 3
    for p, b in zip(params, before):
        moved = (p.float() - b.float()).abs()
        assert torch.isfinite(p).all() and bool(moved.any())
        # |m| / sqrt(v) <= sqrt(t) after bias correction; a bf16 rounding each end
        assert bool((moved <= 3 * 3 ** 0.5 * 2.0 ** -8 * 1.01 + b.float().abs() * 2.0 ** -7).all())


def test_stack_optimizer_steps_the_adapters():
    """The stack's step with its optimizer is the step, then AdamW on the
    gradients that it leaves."""
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    layers = [layer(g, 512, 256, "W4A4G4"), layer(g, 256, 512, "W4A4G4")]
    Xs = [torch.randn(64, L.K, generator=g, device="cuda").to(BF16) for L in layers]
    dYs = [torch.randn(64, L.N, generator=g, device="cuda").to(BF16) for L in layers]
    st = LinearStack(layers, 64, "cuda")
    st.step(Xs, dYs)
    copies = [p.clone() for L in layers for p in (L.A, L.B)]
    grads = [t.clone() for b in st.bufs for t in (b.dA, b.dB)]
    half = torch.full((1,), 0.5, device="cuda")
    ref = ft.AdamW(copies, grads, lr=1e-2, state_bits=8)
    opt = st.optimizer(lr=1e-2, state_bits=8)
    for _ in range(2):
        st.step(Xs, dYs, optimizer=opt, grad_scale=half)
        for t, r in zip([t for b in st.bufs for t in (b.dA, b.dB)], grads):
            r.copy_(t)
        ref.step(grad_scale=half)
        assert all(torch.equal(a, b) for a, b in zip([p for L in layers for p in (L.A, L.B)], copies))


def test_refusals():
    blk, x, mod, pos, dx2 = make()
    with pytest.raises(ValueError):
        ft.DitBlock(blk.out, blk.qkv, blk.up, blk.down, blk.rope)
    with pytest.raises(ValueError):
        ft.DitBlock(blk.qkv, blk.out, blk.down, blk.up, blk.rope)
    with pytest.raises(ValueError):
        blk.forward(x, mod[:, :5], pos, Softmax())
    with pytest.raises(ValueError):
        blk.forward(x[:-1], mod, pos[:-1], Softmax())
