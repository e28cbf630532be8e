"""Rotary positions with several axes against the formula in 64 bits.

Tolerances.  The angle is reduced in FP64 (p f below 2^31 turns: 2^-53 2^31 =
2^-22 of a turn at the very far end, 2^-53 p f / 2 pi in general), passed on
in FP32 (2^-25 of half a turn) and its sine and cosine are good to 2 ulp: the
rotated value is off by less than 8 roundings of 2^-24 of |a| + |b|, plus the
far angle's share.  The head's sum of squares adds eight values in a lane and
five shuffles; with the steps around it 32 roundings bound the norm.
"""
import math

import pytest
import torch

import bit_quantized_lora_b200 as ft
import block_ref as R

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32


class Case:
    def __init__(self, B=1, S=5, Hq=4, Hk=2, hd=64, axes=(16, 24, 24), halves=False, norm=True, far=100, pos32=True,
                 pt=F32, seed=0, pad=0, weights=True):
        g = torch.Generator(device="cuda")
        g.manual_seed(seed)
        rnd = lambda *s, std=1.0, mean=0.0: torch.randn(*s, generator=g, device="cuda") * std + mean  # noqa: E731
        self.B, self.S, self.M, self.Hq, self.Hk, self.hd, self.halves = B, S, B * S, Hq, Hk, hd, halves
        self.width = (Hq + 2 * Hk) * hd
        self.qkv = rnd(self.M, self.width + pad, std=1.5).to(BF16)[:, :self.width]
        pos = torch.randint(-far, far, (self.M, len(axes)), generator=g, device="cuda")
        self.pos = pos.to(torch.int32) if pos32 else pos.to(F32) * 0.37
        self.rope = ft.Rope(Hq, Hk, hd, tuple(axes), ft.rope_freqs(axes), ft.ROPE_HALVES if halves else ft.ROPE_PAIRS,
                            norm, rnd(hd, std=0.3, mean=1.0).to(pt) if norm and weights else None,
                            rnd(hd, std=0.3, mean=1.0).to(pt) if norm and weights else None)
        self.d = {n: rnd(B, H, S, hd, std=0.01).to(BF16) for n, H in (("q", Hq), ("k", Hk), ("v", Hk))}
        rot, which = sum(axes), []
        for a, w in enumerate(axes):
            which += [a] * (w // 2)
        self.ang = self.pos.double()[:, which] * self.rope.freqs
        # roundings of the rotation, the far angle's among them
        self.turn = 8 * R.U32 + (2 * math.pi * 2.0 ** -52 * self.ang.abs().max().item() if self.ang.numel() else 0.0)

    def parts(self):
        x = self.qkv.double().reshape(self.M, -1, self.hd)
        return x[:, :self.Hq], x[:, self.Hq:self.Hq + self.Hk], x[:, self.Hq + self.Hk:]

    def rows(self, t):
        """[B, H, S, hd] -> [M, H, hd]"""
        return t.transpose(1, 2).reshape(self.M, -1, self.hd)

    def partner(self, x):
        """|a| + |b| of each value's pair, the value itself where it is not rotated."""
        rot = sum(self.rope.axes)
        ones = torch.full_like(self.ang, math.pi / 4)
        return R.rope64(x.abs(), ones, rot, self.halves).abs() * 2 + x.abs() * 2

    def check_forward(self, q, k, v):
        rot = sum(self.rope.axes)
        xq, xk, xv = self.parts()
        for got, x, w in ((q, xq, self.rope.w_q), (k, xk, self.rope.w_k)):
            slack = self.turn
            if self.rope.norm:
                x = x / (x.square().mean(-1, keepdim=True) + self.rope.eps).sqrt()
                x = x if w is None else x * w.double()
                slack = slack + 32 * R.U32
            a = x.abs()
            pair = torch.maximum(a, self.partner(x))
            R.check_rounded(self.rows(got), R.rope64(x, self.ang, rot, self.halves), 2 * slack * pair)
        assert torch.equal(self.rows(v), xv.to(BF16))

    def check_backward(self, dqkv, dw_q, dw_k, amax=None):
        rot = sum(self.rope.axes)
        got = dqkv.reshape(self.M, -1, self.hd)
        cut = [0, self.Hq, self.Hq + self.Hk]
        for i, (n, x, w, dw) in enumerate(zip("qk", self.parts(), (self.rope.w_q, self.rope.w_k), (dw_q, dw_k))):
            x = x.contiguous().requires_grad_()
            wl = torch.ones(self.hd, dtype=torch.float64, device="cuda") if w is None else w.double()
            wl = wl.clone().requires_grad_()
            z = x
            if self.rope.norm:
                z = x / (x.square().mean(-1, keepdim=True) + self.rope.eps).sqrt() * wl
            z = R.rope64(z, self.ang, rot, self.halves)
            d = self.rows(self.d[n]).double()
            want = torch.autograd.grad(z, (x, wl) if self.rope.norm else (x,), d)
            size = torch.maximum(d.abs(), self.partner(d))
            slack = 2 * self.turn * size
            if self.rope.norm:
                xd = x.detach()
                rstd = 1 / (xd.square().mean(-1, keepdim=True) + self.rope.eps).sqrt()
                e, xh = size * wl.detach().abs(), xd.abs() * rstd
                slack = (2 * self.turn + 64 * R.U32) * rstd * (e + xh * (e * xh).mean(-1, keepdim=True))
                if dw is not None:
                    # heads of a group in turn, groups, blocks: under 300 additions at these sizes, or 4 rows' heads
                    # a turn times the turns of a block
                    adds = 300 + self.M * (self.Hq + self.Hk) // 1000
                    R.check_rounded(dw, want[1], (2 * self.turn + (64 + adds) * R.U32) * (size * xh).sum((0, 1)))
            R.check_rounded(got[:, cut[i]:cut[i] + x.shape[1]], want[0], slack)
        assert torch.equal(got[:, cut[2]:], self.rows(self.d["v"]))
        if amax is not None:
            assert float(amax) == float(dqkv.float().abs().max())


CASES = [
    dict(S=1, Hq=1, Hk=1, hd=8, axes=(8,)),
    dict(S=1, Hq=24, Hk=24, hd=128, axes=(16, 56, 56)),
    dict(S=7, Hq=3, Hk=1, hd=40, axes=(6, 10, 14)),
    dict(S=7, Hq=4, Hk=2, hd=80, axes=(16, 24), halves=True),
    dict(S=33, Hq=4, Hk=4, hd=64, axes=(64,), halves=True),
    dict(S=33, Hq=5, Hk=5, hd=96, axes=(24, 40), norm=False),
    dict(S=12, B=3, Hq=6, Hk=3, hd=128, axes=(32, 48, 48), halves=True, pt=BF16),
    dict(S=9, B=2, Hq=2, Hk=1, hd=256, axes=(2, 84, 84, 86)),
    dict(S=9, B=2, Hq=2, Hk=1, hd=256, axes=(256,), halves=True, norm=False),
    dict(S=300, Hq=8, Hk=2, hd=64, axes=(16, 24, 24), far=1 << 20),
    dict(S=300, Hq=8, Hk=2, hd=64, axes=(16, 24, 24), far=2_000_000_000),
    dict(S=50, Hq=2, Hk=2, hd=32, axes=(8, 8), pos32=False),
    dict(S=1400, Hq=3, Hk=3, hd=192, axes=(64, 64, 64)),
    dict(S=20, Hq=4, Hk=0, hd=64, axes=(32, 32), weights=False),
    dict(S=20, Hq=2, Hk=2, hd=64, axes=(0, 32)),
    dict(S=4, Hq=70, Hk=70, hd=128, axes=(128,)),
    dict(S=2500, B=2, Hq=3, Hk=1, hd=64, axes=(32, 32)),             # more rows than the device holds warps
    dict(S=9500, Hq=2, Hk=1, hd=40, axes=(16, 24), halves=True),
]


@pytest.mark.parametrize("kw", CASES, ids=lambda k: "-".join(f"{a}{v}" for a, v in k.items()))
@pytest.mark.parametrize("head_major", [True, False])
def test_against_the_formula(kw, head_major):
    c = Case(seed=len(str(kw)), **kw)
    q, k, v = ft.ft_qk_rope_fwd(c.rope, c.qkv, c.pos, tokens=c.S, head_major=head_major)
    assert q.shape == (c.B, c.Hq, c.S, c.hd) and v.shape == (c.B, c.Hk, c.S, c.hd)
    c.check_forward(q, k, v)
    if not head_major:
        c.d = {n: t.transpose(1, 2).contiguous().transpose(1, 2) for n, t in c.d.items()}
    amax = torch.zeros(1, device="cuda")
    dqkv, dw_q, dw_k = ft.ft_qk_rope_bwd(c.rope, c.d["q"], c.d["k"], c.d["v"], c.pos, qkv=c.qkv, amax=amax)
    assert (dw_q is not None) == (c.rope.w_q is not None)
    c.check_backward(dqkv, dw_q, dw_k, amax)


def test_strides_and_in_place():
    c = Case(B=2, S=13, Hq=4, Hk=2, hd=64, pad=24)
    want = [t.clone() for t in ft.ft_qk_rope_fwd(c.rope, c.qkv, c.pos, tokens=c.S)]
    c.check_forward(*want)
    # v as it lies
    _, _, v = ft.ft_qk_rope_fwd(c.rope, c.qkv, c.pos, tokens=c.S, copy_v=False)
    assert torch.equal(v, want[2]) and v.data_ptr() == c.qkv[:, 6 * 64:].data_ptr()
    # the gradient of v may be a broadcast, and dqkv a part of a wider buffer
    c.d["v"] = c.d["v"][:, :, :1].expand(-1, -1, c.S, -1)
    wide = torch.full((c.M, c.width + 8), 5.0, dtype=BF16, device="cuda")
    dqkv, a, b = ft.ft_qk_rope_bwd(c.rope, c.d["q"], c.d["k"], c.d["v"], c.pos, qkv=c.qkv, dqkv=wide[:, :c.width])
    c.check_backward(dqkv, a, b)
    assert bool((wide[:, c.width:] == 5.0).all())
    left = torch.full((c.M, c.width), 3.0, dtype=BF16, device="cuda")
    ft.ft_qk_rope_bwd(c.rope, c.d["q"], c.d["k"], None, c.pos, qkv=c.qkv, dqkv=left, weight_grads=False)
    assert torch.equal(left[:, :6 * 64], dqkv[:, :6 * 64]) and bool((left[:, 6 * 64:] == 3.0).all())
    # in place: q and k over their own columns
    x = c.qkv.clone()
    parts = x.view(c.B, c.S, -1, c.hd).transpose(1, 2)
    q, k, _ = ft.ft_qk_rope_fwd(c.rope, x, c.pos, tokens=c.S, q=parts[:, :4], k=parts[:, 4:6], copy_v=False)
    assert torch.equal(q, want[0]) and torch.equal(k, want[1])
    assert torch.equal(x[:, 6 * 64:], c.qkv[:, 6 * 64:])


@pytest.mark.parametrize("norm", [True, False])
def test_backward_in_place(norm):
    """dq, dk and dv are the columns that dqkv is written to."""
    c = Case(B=2, S=37, Hq=6, Hk=2, hd=64, norm=norm)
    want, a, b = ft.ft_qk_rope_bwd(c.rope, c.d["q"], c.d["k"], c.d["v"], c.pos, qkv=c.qkv)
    buf = torch.cat([c.rows(c.d[n]) for n in "qkv"], 1).reshape(c.M, c.width).contiguous()
    parts = buf.view(c.B, c.S, -1, c.hd).transpose(1, 2)
    got, a2, b2 = ft.ft_qk_rope_bwd(c.rope, parts[:, :6], parts[:, 6:8], parts[:, 8:], c.pos, qkv=c.qkv, dqkv=buf)
    assert got.data_ptr() == buf.data_ptr() and torch.equal(buf, want)
    if norm:
        assert torch.equal(a, a2) and torch.equal(b, b2)


def test_shared_frequencies_and_no_rows():
    axes = (8, 12, 12)
    f = ft.rope_freqs(axes, 500.0, shared=True)
    assert torch.allclose(f, 500.0 ** (-torch.arange(16, dtype=torch.float64, device="cuda") / 16), rtol=1e-14)
    c = Case(S=0, Hq=2, Hk=2, hd=32, axes=axes)
    q, k, v = ft.ft_qk_rope_fwd(c.rope, c.qkv, c.pos)
    assert q.numel() == 0
    dqkv, dw_q, dw_k = ft.ft_qk_rope_bwd(c.rope, torch.zeros(1, 2, 0, 32, dtype=BF16, device="cuda"),
                                         torch.zeros(1, 2, 0, 32, dtype=BF16, device="cuda"), None, c.pos, qkv=c.qkv)
    assert not dw_q.any() and not dw_k.any()


def test_non_finite_heads_stay_apart():
    c = Case(S=3, Hq=2, Hk=1, hd=64)
    q0, k0, _ = ft.ft_qk_rope_fwd(c.rope, c.qkv, c.pos)
    c.qkv[1, 5] = float("nan")
    q, k, _ = ft.ft_qk_rope_fwd(c.rope, c.qkv, c.pos)
    assert bool(q[0, 0, 1].isnan().all())
    q0[0, 0, 1] = q[0, 0, 1] = 0
    assert torch.equal(q, q0) and torch.equal(k, k0)
    c.qkv[:] = 0  # a head of zeros: eps alone
    q, _, _ = ft.ft_qk_rope_fwd(c.rope, c.qkv, c.pos)
    assert not q.any()


def test_repeats_streams_and_graphs():
    cs = [Case(S=777, Hq=8, Hk=8, hd=128, axes=(16, 56, 56), seed=s) for s in (1, 2)]

    def both(c):
        return [*ft.ft_qk_rope_fwd(c.rope, c.qkv, c.pos),
                *ft.ft_qk_rope_bwd(c.rope, c.d["q"], c.d["k"], c.d["v"], c.pos, qkv=c.qkv)]

    want = [both(c) for c in cs]
    same = lambda x, y: all(torch.equal(a, b) for a, b in zip(x, y))  # noqa: E731
    assert same(both(cs[0]), want[0])
    streams, got = [torch.cuda.Stream(), torch.cuda.Stream()], [None, None]
    for _ in range(3):
        for i, s in enumerate(streams):
            s.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(s):
                got[i] = both(cs[i])
    torch.cuda.synchronize()
    assert same(got[0], want[0]) and same(got[1], want[1])
    graphs = []
    for c in cs:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = both(c)
        graphs.append((g, out))
    for i in (0, 1, 0):
        graphs[i][0].replay()
        torch.cuda.synchronize()
        assert same(graphs[i][1], want[i])


def test_refusals():
    c = Case()
    with pytest.raises(TypeError):
        ft.ft_qk_rope_fwd(c.rope, c.qkv.float(), c.pos)
    with pytest.raises(TypeError):
        ft.ft_qk_rope_fwd(c.rope, c.qkv, c.pos.long())
    with pytest.raises(ValueError):
        ft.ft_qk_rope_fwd(c.rope, c.qkv, c.pos[:, :2])
    with pytest.raises(ValueError):
        ft.ft_qk_rope_fwd(c.rope, c.qkv, c.pos, tokens=3)
    with pytest.raises(ValueError):
        ft.ft_qk_rope_fwd(c.rope, c.qkv, c.pos, q=torch.zeros(1, 1, 5, 64, dtype=BF16, device="cuda").expand(1, 4, 5, 64))
    with pytest.raises(ValueError):
        ft.ft_qk_rope_bwd(c.rope, c.d["q"], c.d["k"], c.d["v"], c.pos)
    with pytest.raises(ValueError):
        ft.ft_qk_rope_bwd(c.rope, c.d["q"], c.d["k"][:, :1], c.d["v"], c.pos, qkv=c.qkv)
    with pytest.raises(ft.FtError):  # head strides that are not multiples of eight
        q = torch.zeros(1, 4, 5, 68, dtype=BF16, device="cuda")[..., :64]
        ft.ft_qk_rope_fwd(c.rope, c.qkv, c.pos, q=q)


def test_amax_without_the_gradient_of_v():
    """Without dv the amax is that of the columns written: what lies in the
    value columns, a gradient already there or not yet, does not count."""
    c = Case(B=2, S=13, Hq=4, Hk=2, hd=64)
    cut = 6 * 64
    for fill in (100.0, float("nan")):
        left = torch.full((c.M, c.width), fill, dtype=BF16, device="cuda")
        amax = torch.zeros(1, device="cuda")
        ft.ft_qk_rope_bwd(c.rope, c.d["q"], c.d["k"], None, c.pos, qkv=c.qkv, dqkv=left, amax=amax)
        assert 0.0 < float(amax) == float(left[:, :cut].float().abs().max()) < 1.0
    amax = torch.zeros(1, device="cuda")  # value columns that the call makes are zero: the amax is all of dqkv's
    dqkv, _, _ = ft.ft_qk_rope_bwd(c.rope, c.d["q"], c.d["k"], None, c.pos, qkv=c.qkv, amax=amax)
    assert float(amax) == float(dqkv.float().abs().max())


# Rows of the last round, more than half as many as the device holds warps (2960 backward with the norm, 4736
# otherwise), cut into three slices of its turns of heads in one direction or both, with whole rows before them or not.
SLICED = [
    dict(S=2841, Hq=16, Hk=8, hd=32, axes=(8, 12, 12)),
    dict(S=1700, Hq=16, Hk=8, hd=32, axes=(8, 12, 12)),
    dict(S=4660, Hq=10, Hk=2, hd=40, axes=(16, 24), halves=True),
    dict(S=2841, Hq=10, Hk=2, hd=40, axes=(16, 24), halves=True, norm=False),
    dict(S=7577, Hq=7, Hk=7, hd=64, axes=(16, 24, 24), norm=False),
    dict(S=4608, Hq=24, Hk=24, hd=128, axes=(16, 56, 56)),
]


@pytest.mark.parametrize("kw", SLICED, ids=lambda k: "-".join(f"{a}{v}" for a, v in k.items()))
def test_rows_cut_into_slices(kw):
    c = Case(seed=5, **kw)
    c.check_forward(*ft.ft_qk_rope_fwd(c.rope, c.qkv, c.pos))
    amax = torch.zeros(1, device="cuda")
    c.check_backward(*ft.ft_qk_rope_bwd(c.rope, c.d["q"], c.d["k"], c.d["v"], c.pos, qkv=c.qkv, amax=amax), amax)
