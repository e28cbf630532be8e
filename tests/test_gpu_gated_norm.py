"""The gated norm on the GPU against its formula in 64 bits.

Tolerances.  Every output is the 64-bit value with the FP32 steps' error
(`slack`), rounded once to its type.  A row's sums add at most 16 values in a
thread, 5 shuffles and 16 warps: under 40 roundings, each 2^-24 of the sum of
magnitudes; the few steps before and behind bring less than 60 more, so every
slack below is C = 128 roundings of the largest magnitudes that meet in the
value.  A column's sum over the rows adds at most `chunk` rows in a thread,
then a sixteenth of the chunks and 16 groups: `col_roundings` below, each
2^-24 of the sum of magnitudes, on top of each term's own error.
"""
import pytest
import torch

import bit_quantized_lora_b200 as ft
import block_ref as R

pytestmark = pytest.mark.gpu

C = 128 * R.U32
BF16, F32 = torch.bfloat16, torch.float32


class Case:
    """Inputs of one boundary, and the 64-bit view of them."""

    def __init__(self, M, D, B=1, pre=2, post=0, res=True, mod=True, weights=False, xt=BF16, pt=F32, offsets=None,
                 seed=0, alpha=0.75, pad=0, mean=0.0):
        g = torch.Generator(device="cuda")
        g.manual_seed(seed)
        rnd = lambda *s, std=1.0, mean=0.0: torch.randn(*s, generator=g, device="cuda") * std + mean  # noqa: E731
        self.M, self.D, self.B, self.pre, self.post, self.alpha, self.eps = M, D, B, pre, post, alpha, 1e-6

        def matrix(dtype, **kw):
            return rnd(M, D + pad, **kw).to(dtype)[:, :D]

        self.x = matrix(xt, mean=mean)
        self.y = matrix(BF16, std=0.7, mean=0.1) if res else None
        self.dh = matrix(BF16, std=0.01) if pre else None
        self.dr = matrix(xt, std=0.02)
        m = rnd(B, 3 * D, std=0.5).to(pt)
        self.gate = m[:, :D] if mod and res else None
        self.scale, self.shift = (m[:, D:2 * D], m[:, 2 * D:]) if mod and pre else (None, None)
        self.w = rnd(D, std=0.3, mean=1.0).to(pt) if weights and pre else None
        self.bias = rnd(D, std=0.3).to(pt) if weights and pre else None
        self.w_post = rnd(D, std=0.3, mean=1.0).to(pt) if weights and post else None
        self.offsets = None if offsets is None else torch.tensor(offsets, dtype=torch.int32, device="cuda")
        ends = [M * (b + 1) // B for b in range(B)] if offsets is None else offsets[1:]
        self.last = ends[-1]
        self.sample = torch.searchsorted(torch.tensor(ends, device="cuda"),
                                         torch.arange(self.last, device="cuda"), right=True)
        self.norm = ft.GatedNorm(pre=pre, post=post, alpha=alpha, eps=self.eps, weight=self.w, bias=self.bias,
                                 w_post=self.w_post)

    def forward(self, **kw):
        return ft.ft_gated_norm_fwd(self.norm, self.x, self.y, self.gate, self.scale, self.shift, offsets=self.offsets,
                                    **kw)

    def backward(self, r, stats, **kw):
        return ft.ft_gated_norm_bwd(self.norm, self.dh, r if self.pre else None, stats, dr=self.dr, y=self.y,
                                    gate=self.gate, scale=self.scale, shift=self.shift, offsets=self.offsets,
                                    residual=self.y is not None, **kw)

    def d(self, t, rows=True):
        return None if t is None else t.double()[:self.last] if rows else t.double()


def mag(v):
    return 0.0 if v is None else v.abs()


def check_forward(c, r, h, stats, amax):
    n = c.last
    x, y = c.d(c.x), c.d(c.y)
    gate, scale, shift = (R.rows_of(c.d(t, False), c.sample) for t in (c.gate, c.scale, c.shift))
    wp = 1.0 if c.w_post is None else c.w_post.double()
    if y is not None:
        want, _ = R.gated_norm64(x, y, c.d(c.gate, False), None, None, None, None, c.d(c.w_post, False), 0, c.post,
                                 c.alpha, c.eps, c.sample)
        _, my, ry = R.norm64(y, c.post, c.eps)
        u = ((y.abs() + my.abs() + y.abs().mean(1, keepdim=True)) * ry if c.post else y.abs()) * mag(torch.as_tensor(wp))
        R.check_rounded(r[:n], want, C * (x.abs() + c.alpha * u * (1.0 if gate is None else gate.abs())))
        if stats is not None:
            # the mean's error is of the magnitudes, 1/deviation's of itself and of the mean's share
            avg = y.abs().mean(1)
            assert bool(((stats[:n, 2].double() - my[:, 0]).abs() <= C * avg).all())
            assert bool(((stats[:n, 3].double() - ry[:, 0]).abs() <= C * ry[:, 0] * (1 + avg * ry[:, 0])).all())
    rs = r.double()[:n]
    if c.pre:
        _, want = R.gated_norm64(rs, None, None, c.d(c.scale, False), c.d(c.shift, False), c.d(c.w, False),
                                 c.d(c.bias, False), None, c.pre, 0, 1.0, c.eps, c.sample)
        _, m, rstd = R.norm64(rs, c.pre, c.eps)
        avg = rs.abs().mean(1, keepdim=True)
        a = (rs.abs() + avg) * rstd * (1 + avg * rstd) * (1.0 if c.w is None else c.w.double().abs())
        a = a + (0.0 if c.bias is None else c.bias.double().abs())
        a = a * (1.0 if scale is None else 1 + scale.abs()) + mag(shift)
        R.check_rounded(h[:n], want, C * a)
        assert float(amax) == float(h[:n].float().abs().max() if n else 0.0)
        if stats is not None:
            assert bool(((stats[:n, 0].double() - m[:, 0]).abs() <= C * avg[:, 0]).all())
            assert bool(((stats[:n, 1].double() - rstd[:, 0]).abs()
                         <= C * rstd[:, 0] * (1 + avg[:, 0] * rstd[:, 0])).all())


def check_backward(c, r, stats, out, amax=None):
    """Against autograd of the 64-bit formula at the stored r, whose row
    statistics are the ones given to the kernel to 2^-24 (1 + mean/deviation)
    -- `spread` below, a further factor on the terms that hold them."""
    n = c.last
    leaf = lambda t: None if t is None else t.double().detach().clone().requires_grad_()  # noqa: E731
    rs, y = leaf(r[:n]), leaf(None if c.y is None else c.y[:n])
    gate, scale, shift, w, bias, wp = map(leaf, (c.gate, c.scale, c.shift, c.w, c.bias, c.w_post))
    dr = c.dr.double()[:n]
    total = dr.clone()
    spread = torch.ones(n, 1, dtype=torch.float64, device="cuda")
    size = dr.abs()
    if c.pre:
        _, h = R.gated_norm64(rs, None, None, scale, shift, w, bias, None, c.pre, 0, 1.0, c.eps, c.sample)
        names = [t for t in (rs, scale, shift, w, bias) if t is not None]
        got = dict(zip(map(id, names), torch.autograd.grad(h, names, c.dh.double()[:n])))
        total = dr + got[id(rs)]
        _, m, rstd = R.norm64(rs.detach(), c.pre, c.eps)
        spread = 1 + rs.detach().abs().mean(1, keepdim=True) * rstd
        z = c.dh.double()[:n].abs()
        z = z if scale is None else z * (1 + R.rows_of(scale.detach(), c.sample)).abs()
        z = z if w is None else z * w.detach().abs()
        xh = (rs.detach().abs() + m.abs()) * rstd
        size = size + rstd * spread * (z + z.mean(1, keepdim=True) + xh * (z * xh).mean(1, keepdim=True))
        chunk = 1 + n // 148 + 256
        col = C + (chunk + 200) * R.U32
        dh = c.dh.double()[:n].abs()
        one = torch.ones(c.B, c.D, dtype=torch.float64, device="cuda")

        def by_sample(t):
            o = torch.zeros(c.B, c.D, dtype=torch.float64, device="cuda")
            return o.index_add_(0, c.sample, t)

        xs = xh * spread
        s1, s0 = by_sample(dh * xs), by_sample(dh)
        a = one if scale is None else (1 + scale.detach()).abs().expand(c.B, c.D)
        wd, bd = (1.0 if w is None else w.detach().abs()), (0.0 if bias is None else bias.detach().abs())
        if out.dscale is not None:
            R.check_rounded(out.dscale, got[id(scale)], col * (s1 * wd + s0 * bd))
        if out.dshift is not None:
            R.check_rounded(out.dshift, got[id(shift)], col * s0)
        if out.dweight is not None:
            R.check_rounded(out.dweight, got[id(w)], (col + c.B * R.U32) * (a * s1).sum(0))
        if out.dbias is not None:
            R.check_rounded(out.dbias, got[id(bias)], (col + c.B * R.U32) * (a * s0).sum(0))
    if out.dx is not None:
        R.check_rounded(out.dx[:n], total, C * size)
    if c.y is None:
        return
    _, r2 = None, R.gated_norm64(torch.zeros_like(y), y, gate, None, None, None, None, wp, 0, c.post, c.alpha, c.eps,
                                 c.sample)[0]
    names = [t for t in (y, gate, wp) if t is not None]
    got = dict(zip(map(id, names), torch.autograd.grad(r2, names, total)))
    _, my, ry = R.norm64(y.detach(), c.post, c.eps)
    yh = (y.detach().abs() + my.abs()) * ry if c.post else y.detach().abs()
    sy = 1 + y.detach().abs().mean(1, keepdim=True) * ry if c.post else 1.0
    e = c.alpha * size * (1.0 if gate is None else R.rows_of(gate.detach(), c.sample).abs())
    ew = e * (1.0 if wp is None else wp.detach().abs())
    bound = ew if not c.post else ry * sy * (ew + ew.mean(1, keepdim=True) + yh * (ew * yh).mean(1, keepdim=True))
    R.check_rounded(out.dy[:n], got[id(y)], 2 * C * bound)
    chunk = 1 + n // 148 + 256
    col = 2 * C + (chunk + 200 + c.B) * R.U32
    if out.dgate is not None:
        t = torch.zeros(c.B, c.D, dtype=torch.float64, device="cuda").index_add_(0, c.sample, size * yh * sy)
        R.check_rounded(out.dgate, got[id(gate)], col * c.alpha * t * (1.0 if wp is None else wp.detach().abs()))
    if out.dw_post is not None:
        R.check_rounded(out.dw_post, got[id(wp)], col * (e * yh * sy).sum(0))
    if amax is not None:
        assert float(amax) == float(out.dy[:n].float().abs().max())


SHAPES = [
    dict(M=1, D=8), dict(M=3, D=64), dict(M=33, D=72), dict(M=7, D=128), dict(M=130, D=256), dict(M=19, D=264),
    dict(M=40, D=1000), dict(M=300, D=1152), dict(M=9, D=4096), dict(M=11, D=4104), dict(M=5, D=8192),
]


@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: f"{s['M']}x{s['D']}")
@pytest.mark.parametrize("kind", [(2, 0), (1, 0), (1, 1), (2, 2), (0, 1), (0, 0)], ids=str)
def test_shapes_and_kinds(shape, kind):
    pre, post = kind
    c = Case(**shape, pre=pre, post=post, weights=shape["M"] % 2 == 1, xt=F32 if shape["D"] % 64 else BF16,
             pt=BF16 if shape["M"] % 3 == 0 else F32, seed=shape["D"] + 10 * pre + post)
    amax, amax_dy = torch.zeros(1, device="cuda"), torch.zeros(1, device="cuda")
    r, h, stats = c.forward(amax_h=amax if pre else None)
    check_forward(c, r, h, stats, amax)
    out = c.backward(r, stats, amax_dy=amax_dy)
    check_backward(c, r, stats, out, amax_dy)


@pytest.mark.parametrize("kw", [
    dict(M=64, D=192, res=False, mod=False),                       # a plain norm
    dict(M=64, D=192, res=False, weights=True),                    # a modulated norm of the first block
    dict(M=50, D=320, mod=False, weights=True, post=1),            # no modulation
    dict(M=60, D=320, B=4),                                        # samples of equal length
    dict(M=61, D=328, B=3, pad=24, xt=F32, offsets=[0, 20, 21, 61]),
    dict(M=61, D=96, B=5, post=2, weights=True, offsets=[0, 0, 30, 30, 61, 61]),  # empty samples
    dict(M=500, D=640, B=2, offsets=[0, 499, 500], weights=True, xt=F32),
    dict(M=2000, D=64, B=9, weights=True, post=1, pre=1,
         offsets=[0, 1, 3, 300, 301, 700, 1400, 1401, 1999, 2000]),
    dict(M=700, D=2048, B=2, mean=50.0, xt=F32),                   # a mean far above the deviation
    dict(M=4000, D=1536, B=3, offsets=[0, 1000, 1001, 4000]),      # many rows per block
    dict(M=5001, D=128, B=1, pre=1),
    dict(M=2400, D=4608, B=2, xt=F32, offsets=[0, 1300, 2400], pt=BF16),
], ids=lambda k: "-".join(f"{a}{v}" for a, v in k.items() if a != "offsets"))
def test_samples_strides_and_absent_parts(kw):
    c = Case(seed=7, **kw)
    amax, amax_dy = torch.zeros(1, device="cuda"), torch.zeros(1, device="cuda")
    r, h, stats = c.forward(amax_h=amax)
    check_forward(c, r, h, stats, amax)
    out = c.backward(r, stats, amax_dy=amax_dy if c.y is not None else None)
    check_backward(c, r, stats, out, amax_dy if c.y is not None else None)
    for k in range(c.B):  # an empty sample's gradients are zero
        if not bool((c.sample == k).any()):
            for t in (out.dgate, out.dscale, out.dshift):
                assert not t[k].any()


@pytest.mark.parametrize("D", [64, 1024])
def test_rows_behind_the_last_sample_stay(D):
    c = Case(90, D, B=2, offsets=[0, 31, 50], weights=True, post=1)
    mark = 7.0
    full = lambda *s, dtype=BF16: torch.full(s, mark, dtype=dtype, device="cuda")  # noqa: E731
    r, h, stats = full(90, D), full(90, D), full(90, 4, dtype=F32)
    amax = torch.zeros(1, device="cuda")
    c.x[50:] = 1e30  # what lies behind is not read into anything
    c.y[50:] = float("nan")
    c.forward(r=r, h=h, stats=stats, amax_h=amax)
    check_forward(c, r, h, stats, amax)
    assert bool((r[50:] == mark).all()) and bool((h[50:] == mark).all()) and bool((stats[50:] == mark).all())
    c.dh[50:], c.dr[50:] = float("nan"), float("inf")
    dx, dy = full(90, D), full(90, D)
    out = c.backward(r, stats, dx=dx, dy=dy)
    check_backward(c, r, stats, out)
    assert bool((dx[50:] == mark).all()) and bool((dy[50:] == mark).all())


def test_all_samples_empty():
    c = Case(10, 128, B=2, offsets=[0, 0, 0], weights=True)
    r, h = torch.full_like(c.x, 3.0), torch.full_like(c.x, 3.0)
    _, _, stats = c.forward(r=r, h=h)
    assert bool((r == 3.0).all()) and bool((h == 3.0).all())
    out = c.backward(r, stats)
    for t in (out.dgate, out.dscale, out.dshift, out.dweight, out.dbias):
        assert not t.any()


def test_no_rows():
    c = Case(0, 128, B=1, weights=True)
    r, h, stats = c.forward()
    assert r.shape == (0, 128) and h.shape == (0, 128)
    out = c.backward(r, stats)
    for t in (out.dgate, out.dscale, out.dshift, out.dweight, out.dbias):
        assert not t.any()


def test_parameters_that_all_samples_share():
    """[D] and [1, D] gates serve every sample; their gradient is the sum."""
    a = Case(48, 160, B=3, offsets=[0, 5, 40, 48], seed=3)
    gate, scale, shift = a.gate[:1].clone(), a.scale[0].clone(), a.shift[1:2].clone()
    a.gate, a.scale, a.shift = gate.expand(3, -1).contiguous(), scale.expand(3, -1).contiguous(), \
        shift.expand(3, -1).contiguous()
    r0, h0, s0 = a.forward()
    out0 = a.backward(r0, s0)
    a.gate, a.scale, a.shift = gate, scale, shift
    r1, h1, s1 = a.forward()
    out1 = a.backward(r1, s1)
    assert torch.equal(r0, r1) and torch.equal(h0, h1) and torch.equal(out0.dx, out1.dx)
    assert out1.dgate.shape == (1, 160) and out1.dscale.shape == (160,) and out1.dshift.shape == (1, 160)
    # three FP32 numbers added: two roundings of their magnitudes
    for one, many in ((out1.dgate, out0.dgate), (out1.dscale, out0.dscale), (out1.dshift, out0.dshift)):
        m = many.double()
        R.check_rounded(one.view(-1), m.sum(0), 2 * R.U32 * m.abs().sum(0))


def test_in_place():
    c = Case(70, 512, xt=BF16, post=1, weights=True)
    r, h, stats = c.forward()
    out = c.backward(r, stats)
    x = c.x.clone()
    c.x = x
    r2, h2, _ = c.forward(r=x)
    assert r2.data_ptr() == x.data_ptr() and torch.equal(r2, r) and torch.equal(h2, h)
    dr, dh = c.dr.clone(), c.dh.clone()
    c.dr, c.dh = dr, dh
    out2 = c.backward(r2, stats, dx=dr, dy=dh)
    assert torch.equal(dr, out.dx) and torch.equal(dh, out.dy) and torch.equal(out2.dgate, out.dgate)


@pytest.mark.parametrize("kw", [dict(M=300, D=1536), dict(M=70, D=96, post=2, weights=True)], ids=str)
def test_in_place_of_the_block(kw):
    """h over y, the stream over itself, and dy over y."""
    c = Case(xt=BF16, **kw)
    r, h, stats = c.forward()
    want = c.backward(r, stats)
    x, y = c.x, c.y
    c.x, c.y = x.clone(), y.clone()
    r2, h2, stats2 = c.forward(r=c.x, h=c.y)
    assert torch.equal(c.x, r) and torch.equal(c.y, h) and torch.equal(stats2, stats)
    c.y = y.clone()
    got = c.backward(r2, stats, dy=c.y, dx=c.x)
    assert torch.equal(c.y, want.dy) and torch.equal(c.x, want.dx) and torch.equal(got.dgate, want.dgate)


def test_amax_is_raised_and_never_lowered():
    c = Case(40, 256)
    high = torch.full((1,), 1e6, device="cuda")
    r, h, stats = c.forward(amax_h=high)
    assert float(high) == 1e6
    c.backward(r, stats, amax_dy=high)
    assert float(high) == 1e6


def test_rows_of_one_value_and_non_finite_rows():
    """A constant row has no deviation: h is the shift.  NaN and infinities
    stay in their own row, and the amax does not see NaN."""
    D = 96
    x = torch.randn(6, D, device="cuda")
    x[1] = 5.0
    x[2] = 0.0
    x[3, 7] = float("nan")
    x[4, 3] = float("inf")
    shift = torch.randn(1, D, device="cuda")
    scale = torch.randn(1, D, device="cuda")
    amax = torch.zeros(1, device="cuda")
    _, h, stats = ft.ft_gated_norm_fwd(ft.GatedNorm(), x, None, None, scale, shift, amax_h=amax)
    assert torch.equal(h[1], shift[0].to(BF16)) and torch.equal(h[2], shift[0].to(BF16))
    assert bool(h[3].isnan().all()) and bool(h[4].isnan().all())
    good = h[[0, 1, 2, 5]]
    assert bool(good.isfinite().all())
    assert float(amax) == float(good.float().abs().max())


def test_large_offsets_into_the_residual_stream():
    """Rows whose byte offset passes 2^31: 300000 rows of 8192 bytes."""
    M, D = 300_000, 4096
    x = torch.randn(1, D, device="cuda").to(BF16).expand(M, D).contiguous()
    x[-1] *= 2
    _, h, stats = ft.ft_gated_norm_fwd(ft.GatedNorm(pre=1), x)
    assert torch.equal(h[0], h[M - 2]) and torch.equal(stats[0], stats[M - 2])
    assert abs(float(stats[M - 1, 1] / stats[0, 1]) - 0.5) < 1e-6


def test_repeats_streams_and_graphs():
    """The same bits again, on another stream next to other work, and from a
    captured graph whose inputs change between replays."""
    a = Case(700, 1536, B=2, weights=True, post=1, seed=1)
    b = Case(700, 1536, B=2, weights=True, post=1, seed=2)

    def both(c):
        r, h, stats = c.forward()
        o = c.backward(r, stats)
        return [r, h, stats, o.dx, o.dy, o.dgate, o.dscale, o.dshift, o.dweight, o.dbias, o.dw_post]

    want_a, want_b = both(a), both(b)
    torch.cuda.synchronize()
    for got, want in zip(both(a), want_a):
        assert torch.equal(got, want)
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    got = {}
    for _ in range(3):
        for s, c, k in ((s1, a, "a"), (s2, b, "b")):
            with torch.cuda.stream(s):
                got[k] = both(c)
    torch.cuda.synchronize()
    for k, want in (("a", want_a), ("b", want_b)):
        assert all(torch.equal(x, y) for x, y in zip(got[k], want))
    # the stream argument, next to a current stream of its own
    s1.wait_stream(torch.cuda.current_stream())
    r, h, _ = a.forward(stream=s1)
    s1.synchronize()
    assert torch.equal(r, want_a[0]) and torch.equal(h, want_a[1])
    # two graphs that own their scratch, replayed in turn
    graphs = []
    for c in (a, b):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = both(c)
        graphs.append((g, out))
    for _ in range(2):
        for (g, out), want in zip(graphs, (want_a, want_b)):
            g.replay()
            torch.cuda.synchronize()
            assert all(torch.equal(x, y) for x, y in zip(out, want))
    a.x.copy_(b.x), a.y.copy_(b.y), a.dh.copy_(b.dh), a.dr.copy_(b.dr)
    for n in ("gate", "scale", "shift", "w", "bias", "w_post"):
        getattr(a, n).copy_(getattr(b, n))
    graphs[0][0].replay()
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(graphs[0][1], want_b))


def test_selected_gradients_and_a_workspace():
    c = Case(333, 768, weights=True, post=1, B=1)
    r, h, stats = c.forward()
    all_ = c.backward(r, stats)
    ws = ft.Workspace()
    some = c.backward(r, stats, param_grads=("scale", "w_post"), ws=ws)
    assert some.dgate is None and some.dweight is None
    assert torch.equal(some.dscale, all_.dscale) and torch.equal(some.dw_post, all_.dw_post)
    assert torch.equal(some.dx, all_.dx) and torch.equal(some.dy, all_.dy)
    none = c.backward(r, stats, param_grads=False, need_dx=False)
    assert none.dx is None and none.dscale is None and torch.equal(none.dy, all_.dy)


def test_python_refusals():
    c = Case(12, 64, B=2)
    with pytest.raises(TypeError):
        ft.ft_gated_norm_fwd(c.norm, c.x.half())
    with pytest.raises(TypeError):
        ft.ft_gated_norm_fwd(c.norm, c.x, c.y.float())
    with pytest.raises(ValueError):
        ft.ft_gated_norm_fwd(c.norm, c.x, c.y[:6])
    with pytest.raises(ValueError):
        ft.ft_gated_norm_fwd(c.norm, c.x, c.y, c.gate, c.scale[:, :32], c.shift)
    with pytest.raises(ValueError):
        ft.ft_gated_norm_fwd(c.norm, c.x, c.y, c.gate, torch.zeros(3, 64, device="cuda"))
    with pytest.raises(TypeError):
        ft.ft_gated_norm_fwd(c.norm, c.x, c.y, c.gate, c.scale.bfloat16())
    with pytest.raises(ValueError):
        ft.ft_gated_norm_fwd(c.norm, c.x.t().contiguous().t())
    with pytest.raises(ft.FtError):
        ft.ft_gated_norm_fwd(ft.GatedNorm(), torch.zeros(4, 60, device="cuda"))
    with pytest.raises(TypeError):
        ft.ft_gated_norm_fwd(c.norm, c.x, offsets=torch.tensor([0, 12], device="cuda"))
    with pytest.raises(ValueError):
        ft.ft_gated_norm_bwd(c.norm, None, None, None)
    r, h, stats = c.forward()
    with pytest.raises(ValueError):
        ft.ft_gated_norm_bwd(c.norm, c.dh, r, stats, gate=c.gate)
    with pytest.raises(ValueError):
        ft.ft_gated_norm_bwd(c.norm, c.dh, r, stats, param_grads=("bias",))


@pytest.mark.parametrize("D,xt", [(1024, BF16), (264, F32), (4096, F32)], ids=str)
def test_a_scale_next_to_minus_one(D, xt):
    """1 + scale of a few 2^-24 (a channel that the modulation all but
    closes): h is still (N(r)) (1 + scale) to its own rounding, not to that
    of the scale."""
    c = Case(6, D, xt=xt, seed=D)
    k = torch.arange(D, device="cuda") % 5
    c.scale = (k * 2.0 ** -24 - 1.0).view(1, D)
    c.shift = torch.zeros(1, D, device="cuda")
    assert c.scale.dtype == F32 and torch.equal(c.scale.double(), (k.double() * 2.0 ** -24 - 1.0).view(1, D))
    r, h, _ = c.forward()
    rs = r.double()
    n, m, rstd = R.norm64(rs, c.pre, c.eps)
    avg = rs.abs().mean(1, keepdim=True)
    a = 1 + c.scale.double()
    R.check_rounded(h, n * a, C * (rs.abs() + avg) * rstd * (1 + avg * rstd) * a)
