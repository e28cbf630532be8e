"""AdamW over many tensors: 32-bit states against the formula in 64 bits,
8-bit states bit for bit against the same IEEE FP32 steps in numpy.

Tolerances of the 32-bit step: m takes three roundings, v four, each 2^-24 of
the magnitudes that meet; the update lr m / (sqrt(v) rc + eps) at most 16
more, and the parameter two.
"""
import copy
import pickle

import numpy as np
import pytest
import torch

import bit_quantized_lora_b200 as ft
import block_ref as R

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32
f32 = np.float32


def make(sizes, pdt=BF16, gdt=F32, seed=0, offset=0):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)

    def one(n, std, dt):
        return (torch.randn(n + offset, generator=g, device="cuda") * std).to(dt)[offset:]

    return [one(n, 0.05, pdt) for n in sizes], [one(n, 1e-3, gdt) for n in sizes]


def parts(flat, sizes):
    out, at = [], 0
    for n in sizes:
        out.append(flat[at:at + n])
        at += -(-n // 256) * 256
    return out


def check_step32(p0, m0, v0, g, t, opt_args, got_p, got_p16, m1, v1):
    lr, (b1, b2), eps, wd = opt_args
    p, m, v, gd = p0.double(), m0.double(), v0.double(), g.double()
    m = m * b1 + (1 - b1) * gd
    v = v * b2 + (1 - b2) * gd * gd
    R.check_rounded(m1, m, 4 * R.U32 * (m0.double().abs() + gd.abs()))
    R.check_rounded(v1, v, 5 * R.U32 * v)
    upd = lr / (1 - b1 ** t) * m / ((v / (1 - b2 ** t)).sqrt() + eps)
    mag = lr / (1 - b1 ** t) * (m0.double().abs() + gd.abs()) / ((v / (1 - b2 ** t)).sqrt() + eps)
    want = p * (1 - lr * wd) - upd
    slack = 4 * R.U32 * p.abs() + 24 * R.U32 * mag
    if got_p is not None:
        R.check_rounded(got_p, want, slack)
    if got_p16 is not None:
        R.check_rounded(got_p16, want, slack)


SIZES = [[1], [7, 8, 9], [255, 256, 257, 1], [2048], [2047, 4097, 12], [100_000, 3, 70_001], [0, 5, 0, 300]]


@pytest.mark.parametrize("sizes", SIZES, ids=str)
@pytest.mark.parametrize("kind", ["master", "bf16", "f32"])
def test_three_steps_with_32_bit_states(sizes, kind):
    gdt = BF16 if sizes[0] == 2048 else F32
    params, grads = make(sizes, F32 if kind == "f32" else BF16, gdt, seed=len(sizes))
    args = (1e-2, (0.9, 0.99), 1e-8, 0.1)
    opt = ft.AdamW(params, grads, lr=args[0], betas=args[1], eps=args[2], weight_decay=args[3], master=kind == "master")
    for t in (1, 2, 3):
        before = [x.clone() for x in params]
        masters = parts(opt.master.clone(), sizes) if kind == "master" else before
        m0, v0 = parts(opt.exp_avg.clone(), sizes), parts(opt.exp_avg_sq.clone(), sizes)
        opt.step()
        assert int(opt.step_count) == t and int(opt._step[1]) == 0
        for i, n in enumerate(sizes):
            if n == 0:
                continue
            got_p = parts(opt.master, sizes)[i] if kind == "master" else params[i] if kind == "f32" else None
            got16 = params[i] if kind != "f32" else None
            check_step32(masters[i], m0[i], v0[i], grads[i], t, args, got_p, got16, parts(opt.exp_avg, sizes)[i],
                         parts(opt.exp_avg_sq, sizes)[i])
            if kind == "master":  # the copy is the master's own rounding
                assert torch.equal(params[i], parts(opt.master, sizes)[i].to(BF16))
        for gr in grads:
            gr.mul_(-0.7)
    # the flat state's gaps stay empty
    at = 0
    for n in sizes:
        end = at + -(-n // 256) * 256
        assert not opt.exp_avg[at + n:end].any() and not opt.exp_avg_sq[at + n:end].any()
        at = end


# ---------------------------------------------------------------- 8 bits
def np_blocks(x):
    pad = np.zeros(-len(x) % 256, f32)
    return np.concatenate([x.astype(f32), pad]).reshape(-1, 256)


def np_encode_m(m):
    b = np_blocks(m)
    top = np.abs(b).max(1)
    with np.errstate(divide="ignore", over="ignore"):
        inv = np.where(top >= f32(2.0 ** -126), f32(1) / top, f32(0)).astype(f32)
    c = np.rint(np.sqrt((np.abs(b) * inv[:, None]).astype(f32)).astype(f32) * f32(127)).astype(np.int32)
    return (np.where(b < 0, -c, c)).reshape(-1)[:len(m)].astype(np.int8), top


def np_encode_v(v):
    b = np_blocks(v)
    top = b.max(1)
    with np.errstate(divide="ignore", over="ignore"):
        inv = np.where(top >= f32(2.0 ** -126), f32(1) / top, f32(0)).astype(f32)
    c = np.rint(np.sqrt(np.sqrt((b * inv[:, None]).astype(f32))) * f32(255)).astype(np.int32)
    return c.reshape(-1)[:len(v)].astype(np.uint8), top


def np_decode_m(c, top):
    c = c.astype(np.int32)
    return ((c * np.abs(c)).astype(f32) * f32(1 / 16129)) * np.repeat(top, 256)[:len(c)]


def np_decode_v(c, top):
    r = (c.astype(np.int32) ** 2).astype(f32) * f32(1 / 65025)
    return (r * r) * np.repeat(top, 256)[:len(c)]


def host(t):
    return t.float().cpu().numpy()


@pytest.mark.parametrize("sizes", SIZES, ids=str)
@pytest.mark.parametrize("offset", [0, 1])
def test_8_bit_states_bit_for_bit(sizes, offset):
    """Five steps from zero; parameters at odd addresses with offset 1."""
    params, grads = make(sizes, seed=3, offset=offset)
    args = (1e-2, (0.9, 0.999), 1e-8, 0.0)
    opt = ft.AdamW(params, grads, lr=args[0], betas=args[1], eps=args[2], weight_decay=args[3], state_bits=8)
    state = [(np.zeros(n, np.int8), np.zeros(-(-n // 256), f32), np.zeros(n, np.uint8), np.zeros(-(-n // 256), f32))
             for n in sizes]
    for t in range(1, 6):
        masters = parts(opt.master.clone(), sizes)
        opt.step()
        m_flat, v_flat = opt.state_values()
        for i, n in enumerate(sizes):
            if n == 0:
                continue
            cm, tm, cv, tv = state[i]
            g = host(grads[i])
            m0, v0 = np_decode_m(cm, tm), np_decode_v(cv, tv)
            m = m0 * f32(0.9) + g * f32(1 - 0.9)
            v = v0 * f32(0.999) + (g * f32(1 - 0.999)) * g
            assert m.dtype == f32 and v.dtype == f32
            state[i] = (*np_encode_m(m), *np_encode_v(v))
            got = [host_codes(parts(opt.exp_avg, sizes)[i]), block_part(opt.exp_avg_scale, sizes, i),
                   host_codes(parts(opt.exp_avg_sq, sizes)[i]), block_part(opt.exp_avg_sq_scale, sizes, i)]
            for a, b in zip(got, state[i]):
                np.testing.assert_array_equal(a, b)
            np.testing.assert_array_equal(host(parts(m_flat, sizes)[i]), np_decode_m(*state[i][:2]))
            np.testing.assert_array_equal(host(parts(v_flat, sizes)[i]), np_decode_v(*state[i][2:]))
            dev = lambda a: torch.from_numpy(np.ascontiguousarray(a)).cuda()  # noqa: E731
            # the update reads the moments before they are encoded
            check_step32(masters[i], dev(m0), dev(v0), grads[i], t, args, parts(opt.master, sizes)[i], params[i],
                         dev(m), dev(v))
        for gr in grads:
            gr.mul_(-1.3)


def host_codes(t):
    return t.cpu().numpy()


def block_part(scales, sizes, i):
    at = sum(-(-n // 256) for n in sizes[:i])
    return scales[at:at + -(-sizes[i] // 256)].cpu().numpy()


def test_codes_and_their_values():
    """All codes decode to their power of the block's largest, and a block
    whose largest is subnormal, zero or not finite keeps to its rule."""
    c = torch.arange(-127, 128, dtype=torch.int16).to(torch.int8).cuda()
    top = torch.tensor([3.0], device="cuda")
    got = ft.ft_adamw_decode(c, top).double()
    cd = c.double()
    # two roundings
    assert bool(((got - 3 * cd * cd.abs() / 16129).abs() <= 3 * R.U32 * got.abs()).all())
    assert float(got[-1]) == 3.0 and float(got[0]) == -3.0 and float(got[127]) == 0.0
    u = torch.arange(256, dtype=torch.int16).to(torch.uint8).cuda()
    got = ft.ft_adamw_decode(u, top).double()
    assert bool(((got - 3 * (u.double() / 255) ** 4).abs() <= 5 * R.U32 * got).all()) and float(got[255]) == 3.0
    p, _ = make([256 * 4], F32)
    g = torch.zeros(1024, device="cuda")
    g[0:256] = 1e-30     # m ~ 1e-31 normal, v = 0 by underflow
    g[256:512] = 1e-38   # m subnormal
    g[513] = float("nan")
    g[768:1024] = 1.0
    g[769] = float("inf")
    opt = ft.AdamW(p, [g], state_bits=8)
    opt.step()
    m, v = opt.state_values()
    assert bool((m[:256] > 0).all()) and not v[:256].any()
    assert not opt.exp_avg[256:512].any() and not m[256:512].any()
    assert bool(m[512:].isnan().all()) and bool(v[512:].isnan().all())
    assert bool(p[0][:512].isfinite().all()) and bool(p[0][514:768].isfinite().all())


# ---------------------------------------------------------------- the call
def test_many_tensors_few_tensors_and_any_alignment_agree():
    """500 tensors (two launches) step as each does alone, aligned or not."""
    sizes = [1 + (37 * i) % 700 for i in range(500)]
    for bits in (32, 8):
        params, grads = make(sizes, seed=5, offset=1)
        alone = [p.clone() for p in params]
        all_ = ft.AdamW(params, grads, state_bits=bits, weight_decay=[0.01 * (i % 3) for i in range(500)])
        all_.step()
        all_.step()
        assert int(all_.step_count) == 2
        for i in range(0, 500, 31):
            one = ft.AdamW([alone[i]], [grads[i]], state_bits=bits, weight_decay=0.01 * (i % 3))
            one.step()
            one.step()
            assert torch.equal(alone[i], params[i])


def test_learning_rate_scale_and_gradients_of_the_call():
    params, grads = make([1000, 77], seed=8)
    same = [p.clone() for p in params]
    a = ft.AdamW(params, lr=123.0)
    b = ft.AdamW(same, [g * 0.25 for g in grads], lr=2.0 ** -7)
    with pytest.raises(ValueError):
        a.step()
    a.step(grads, lr=torch.full((1,), 2.0 ** -7, device="cuda"), grad_scale=torch.full((1,), 0.25, device="cuda"))
    b.step()
    assert all(torch.equal(x, y) for x, y in zip(params, same))
    assert torch.equal(a.exp_avg, b.exp_avg) and torch.equal(a.exp_avg_sq, b.exp_avg_sq)


@pytest.mark.parametrize("eps,scale", [(0.0, 1e-3), (0.0, 1e-21), (1e-12, 1e-20), (1e-8, 1e-20), (1e-8, 1e15)])
def test_eps_and_extreme_gradients(eps, scale):
    """No eps at all, second moments that are subnormal or near the top of
    FP32's range: still the formula (a subnormal keeps 2^-149 of spacing)."""
    g = torch.Generator(device="cuda")
    g.manual_seed(4)
    p = torch.randn(3000, generator=g, device="cuda")
    p0 = p.clone()
    grad = (1 + torch.rand(3000, generator=g, device="cuda")) * scale
    opt = ft.AdamW([p], [grad], lr=2.0 ** -7, betas=(0.9, 0.999), eps=eps, weight_decay=0.0)
    opt.step()
    m, v = opt.exp_avg[:3000].double(), opt.exp_avg_sq[:3000].double()
    gd = grad.double()
    assert bool(((v - 0.001 * gd * gd).abs() <= 5 * R.U32 * 0.001 * gd * gd + 2.0 ** -148).all())
    # the step from the moments as they are stored
    upd = 2.0 ** -7 / 0.1 * m / ((v / 0.001).sqrt() + eps)
    upd = torch.where(m == 0, torch.zeros_like(upd), upd)
    fine = torch.isfinite(upd)
    R.check_rounded(p[fine], (p0.double() - upd)[fine], 4 * R.U32 * p0[fine].double().abs() + 24 * R.U32 * upd[fine].abs())


def test_state_is_saved_and_loaded():
    for bits in (32, 8):
        params, grads = make([3000, 10], seed=9)
        a = ft.AdamW(params, grads, state_bits=bits)
        a.step()
        saved, copies = a.state_dict(), [p.clone() for p in params]
        a.step()
        b = ft.AdamW(copies, grads, state_bits=bits)
        b.load_state_dict(saved)
        b.step()
        assert all(torch.equal(x, y) for x, y in zip(params, copies)) and int(b.step_count) == 2
        with pytest.raises(ValueError):
            ft.AdamW(copies, grads, state_bits=40 - bits).load_state_dict(saved)


def test_captured_step_counts_and_takes_a_new_rate():
    params, grads = make([5000, 300], seed=10)
    other = [p.clone() for p in params]
    lr, scale = torch.full((1,), 1e-3, device="cuda"), torch.ones(1, device="cuda")
    a = ft.AdamW(params, grads, state_bits=8)
    b = ft.AdamW(other, grads, state_bits=8)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        a.step(lr=lr, grad_scale=scale)
    for i in range(4):
        lr.fill_(2.0 ** -(8 + i))
        for gr in grads:
            gr.mul_(-0.9)
        g.replay()
        b.step(lr=2.0 ** -(8 + i))
        torch.cuda.synchronize()
        assert int(a.step_count) == i + 1
        assert all(torch.equal(x, y) for x, y in zip(params, other)), i
    assert torch.equal(a.exp_avg_sq, b.exp_avg_sq)


def test_two_optimizers_on_two_streams():
    made = [make([40_000, 999], seed=s) for s in (11, 12)]
    want = []
    for params, grads in made:
        copies = [p.clone() for p in params]
        o = ft.AdamW(copies, grads)
        for _ in range(3):
            o.step()
        want.append(copies)
    torch.cuda.synchronize()
    opts = [ft.AdamW(p, g) for p, g in made]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    for _ in range(3):
        for o, s in zip(opts, streams):
            o.step(stream=s)
    torch.cuda.synchronize()
    for (params, _), w in zip(made, want):
        assert all(torch.equal(x, y) for x, y in zip(params, w))


def test_refusals():
    p, g = make([64])
    with pytest.raises(TypeError):
        ft.AdamW([p[0].half()])
    with pytest.raises(ValueError):
        ft.AdamW([p[0].view(8, 8).t()])
    with pytest.raises(ValueError):
        ft.AdamW(p, betas=(0.9, 1.0))
    with pytest.raises(ValueError):
        ft.AdamW(p, state_bits=16)
    with pytest.raises(ValueError):
        ft.AdamW(p, weight_decay=[0.1, 0.2])
    with pytest.raises(ValueError):  # the same parameter twice
        ft.AdamW([p[0], p[0]])
    o = ft.AdamW(p)
    with pytest.raises(ValueError):
        o.step([g[0][:32]])
    with pytest.raises(TypeError):
        o.step([g[0].half()])
    with pytest.raises(TypeError):
        o.step(g, lr=torch.zeros(1, dtype=torch.float64, device="cuda"))
    with pytest.raises(TypeError):
        ft.ft_adamw_decode(g[0], g[0])


def test_exchanged_memory_is_looked_at_before_it_is_stepped():
    """A parameter or gradient may move to other memory between steps; memory
    of another size or type is refused, and nothing is stepped."""
    sizes = [1000, 256]
    params, grads = make(sizes, pdt=F32)
    twin = [p.clone() for p in params]
    opt, ref = ft.AdamW(params, grads), ft.AdamW(twin, [g.clone() for g in grads])
    opt.step(), ref.step()
    params[0].data = params[0].data.clone()
    grads[1].data = grads[1].data.to(BF16).float()
    ref.grads[1].copy_(grads[1])
    opt.step(), ref.step()
    for a, b in zip(params, twin):
        assert torch.equal(a, b)
    kept = params[0].data
    for other in (kept[:10].clone(), kept.to(BF16), torch.empty(0, device="cuda"), kept.cpu()):
        params[0].data = other
        with pytest.raises((ValueError, TypeError)):
            opt.step()
    params[0].data = kept
    held = grads[0].data
    for other in (held[:10].clone(), torch.empty(0, device="cuda"), held.cpu()):
        grads[0].data = other
        with pytest.raises((ValueError, TypeError)):
            opt.step()
    grads[0].data = held
    opt.step(), ref.step()
    for a, b in zip(params, twin):
        assert torch.equal(a, b)
    assert int(opt.step_count) == 3
    flat = torch.zeros(512, device="cuda")
    with pytest.raises(ValueError):  # two that overlap
        ft.AdamW([flat[:300], flat[256:]])


@pytest.mark.parametrize("bits", [32, 8])
def test_an_optimizer_is_not_copied_and_keeps_its_state(bits):
    params, grads = make([300])
    opt = ft.AdamW(params, grads, state_bits=bits)
    for copied in (copy.copy, copy.deepcopy, pickle.dumps):
        with pytest.raises(TypeError, match="state_dict"):
            copied(opt)
    for name in ("master", "exp_avg", "exp_avg_sq") + (("exp_avg_scale", "exp_avg_sq_scale") if bits == 8 else ()):
        mine = getattr(opt, name)
        setattr(opt, name, mine.clone())
        with pytest.raises(ValueError, match="load_state_dict"):
            opt.step()
        setattr(opt, name, mine)
    assert int(opt.step_count) == 0
    opt.step()
    assert int(opt.step_count) == 1


def test_a_refused_step_on_lent_gradients_leaves_no_trace():
    params, grads = make([700, 40])
    twin = [p.clone() for p in params]
    opt, ref = ft.AdamW(params, grads), ft.AdamW(twin, grads)
    opt.step(), ref.step()
    mine, opt.exp_avg = opt.exp_avg, opt.exp_avg.clone()
    with pytest.raises(ValueError):
        opt.step([g.clone().fill_(1.0) for g in grads])
    opt.exp_avg = mine
    opt.step(), ref.step()
    others = [g * 3 for g in grads]
    opt.step(others), ref.step(iter(others))
    opt.step(), ref.step()
    assert all(torch.equal(a, b) for a, b in zip(params, twin)) and int(opt.step_count) == 4


def test_memory_seen_another_way_is_looked_at_too():
    """The same bytes under other strides or as another type: refused like
    other memory, before anything is stepped; the old view steps on."""
    for gdt in (F32, BF16):
        params, grads = make([256, 64], pdt=gdt, gdt=gdt, seed=21)
        params, grads = [p.view(-1, 8) for p in params], [g.view(-1, 8) for g in grads]
        params[0], grads[0] = params[0].view(16, 16), grads[0].view(16, 16)
        twin = [p.clone() for p in params]
        opt, ref = ft.AdamW(params, grads, master=False), ft.AdamW(twin, [g.clone() for g in grads], master=False)
        opt.step(), ref.step()
        p, g = params[0].data, grads[0].data
        other = torch.float16 if gdt == BF16 else BF16
        for t, held, views in ((params[0], p, (p.t(), p.view(torch.int16), p.view(other))),
                               (grads[0], g, (g.t(), g.view(torch.int16), g.view(other), g.view(8, 32)))):
            for view in views:
                assert view.data_ptr() == held.data_ptr() and view.nbytes == held.nbytes
                t.data = view
                with pytest.raises((ValueError, TypeError)):
                    opt.step()
                t.data = held
        assert int(opt.step_count) == 1
        opt.step(), ref.step()
        assert all(torch.equal(a, b) for a, b in zip(params, twin)) and int(opt.step_count) == 2
