"""Cases that measure the operators around a block's 4-bit linears: the gated norm (forward, backward), the rotary
positions of queries and keys (forward, backward), GELU's backward and the AdamW step.

`run` computes a pass either in its plain form (elementary torch operations in 32 bits, each output rounded once) or,
with `own` set, by the package's entry points.  `exact` computes the same outputs in 64 bits.
"""
import math
import random

import torch

own = False

BF16, F32, F64 = torch.bfloat16, torch.float32, torch.float64
BLOCK = 256  # values of an optimizer state that share one 8-bit scale


# ------------------------------------------------------------------ cases
def listed():
    return [
        # the text tokens of one prompt before a block's first linear: a call that is all latency
        dict(name="norm_fwd text", op="norm_fwd", M=77, D=768, B=1, ragged=False, pre="rms", post="none", res=False,
             mod=False, weights=True, x32=False, p32=True),
        # between the attention and the MLP of a DiT block: 4608 tokens (4096 of the image, 512 of the text), width 3072
        dict(name="norm_fwd dit", op="norm_fwd", M=4608, D=3072, B=1, ragged=False, pre="layer", post="none", res=True,
             mod=True, weights=False, x32=False, p32=False),
        # five images of different sizes packed into one batch, residual stream in fp32, norms on both sides of the
        # block and their weights trained
        dict(name="norm_bwd packed", op="norm_bwd", M=2077, D=1160, B=5, ragged=True, pre="rms", post="rms", res=True,
             mod=True, weights=True, x32=True, p32=True),
        # the backward of the DiT block's norm, with the gradients of its modulation
        dict(name="norm_bwd dit", op="norm_bwd", M=4608, D=3072, B=1, ragged=False, pre="layer", post="none", res=True,
             mod=True, weights=False, x32=False, p32=False),
        # the MLP of a small layer on few tokens
        dict(name="gelu_bwd few", op="gelu_bwd", n=37 * 512),
        # the MLP-up output of the DiT block
        dict(name="gelu_bwd dit", op="gelu_bwd", n=4608 * 12288),
        # one new token of a video model, grouped key heads, half-split pairs, positions far along the time axis
        dict(name="rope_fwd token", op="rope_fwd", M=1, Hq=16, Hk=4, hd=64, axes="16,24,24", halves=True, norm=True,
             far=1000000, head_major=False),
        # the QKV output of the DiT block, three axes, interleaved pairs, query and key norms
        dict(name="rope_fwd dit", op="rope_fwd", M=4608, Hq=24, Hk=24, hd=128, axes="16,56,56", halves=False, norm=True,
             far=64, head_major=True),
        # grouped heads of an odd size at an odd number of tokens, no norms, part of the head not rotated
        dict(name="rope_bwd grouped", op="rope_bwd", M=1333, Hq=10, Hk=2, hd=96, axes="24,40", halves=True, norm=False,
             far=5000, head_major=False),
        # the backward of the DiT block's rotation: the gradient of the QKV linear's output and of the norms' weights
        dict(name="rope_bwd dit", op="rope_bwd", M=4608, Hq=24, Hk=24, hd=128, axes="16,56,56", halves=False, norm=True,
             far=64, head_major=True),
        # the adapter of one small layer (two tensors)
        dict(name="adamw layer", op="adamw", bits=32, tensors=2, least=256 * 16, most=256 * 16, sizes=1, g16=False, step=0),
        # the adapters of eight DiT blocks (32 linears), states in 8 bits
        dict(name="adamw stack", op="adamw", bits=8, tensors=64, least=3072 * 32, most=12288 * 64, sizes=2, g16=False,
             step=400),
    ]


def _log(rng, a, b):
    return min(b, max(a, int(round(math.exp(rng.uniform(math.log(a), math.log(b)))))))


def draw(rng):
    op = rng.choice(["norm_fwd", "norm_bwd", "norm_fwd", "norm_bwd", "gelu_bwd", "rope_fwd", "rope_bwd", "adamw"])
    if op in ("norm_fwd", "norm_bwd"):
        D = 8 * _log(rng, 8, 1024)
        M = _log(rng, 1, min(16384, 12_000_000 // D))
        ragged = rng.random() < 0.5
        B = rng.randint(1, min(9, M)) if ragged else 1
        res = rng.random() < 0.75
        post = rng.choice(["none", "rms", "layer"]) if res else "none"
        pre = rng.choice(["rms", "layer", "layer"] + (["none"] if res else []))
        return dict(op=op, M=M, D=D, B=B, ragged=ragged, pre=pre, post=post, res=res, mod=rng.random() < 0.7,
                    weights=rng.random() < 0.5, x32=rng.random() < 0.4, p32=rng.random() < 0.5)
    if op == "gelu_bwd":
        return dict(op=op, n=8 * _log(rng, 1, 6_000_000))
    if op in ("rope_fwd", "rope_bwd"):
        hd = rng.choice([32, 64, 80, 96, 128, 192, 256])
        Hk = rng.choice([1, 2, 3, 4, 8])
        Hq = Hk * rng.choice([1, 2, 4, 5])
        M = _log(rng, 1, min(16384, 40_000_000 // ((Hq + 2 * Hk) * hd)))
        rot = hd if rng.random() < 0.7 else hd // 16 * 8
        n = rng.randint(1, 3)
        cuts = sorted(rng.sample(range(1, rot // 2), n - 1)) if n > 1 else []
        axes = [2 * (b - a) for a, b in zip([0] + cuts, cuts + [rot // 2])]
        return dict(op=op, M=M, Hq=Hq, Hk=Hk, hd=hd, axes=",".join(map(str, axes)), halves=rng.random() < 0.5,
                    norm=rng.random() < 0.5, far=_log(rng, 8, 2_000_000), head_major=rng.random() < 0.5)
    least = _log(rng, 1, 20000)
    most = _log(rng, least, 400_000)
    return dict(op=op, bits=rng.choice([8, 32]), tensors=_log(rng, 1, 60), least=least, most=most,
                sizes=rng.randint(0, 1 << 20), g16=rng.random() < 0.3, step=_log(rng, 1, 5000))


# ------------------------------------------------------------------ inputs
def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _randn(g, *shape, std=1.0, mean=0.0, dtype=F32):
    return (torch.randn(*shape, generator=g, device="cuda") * std + mean).to(dtype)


def _axes(c):
    return [int(a) for a in c["axes"].split(",")]


def _sizes(c):
    """Tensor sizes of an optimizer case: the largest and the smallest, and others spread between them."""
    r = random.Random(c["sizes"])
    n = [c["most"], c["least"]] + [_log(r, c["least"], c["most"]) for _ in range(c["tensors"] - 2)]
    return n[:c["tensors"]]


def _stream(g, M, D, dtype):
    """A residual stream: a few channels run far above the others, and rows have a mean of their own."""
    x = torch.randn(M, D, generator=g, device="cuda")
    x[:, :: max(1, D // 7)] *= 12.0
    return (x + 0.3 * torch.randn(M, 1, generator=g, device="cuda")).to(dtype)


def _norm_inputs(c, g):
    M, D, B = c["M"], c["D"], c["B"]
    xt, pt = (F32 if c["x32"] else BF16), (F32 if c["p32"] else BF16)
    s = dict(case=c, offsets=None)
    if c["ragged"]:
        cuts = torch.randperm(M - 1, generator=g, device="cuda")[: B - 1].sort().values + 1 if B > 1 else \
            torch.zeros(0, dtype=torch.int64, device="cuda")
        ends = torch.full((1,), M, dtype=torch.int64, device="cuda")
        s["offsets"] = torch.cat([torch.zeros_like(ends), cuts, ends]).to(torch.int32)
    s["x"] = _stream(g, M, D, xt)
    s["y"] = _randn(g, M, D, std=0.7, mean=0.05, dtype=BF16) if c["res"] else None
    # the modulation vectors are slices of one tensor, as the linear that makes them leaves it
    mod = _randn(g, B, 3 * D, std=0.4, dtype=pt)
    s["gate"] = mod[:, :D] if c["mod"] and c["res"] else None
    s["scale"], s["shift"] = (mod[:, D:2 * D], mod[:, 2 * D:]) if c["mod"] and c["pre"] != "none" else (None, None)
    w = c["weights"]
    s["weight"] = _randn(g, D, std=0.2, mean=1.0, dtype=pt) if w and c["pre"] != "none" else None
    s["bias"] = _randn(g, D, std=0.2, dtype=pt) if w and c["pre"] == "layer" else None
    s["w_post"] = _randn(g, D, std=0.2, mean=1.0, dtype=pt) if w and c["post"] != "none" else None
    s["alpha"] = 0.7 if c["post"] != "none" else 1.0
    s["eps"] = 1e-6
    return s


def _stats64(x, kind, eps):
    """(mean, 1 / deviation) of each row, in 64 bits."""
    x = x.to(F64)
    mean = x.mean(1) if kind == "layer" else torch.zeros(x.shape[0], dtype=F64, device=x.device)
    if kind == "none":
        return mean, torch.ones_like(mean)
    return mean, (((x - mean[:, None]) ** 2).mean(1) + eps).rsqrt()


def prepare(case, seed):
    g, c = _gen(seed), case
    op = c["op"]
    if op == "norm_fwd":
        return _norm_inputs(c, g)
    if op == "norm_bwd":
        s = _norm_inputs(c, g)
        M, D = c["M"], c["D"]
        # what the forward left: the stream behind the block and the rows' statistics
        s["r"] = s.pop("x")
        m0, r0 = _stats64(s["r"], c["pre"], s["eps"])
        m1, r1 = _stats64(s["y"], c["post"], s["eps"]) if c["res"] else (torch.zeros_like(m0), torch.ones_like(m0))
        s["stats"] = torch.stack([m0, r0, m1, r1], 1).to(F32)
        s["dh"] = _randn(g, M, D, std=1e-3, dtype=BF16) if c["pre"] != "none" else None
        s["dr"] = _randn(g, M, D, std=2e-3, dtype=s["r"].dtype)
        return s
    if op == "gelu_bwd":
        return dict(case=c, y=_randn(g, c["n"], std=1.2, dtype=BF16), dh=_randn(g, c["n"], std=1e-3, dtype=BF16))
    if op in ("rope_fwd", "rope_bwd"):
        M, hd, axes, rot = c["M"], c["hd"], _axes(c), sum(_axes(c))
        H = c["Hq"] + 2 * c["Hk"]
        s = dict(case=c, qkv=_randn(g, M, H * hd, std=1.5, dtype=BF16))
        s["pos"] = torch.randint(0, c["far"], (M, len(axes)), generator=g, device="cuda", dtype=torch.int32)
        # radians a position, per pair: each axis runs through its own powers of theta (the rotation's plan)
        s["freqs"] = torch.cat([10000.0 ** (-2.0 * torch.arange(a // 2, dtype=F64, device="cuda") / a) for a in axes])
        s["w_q"] = _randn(g, hd, std=0.2, mean=1.0, dtype=F32) if c["norm"] else None
        s["w_k"] = _randn(g, hd, std=0.2, mean=1.0, dtype=F32) if c["norm"] else None
        if op == "rope_bwd":
            for n, heads in (("dq", c["Hq"]), ("dk", c["Hk"]), ("dv", c["Hk"])):
                shape = (1, heads, M, hd) if c["head_major"] else (1, M, heads, hd)
                t = _randn(g, *shape, std=1e-3, dtype=BF16)
                s[n] = t if c["head_major"] else t.transpose(1, 2)
        return s
    # AdamW: every tensor starts at a multiple of BLOCK in one flat buffer, the rest of its last block is zero
    sizes = _sizes(c)
    starts, total = [], 0
    for n in sizes:
        starts.append(total)
        total += -(-n // BLOCK) * BLOCK
    at = torch.arange(total, device="cuda")
    ends = torch.tensor([a + n for a, n in zip(starts, sizes)], device="cuda")
    tops = torch.tensor(starts[1:] + [total], device="cuda")
    real = at < ends[torch.searchsorted(tops, at, right=True)]
    size = torch.exp(_randn(g, total)) * 1e-4  # gradients differ in size from value to value
    s = dict(case=c, sizes=sizes, starts=starts, lr=1e-3, betas=(0.9, 0.999), eps=1e-8, wd=0.01)
    s["p"] = _randn(g, total, std=0.01) * real
    s["p16"] = s["p"].to(BF16)
    s["g"] = (torch.randn(total, generator=g, device="cuda") * size * real).to(BF16 if c["g16"] else F32)
    s["step"] = torch.full((1,), c["step"], dtype=torch.int64, device="cuda")
    age = min(1.0, 0.001 * c["step"])
    m = torch.randn(total, generator=g, device="cuda") * size * real * (0.2 if c["step"] else 0.0)
    v = (size * (0.5 + torch.rand(total, generator=g, device="cuda"))) ** 2 * real * age
    if c["bits"] == 8:
        s["m"], s["m_scale"] = _encode_m(m)
        s["v"], s["v_scale"] = _encode_v(v)
    else:
        s["m"], s["v"] = m, v
    if own:  # the optimizer that a training program keeps from step to step
        import bit_quantized_lora_b200 as ft
        views = [s["p16"][a:a + n] for a, n in zip(starts, sizes)]
        grads = [s["g"][a:a + n] for a, n in zip(starts, sizes)]
        opt = ft.AdamW(views, grads, lr=s["lr"], betas=s["betas"], eps=s["eps"], weight_decay=s["wd"],
                       state_bits=c["bits"])
        opt.master.copy_(s["p"])
        opt.exp_avg.copy_(s["m"])
        opt.exp_avg_sq.copy_(s["v"])
        opt.step_count.copy_(s["step"])
        if c["bits"] == 8:
            opt.exp_avg_scale.copy_(s["m_scale"])
            opt.exp_avg_sq_scale.copy_(s["v_scale"])
        s["opt"] = opt
    return s


# ------------------------------------------------------------------ plain forms
def _blocks_scaled(a):
    """|values| over their block's largest, by one reciprocal a block (0 where that is subnormal)."""
    top = a.amax(1, keepdim=True)
    return a * torch.where(top >= 2.0 ** -126, top.reciprocal(), 0.0), top.squeeze(1)


def _encode_m(m):
    """First moments in 8 bits: sign and a code c in 0..127 that stands for (c / 127)^2 of the block's largest."""
    b = m.view(-1, BLOCK)
    q, top = _blocks_scaled(b.abs())
    return ((q.sqrt() * 127.0).round() * b.sign()).to(torch.int8).view(-1), top


def _encode_v(v):
    """Second moments in 8 bits: a code c in 0..255 that stands for (c / 255)^4 of the block's largest."""
    q, top = _blocks_scaled(v.view(-1, BLOCK))
    return (q.sqrt().sqrt() * 255.0).round().to(torch.uint8).view(-1), top


def _decode_m(c, top):
    c = c.to(F32).view(-1, BLOCK)
    return (c * c.abs() * (1.0 / 16129.0) * top[:, None]).view(-1)


def _decode_v(c, top):
    c = c.to(F32).view(-1, BLOCK)
    r = c * c * (1.0 / 65025.0)
    return (r * r * top[:, None]).view(-1)


def _sample_of(s, M):
    """The sample that each row belongs to."""
    if s["offsets"] is None:
        return torch.arange(M, device="cuda") * s["case"]["B"] // M
    return torch.searchsorted(s["offsets"][1:].contiguous().long(), torch.arange(M, device="cuda"), right=True)


def _rows(v, b):
    return None if v is None else v.to(F32)[b]


def _normed(x, kind, eps):
    if kind == "rms":
        return x * ((x * x).mean(1, keepdim=True) + eps).rsqrt()
    d = x - x.mean(1, keepdim=True)
    return d * ((d * d).mean(1, keepdim=True) + eps).rsqrt()


def _row_stats(x, kind, eps):
    mean = x.mean(1) if kind == "layer" else torch.zeros(x.shape[0], device="cuda")
    if kind == "none":
        return mean, torch.ones_like(mean)
    return mean, (((x - mean[:, None]) ** 2).mean(1) + eps).rsqrt()


def _norm_fwd(s):
    c = s["case"]
    b = _sample_of(s, c["M"])
    r, out = s["x"], {}
    zero, one = torch.zeros(c["M"], device="cuda"), torch.ones(c["M"], device="cuda")
    post = (zero, one)
    if c["res"]:
        u = s["y"].to(F32)
        if c["post"] != "none":
            post = _row_stats(u, c["post"], s["eps"])
            u = _normed(u, c["post"], s["eps"])
            u = u if s["w_post"] is None else u * s["w_post"].to(F32)
        u = u if s["gate"] is None else u * _rows(s["gate"], b)
        r = (s["x"].to(F32) + s["alpha"] * u).to(s["x"].dtype)
        out["r"] = r
    x = r.to(F32)
    pre = _row_stats(x, c["pre"], s["eps"])
    out["stats"] = torch.stack([*pre, *post], 1)
    if c["pre"] != "none":
        h = _normed(x, c["pre"], s["eps"])
        h = h if s["weight"] is None else h * s["weight"].to(F32)
        h = h if s["bias"] is None else h + s["bias"].to(F32)
        h = h if s["scale"] is None else h * (1 + _rows(s["scale"], b)) + _rows(s["shift"], b)
        out["h"] = h.to(BF16)
        out["amax_h"] = out["h"].abs().max().to(F32).view(1)
    return out


def _through_norm(g, xhat, rstd, kind):
    """The gradient of a row before a norm, from the one behind it."""
    k = (g * xhat).mean(1, keepdim=True)
    return rstd[:, None] * (g - xhat * k - (g.mean(1, keepdim=True) if kind == "layer" else 0.0))


def _per_sample(t, b, B):
    """Sums of the rows of each sample."""
    return (b == torch.arange(B, device="cuda")[:, None]).to(F32) @ t if B > 1 else t.sum(0, keepdim=True)


def _norm_bwd(s):
    c, st = s["case"], s["stats"]
    b, B = _sample_of(s, c["M"]), c["B"]
    d, out = s["dr"].to(F32), {}
    if c["pre"] != "none":
        dh = s["dh"].to(F32)
        xhat = (s["r"].to(F32) - st[:, 0:1]) * st[:, 1:2]
        n = xhat if s["weight"] is None else xhat * s["weight"].to(F32)
        n = n if s["bias"] is None else n + s["bias"].to(F32)
        dn = dh if s["scale"] is None else dh * (1 + _rows(s["scale"], b))
        if s["scale"] is not None:
            out["dscale"], out["dshift"] = _per_sample(dh * n, b, B), _per_sample(dh, b, B)
        if s["weight"] is not None:
            out["dweight"] = (dn * xhat).sum(0)
        if s["bias"] is not None:
            out["dbias"] = dn.sum(0)
        g = dn if s["weight"] is None else dn * s["weight"].to(F32)
        d = d + _through_norm(g, xhat, st[:, 1], c["pre"])
    out["dx"] = d.to(s["dr"].dtype)
    if c["res"]:
        y = s["y"].to(F32)
        yhat = y if c["post"] == "none" else (y - st[:, 2:3]) * st[:, 3:4]
        u = yhat if s["w_post"] is None else yhat * s["w_post"].to(F32)
        if s["gate"] is not None:
            out["dgate"] = s["alpha"] * _per_sample(u * d, b, B)
        du = s["alpha"] * (d if s["gate"] is None else d * _rows(s["gate"], b))
        if s["w_post"] is not None:
            out["dw_post"] = (du * yhat).sum(0)
            du = du * s["w_post"].to(F32)
        if c["post"] != "none":
            du = _through_norm(du, yhat, st[:, 3], c["post"])
        out["dy"] = du.to(BF16)
        out["amax_dy"] = out["dy"].abs().max().to(F32).view(1)
    return out


def _gelu_bwd(s):
    y = s["y"].to(F32)
    cdf = 0.5 * torch.special.erfc(y * -math.sqrt(0.5))
    dy = (s["dh"].to(F32) * (cdf + y * torch.exp(-0.5 * y * y) * (1.0 / math.sqrt(2.0 * math.pi)))).to(BF16)
    return dict(dy=dy, amax_dy=dy.abs().max().to(F32).view(1))


def _angles(s):
    """The angle of each row's pairs, in 64 bits: a far position times a frequency loses its turn in 32."""
    axes = _axes(s["case"])
    which = torch.repeat_interleave(torch.arange(len(axes), device="cuda"), torch.tensor(axes, device="cuda") // 2)
    return s["pos"].to(F64)[:, which] * s["freqs"]


def _rotate(x, cos, sin, c):
    """x [M, heads, hd] with its first `rot` values rotated, pair by pair."""
    rot = sum(_axes(c))
    cos, sin = cos[:, None], sin[:, None]
    if c["halves"]:
        a, b = x[..., : rot // 2], x[..., rot // 2: rot]
        return torch.cat([a * cos - b * sin, b * cos + a * sin, x[..., rot:]], -1)
    a, b = x[..., 0:rot:2], x[..., 1:rot:2]
    return torch.cat([torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2), x[..., rot:]], -1)


def _split(s):
    c = s["case"]
    x = s["qkv"].view(c["M"], -1, c["hd"])
    return x[:, : c["Hq"]], x[:, c["Hq"]: c["Hq"] + c["Hk"]], x[:, c["Hq"] + c["Hk"]:]


def _out_heads(t, c):
    """[M, heads, hd] as the attention takes it: [1, heads, M, hd], head by head in memory or token by token."""
    t = t.to(BF16).transpose(0, 1)
    return (t.contiguous() if c["head_major"] else t.transpose(0, 1).contiguous().transpose(0, 1))[None]


def _rope_fwd(s):
    c, out = s["case"], {}
    ang = _angles(s)
    cos, sin = ang.cos().to(F32), ang.sin().to(F32)
    q, k, v = _split(s)
    for name, t, w in (("q", q, s["w_q"]), ("k", k, s["w_k"])):
        t = t.to(F32)
        if c["norm"]:
            t = t * ((t * t).mean(-1, keepdim=True) + 1e-6).rsqrt() * w
        out[name] = _out_heads(_rotate(t, cos, sin, c), c)
    out["v"] = _out_heads(v, c)
    return out


def _rope_bwd(s):
    c, out = s["case"], {}
    ang = _angles(s)
    cos, sin = ang.cos().to(F32), ang.sin().to(F32)
    q, k, _ = _split(s)
    parts = []
    for name, t, w in (("q", q, s["w_q"]), ("k", k, s["w_k"])):
        d = _rotate(s["d" + name][0].transpose(0, 1).to(F32), cos, -sin, c)
        if c["norm"]:
            t = t.to(F32)
            rstd = ((t * t).mean(-1, keepdim=True) + 1e-6).rsqrt()
            that = t * rstd
            out["dw_" + name] = (d * that).sum((0, 1))
            d = d * w
            d = rstd * (d - that * (d * that).mean(-1, keepdim=True))
        parts.append(d)
    parts.append(s["dv"][0].transpose(0, 1).to(F32))
    out["dqkv"] = torch.cat(parts, 1).to(BF16).view(c["M"], -1)
    out["amax"] = out["dqkv"].abs().max().to(F32).view(1)
    return out


def _adamw(s):
    c, (b1, b2) = s["case"], s["betas"]
    s["step"] += 1
    t = s["step"].to(F64)
    c1, c2 = 1 - b1 ** t, 1 - b2 ** t  # in 64 bits: 1 - beta^t cancels
    g = s["g"].to(F32)
    m, v = (_decode_m(s["m"], s["m_scale"]), _decode_v(s["v"], s["v_scale"])) if c["bits"] == 8 else (s["m"], s["v"])
    m = m * b1 + g * (1 - b1)
    v = v * b2 + (g * (1 - b2)) * g
    p = s["p"] * (1 - s["lr"] * s["wd"])
    s["p"] = p - (s["lr"] / c1).to(F32) * (m / (v.sqrt() * c2.rsqrt().to(F32) + s["eps"]))
    s["p16"] = s["p"].to(BF16)
    if c["bits"] == 8:
        s["m"], s["m_scale"] = _encode_m(m)
        s["v"], s["v_scale"] = _encode_v(v)
        m, v = _decode_m(s["m"], s["m_scale"]), _decode_v(s["v"], s["v_scale"])
    else:
        s["m"], s["v"] = m, v
    return dict(p=s["p"], p16=s["p16"], m=m, v=v, step=s["step"])


_PLAIN = dict(norm_fwd=_norm_fwd, norm_bwd=_norm_bwd, gelu_bwd=_gelu_bwd, rope_fwd=_rope_fwd, rope_bwd=_rope_bwd,
              adamw=_adamw)


# ------------------------------------------------------------------ the framework's calls
def _own_norm(s):
    import bit_quantized_lora_b200 as ft
    c = s["case"]
    kinds = dict(none=ft.NORM_NONE, rms=ft.NORM_RMS, layer=ft.NORM_LAYER)
    return ft, ft.GatedNorm(pre=kinds[c["pre"]], post=kinds[c["post"]], alpha=s["alpha"], eps=s["eps"],
                            weight=s["weight"], bias=s["bias"], w_post=s["w_post"])


def _own_norm_fwd(s):
    ft, norm = _own_norm(s)
    amax = torch.zeros(1, device="cuda") if s["case"]["pre"] != "none" else None
    r, h, stats = ft.ft_gated_norm_fwd(norm, s["x"], s["y"], s["gate"], s["scale"], s["shift"], offsets=s["offsets"],
                                       amax_h=amax)
    return {k: v for k, v in dict(r=r if s["case"]["res"] else None, h=h, stats=stats, amax_h=amax).items()
            if v is not None}


def _own_norm_bwd(s):
    ft, norm = _own_norm(s)
    amax = torch.zeros(1, device="cuda") if s["case"]["res"] else None
    d = ft.ft_gated_norm_bwd(norm, s["dh"], s["r"], s["stats"], dr=s["dr"], y=s["y"], gate=s["gate"],
                             scale=s["scale"], shift=s["shift"], offsets=s["offsets"], amax_dy=amax)
    return {k: v for k, v in dict(dx=d.dx, dy=d.dy, dgate=d.dgate, dscale=d.dscale, dshift=d.dshift,
                                  dweight=d.dweight, dbias=d.dbias, dw_post=d.dw_post, amax_dy=amax).items()
            if v is not None}


def _own_gelu_bwd(s):
    import bit_quantized_lora_b200 as ft
    amax = torch.zeros(1, device="cuda")
    return dict(dy=ft.ft_gelu_bwd_bf16(s["y"], s["dh"], amax_dy=amax), amax_dy=amax)


def _own_rope(s):
    import bit_quantized_lora_b200 as ft
    c = s["case"]
    return ft, ft.Rope(heads=c["Hq"], kv_heads=c["Hk"], head_dim=c["hd"], axes=tuple(_axes(c)), freqs=s["freqs"],
                       layout=ft.ROPE_HALVES if c["halves"] else ft.ROPE_PAIRS, norm=c["norm"], w_q=s["w_q"],
                       w_k=s["w_k"], eps=1e-6)


def _own_rope_fwd(s):
    ft, rope = _own_rope(s)
    q, k, v = ft.ft_qk_rope_fwd(rope, s["qkv"], s["pos"], head_major=s["case"]["head_major"])
    return dict(q=q, k=k, v=v)


def _own_rope_bwd(s):
    ft, rope = _own_rope(s)
    amax = torch.zeros(1, device="cuda")
    dqkv, dw_q, dw_k = ft.ft_qk_rope_bwd(rope, s["dq"], s["dk"], s["dv"], s["pos"], qkv=s["qkv"], amax=amax)
    return {k: v for k, v in dict(dqkv=dqkv, dw_q=dw_q, dw_k=dw_k, amax=amax).items() if v is not None}


def _own_adamw(s):
    s["opt"].step()
    m, v = s["opt"].state_values()
    return dict(p=s["opt"].master, p16=s["p16"], m=m, v=v, step=s["opt"].step_count)


_OWN = dict(norm_fwd=_own_norm_fwd, norm_bwd=_own_norm_bwd, gelu_bwd=_own_gelu_bwd, rope_fwd=_own_rope_fwd,
            rope_bwd=_own_rope_bwd, adamw=_own_adamw)


def run(state):
    return (_OWN if own else _PLAIN)[state["case"]["op"]](state)


# ------------------------------------------------------------------ work
def work(case):
    c, op = case, case["op"]
    if op in ("norm_fwd", "norm_bwd"):
        M, D, x, p = c["M"], c["D"], 4 if c["x32"] else 2, 4 if c["p32"] else 2
        pre, post = c["pre"] != "none", c["post"] != "none"
        vectors = (c["B"] * (int(c["res"]) + 2 * int(pre)) if c["mod"] else 0) + (2 * c["weights"])
        if op == "norm_fwd":
            bytes_ = M * D * (x + (2 + x if c["res"] else 0) + (2 if pre else 0)) + 16 * M + vectors * D * p
            return dict(bytes=bytes_, flops=M * D * (3 * c["res"] + 8 * pre + 6 * post))
        bytes_ = M * D * (2 * x + (x + 2 if pre else 0) + (4 if c["res"] else 0)) + 16 * M + vectors * D * (p + 4)
        return dict(bytes=bytes_, flops=M * D * (6 * c["res"] + 14 * pre + 12 * post))
    if op == "gelu_bwd":
        return dict(bytes=6 * c["n"], flops=30 * c["n"])
    if op in ("rope_fwd", "rope_bwd"):
        qk, v = c["M"] * (c["Hq"] + c["Hk"]) * c["hd"], c["M"] * c["Hk"] * c["hd"]
        bytes_ = 4 * (qk + v) + 4 * c["M"] * len(_axes(c))
        if op == "rope_bwd" and c["norm"]:
            bytes_ += 2 * qk
        return dict(bytes=bytes_, flops=qk * (4 + (6 if c["norm"] else 0)))
    n = sum(_sizes(c))
    state = 16 if c["bits"] == 32 else 4 + 16 / BLOCK
    return dict(bytes=n * (10 + (2 if c["g16"] else 4) + state), flops=n * (18 if c["bits"] == 32 else 40))


# ------------------------------------------------------------------ in 64 bits
def _x64(t):
    return None if t is None else t.double()


def _exact_norm(s, backward):
    c, B, M = s["case"], s["case"]["B"], s["case"]["M"]
    ends = [M * (k + 1) // B for k in range(B)] if s["offsets"] is None else s["offsets"].tolist()[1:]
    x, y = _x64(s["r"] if backward else s["x"]), _x64(s["y"])
    gate, scale, shift = _x64(s["gate"]), _x64(s["scale"]), _x64(s["shift"])
    ones = torch.ones(c["D"], dtype=F64, device="cuda")
    w, wp = ones if s["weight"] is None else _x64(s["weight"]), ones if s["w_post"] is None else _x64(s["w_post"])
    bias = 0.0 if s["bias"] is None else _x64(s["bias"])
    rows = []
    begin = 0
    sums = {k: [] for k in ("dgate", "dscale", "dshift", "dweight", "dbias", "dw_post")}
    for k, end in enumerate(ends):  # one sample after another
        i = slice(begin, end)
        begin = end
        g = ones if gate is None else gate[k]
        a, t = (ones if scale is None else 1 + scale[k]), (0.0 if shift is None else shift[k])
        o = {}
        if backward:
            st = s["stats"][i].double()
            d = _x64(s["dr"][i])
            if c["pre"] != "none":
                dh, xh = _x64(s["dh"][i]), (x[i] - st[:, :1]) * st[:, 1:2]
                z = dh * a * w
                d = d + st[:, 1:2] * (z - xh * (z * xh).mean(1, True) - (z.mean(1, True) if c["pre"] == "layer" else 0))
                sums["dscale"].append((dh * (xh * w + bias)).sum(0))
                sums["dshift"].append(dh.sum(0))
                sums["dweight"].append((dh * a * xh).sum(0))
                sums["dbias"].append((dh * a).sum(0))
            o["dx"] = d
            if y is not None:
                yh = y[i] if c["post"] == "none" else (y[i] - st[:, 2:3]) * st[:, 3:4]
                sums["dgate"].append((d * yh * wp).sum(0) * s["alpha"])
                z = s["alpha"] * g * d
                sums["dw_post"].append((z * yh).sum(0))
                z = z * wp
                if c["post"] != "none":
                    z = st[:, 3:4] * (z - yh * (z * yh).mean(1, True) - (z.mean(1, True) if c["post"] == "layer" else 0))
                o["dy"] = z
        else:
            r = x[i]
            m1, r1 = torch.zeros(len(r), 1, dtype=F64, device="cuda"), torch.ones(len(r), 1, dtype=F64, device="cuda")
            m0, r0 = m1, r1
            if y is not None:
                u = y[i]
                if c["post"] != "none":
                    m1 = u.mean(1, True) if c["post"] == "layer" else m1
                    r1 = 1 / torch.sqrt((u - m1).square().mean(1, True) + s["eps"])
                    u = (u - m1) * r1 * wp
                r = r + s["alpha"] * g * u
                o["r"] = r
                r = r.to(s["x"].dtype).double()  # the norm reads the stream as it is stored
            if c["pre"] != "none":
                m0 = r.mean(1, True) if c["pre"] == "layer" else m0
                r0 = 1 / torch.sqrt((r - m0).square().mean(1, True) + s["eps"])
                o["h"] = ((r - m0) * r0 * w + bias) * a + t
            o["stats"] = torch.cat([m0, r0, m1, r1], 1)
        rows.append(o)
    out = {k: torch.cat([o[k] for o in rows]) for k in rows[0]}
    if not backward:
        if "h" in out:
            out["amax_h"] = out["h"].to(BF16).abs().max().double().view(1)
        return out
    given = dict(dgate=gate, dscale=scale, dshift=shift)
    out.update({k: torch.stack(sums[k]) for k, v in given.items() if v is not None})
    given = dict(dweight=s["weight"], dbias=s["bias"], dw_post=s["w_post"])
    out.update({k: torch.stack(sums[k]).sum(0) for k, v in given.items() if v is not None})
    if "dy" in out:
        out["amax_dy"] = out["dy"].to(BF16).abs().max().double().view(1)
    return out


def _exact_rope(s, backward):
    """The rotation as a complex product."""
    c = s["case"]
    M, hd, axes, rot = c["M"], c["hd"], _axes(c), sum(_axes(c))
    p = s["pos"].double()
    ang, at = [], 0
    for a, width in enumerate(axes):
        ang.append(p[:, a:a + 1] * s["freqs"][at:at + width // 2])
        at += width // 2
    turn = torch.polar(torch.ones(M, rot // 2, dtype=F64, device="cuda"), torch.cat(ang, 1) * (-1 if backward else 1))

    def spun(x):
        pair = x[..., :rot].unflatten(-1, (2, rot // 2)).transpose(-1, -2) if c["halves"] else \
            x[..., :rot].unflatten(-1, (rot // 2, 2))
        z = torch.view_as_real(torch.view_as_complex(pair.contiguous()) * turn[:, None])
        z = z.transpose(-1, -2).flatten(-2) if c["halves"] else z.flatten(-2)
        return torch.cat([z, x[..., rot:]], -1)

    x = s["qkv"].double().view(M, -1, hd)
    parts = dict(q=x[:, :c["Hq"]], k=x[:, c["Hq"]:c["Hq"] + c["Hk"]], v=x[:, c["Hq"] + c["Hk"]:])
    out, grads = {}, []
    for n, t in parts.items():
        w, norm = s.get("w_" + n), c["norm"] and n != "v"
        rstd = 1 / torch.sqrt(t.square().mean(-1, True) + 1e-6) if norm else None
        if not backward:
            z = t * rstd * w.double() if norm else t
            out[n] = (spun(z) if n != "v" else z).transpose(0, 1)[None]
            continue
        d = s["d" + n][0].transpose(0, 1).double()
        d = spun(d) if n != "v" else d
        if norm:
            out["dw_" + n] = (d * t * rstd).sum((0, 1))
            d = d * w.double() * rstd
            d = d - t * rstd.square() * (d * t).mean(-1, True)
        grads.append(d)
    if backward:
        out["dqkv"] = torch.cat(grads, 1).view(M, -1)
        out["amax"] = out["dqkv"].to(BF16).abs().max().double().view(1)
    return out


def _exact_adamw(s):
    """32-bit states: the update in 64 bits.  8-bit states are defined by steps that are each rounded to 32 bits, so
    that their codes are the same everywhere; each step is computed in 64 bits and rounded."""
    c, (b1, b2), t = s["case"], s["betas"], s["case"]["step"] + 1
    g, p = s["g"].double(), s["p"].double()
    r = (lambda z: z.float().double()) if c["bits"] == 8 else (lambda z: z)
    k = (lambda z: torch.tensor(z, dtype=F32, device="cuda").double()) if c["bits"] == 8 else (lambda z: z)

    def m_of(code, top):
        code = code.double().view(-1, BLOCK)
        return r(r(code * code.abs() * r(1 / k(16129.0))) * top.double()[:, None]).view(-1)

    def v_of(code, top):
        code = code.double().view(-1, BLOCK)
        q = r(code * code * r(1 / k(65025.0)))
        return r(r(q * q) * top.double()[:, None]).view(-1)

    m, v = (m_of(s["m"], s["m_scale"]), v_of(s["v"], s["v_scale"])) if c["bits"] == 8 else (s["m"].double(), s["v"].double())
    m = r(r(m * k(b1)) + r(g * k(1 - b1)))
    v = r(r(v * k(b2)) + r(r(g * k(1 - b2)) * g))
    p = p * (1 - s["lr"] * s["wd"]) - s["lr"] / (1 - b1 ** t) * m / (torch.sqrt(v / (1 - b2 ** t)) + s["eps"])
    if c["bits"] == 8:
        top = m.view(-1, BLOCK).abs().amax(1, True)
        q = r(m.view(-1, BLOCK).abs() * torch.where(top >= 2.0 ** -126, r(1 / top), torch.zeros_like(top)))
        m = m_of(torch.round(r(r(q.sqrt()) * 127)).mul(m.view(-1, BLOCK).sign()).view(-1), top.view(-1))
        top = v.view(-1, BLOCK).amax(1, True)
        q = r(v.view(-1, BLOCK) * torch.where(top >= 2.0 ** -126, r(1 / top), torch.zeros_like(top)))
        v = v_of(torch.round(r(r(r(q.sqrt()).sqrt()) * 255)).view(-1), top.view(-1))
    return dict(p=p, p16=p, m=m, v=v, step=s["step"] + 1)


def exact(case, seed):
    s, op = prepare(case, seed), case["op"]
    if op in ("norm_fwd", "norm_bwd"):
        return _exact_norm(s, op == "norm_bwd")
    if op in ("rope_fwd", "rope_bwd"):
        return _exact_rope(s, op == "rope_bwd")
    if op == "adamw":
        return _exact_adamw(s)
    y = s["y"].double()
    slope = 0.5 * torch.special.erfc(-y / math.sqrt(2.0)) + y * torch.exp(-0.5 * y * y) / math.sqrt(2.0 * math.pi)
    dy = s["dh"].double() * slope
    return dict(dy=dy, amax_dy=dy.to(BF16).abs().max().double().view(1))
