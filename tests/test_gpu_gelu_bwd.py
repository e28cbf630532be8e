"""GELU's backward against the formula in 64 bits.

The slope Phi(y) + y phi(y) in FP32: erfc's argument is rounded once, which
moves erfc by 2 t^2 = y^2 of its value per 2^-24; erfc and exp add a few ulp,
exp's argument -y^2 / 2 another y^2 / 2 of 2^-24.  16 roundings (1 + y^2) of
the two terms' magnitudes bound it.
"""
import pytest
import torch

import bit_quantized_lora_b200 as ft
import block_ref as R

pytestmark = pytest.mark.gpu


def check(y, dh, dy):
    yd, dd = y.double(), dh.double()
    phi = torch.exp(-0.5 * yd * yd) / (2 * torch.pi) ** 0.5
    cdf = 0.5 * torch.special.erfc(-yd / 2 ** 0.5)
    # below 2^-126 the terms are FP32 subnormals: 2^-149 of spacing each
    slack = dd.abs() * (16 * R.U32 * (1 + yd * yd) * (cdf + yd.abs() * phi) + 2.0 ** -145)
    R.check_rounded(dy, dd * R.gelu_slope64(yd), slack)


def test_every_finite_value():
    u = torch.arange(65536, dtype=torch.int32).to(torch.int16)
    y = u.view(torch.bfloat16).cuda()
    y = y[y.isfinite()]
    y = torch.cat([y, torch.zeros(-len(y) % 8, dtype=y.dtype, device="cuda")])
    for v in (1.0, -0.3046875):
        dh = torch.full_like(y, v)
        check(y, dh, ft.ft_gelu_bwd_bf16(y, dh))


@pytest.mark.parametrize("n", [0, 8, 16, 2040, 2048, 2056, 100_000, 3_000_008])
def test_sizes_and_amax(n):
    g = torch.Generator(device="cuda")
    g.manual_seed(n)
    y = (torch.randn(n, generator=g, device="cuda") * 2).bfloat16()
    dh = (torch.randn(n, generator=g, device="cuda") * 0.01).bfloat16()
    amax = torch.zeros(1, device="cuda")
    dy = ft.ft_gelu_bwd_bf16(y, dh, amax_dy=amax)
    check(y, dh, dy)
    assert float(amax) == (float(dy.float().abs().max()) if n else 0.0)
    again = ft.ft_gelu_bwd_bf16(y, dh)
    assert torch.equal(again, dy)
    if n:
        assert torch.equal(ft.ft_gelu_bwd_bf16(y, dh, out=dh), dy)  # in place


def test_values_beyond_the_finite():
    inf, nan = float("inf"), float("nan")
    y = torch.tensor([inf, -inf, nan, 1.0, 1.0, 200.0, -200.0, 0.0], device="cuda").bfloat16()
    dh = torch.tensor([2.0, 2.0, 2.0, inf, nan, 3.0, 3.0, 4.0], device="cuda").bfloat16()
    amax = torch.zeros(1, device="cuda")
    dy = ft.ft_gelu_bwd_bf16(y, dh, amax_dy=amax)
    assert dy.tolist()[:2] == [2.0, 0.0] and dy.tolist()[3] == inf and dy.tolist()[5:] == [3.0, 0.0, 2.0]
    assert bool(dy[2].isnan()) and bool(dy[4].isnan()) and float(amax) == inf


def test_past_two_to_the_31_bytes():
    n = (1 << 30) + 4096
    y = torch.zeros(n, dtype=torch.bfloat16, device="cuda")
    y[-8:] = 1.0
    dh = torch.ones(n, dtype=torch.bfloat16, device="cuda")
    dy = ft.ft_gelu_bwd_bf16(y, dh)
    check(y[-16:], dh[-16:], dy[-16:])
    assert bool((dy[:-8] == 0.5).all())


def test_graph_and_stream():
    y, dh = torch.randn(4096, device="cuda").bfloat16(), torch.randn(4096, device="cuda").bfloat16()
    want = ft.ft_gelu_bwd_bf16(y, dh)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = ft.ft_gelu_bwd_bf16(y, dh, stream=s)
    s.synchronize()
    assert torch.equal(got, want)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = ft.ft_gelu_bwd_bf16(y, dh)
    y.mul_(-1)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, ft.ft_gelu_bwd_bf16(y, dh))


def test_refusals():
    y = torch.zeros(4, 16, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(TypeError):
        ft.ft_gelu_bwd_bf16(y, y.float())
    with pytest.raises(ValueError):
        ft.ft_gelu_bwd_bf16(y, y[:2])
    with pytest.raises(ValueError):
        ft.ft_gelu_bwd_bf16(y.t(), y.t())
    with pytest.raises(ft.FtError):
        ft.ft_gelu_bwd_bf16(y.view(-1)[:12], y.view(-1)[:12])
