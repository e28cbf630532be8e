"""One workspace for the linears and the operators around them, used in turn:
the operators' sums stay out of the words that the linears keep in it."""
import pytest
import torch

import bit_quantized_lora_b200 as ft

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16
M, N, K = 300, 512, 256


def inputs(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return lambda *s, std=1.0: (torch.randn(*s, generator=g, device="cuda") * std).to(BF16)


def made(seed=1):
    """The two backward calls that keep sums in a workspace, as functions of
    it."""
    rnd = inputs(seed)
    norm = ft.GatedNorm(pre=ft.NORM_LAYER, post=ft.NORM_RMS, weight=rnd(K), bias=rnd(K), w_post=rnd(K))
    x, y, dh, dr, mod = rnd(M, K), rnd(M, K), rnd(M, K), rnd(M, K), rnd(2, 3 * K)
    gate, scale, shift = mod[:, :K], mod[:, K:2 * K], mod[:, 2 * K:]
    r, h, stats = ft.ft_gated_norm_fwd(norm, x, y, gate, scale, shift)
    rope = ft.Rope(6, 3, 64, (32, 32), ft.rope_freqs((32, 32)), norm=True, w_q=rnd(64), w_k=rnd(64))
    pos = torch.arange(2 * M, device="cuda", dtype=torch.int32).view(M, 2)
    dq, dk, dv = (rnd(1, n, M, 64) for n in (6, 3, 3))
    qkv = rnd(M, rope.width)

    def run(ws):
        d = ft.ft_gated_norm_bwd(norm, dh, r, stats, dr=dr, y=y, gate=gate, scale=scale, shift=shift, ws=ws)
        out = ft.ft_qk_rope_bwd(rope, dq, dk, dv, pos, qkv=qkv, ws=ws)
        return [d.dx, d.dy, d.dgate, d.dscale, d.dshift, d.dweight, d.dbias, d.dw_post, *out]

    return run


def linears(ws, layer, seed=2):
    rnd = inputs(seed)
    X, dY = rnd(M, K), rnd(M, N, std=0.1)
    Y, P = ft.ft_linear_fwd(layer, X, ws=ws)
    return [Y, P, *ft.ft_linear_bwd(layer, dY, X, P, ws=ws)]


def test_the_words_are_left_alone():
    words = ft.ft_workspace_qact(M, N, K, 16, 16)[2]  # what follows the words
    ws = ft.Workspace()
    buf = ws.get(1 << 24, torch.device("cuda", 0))
    buf.fill_(0xA5)
    operators = made()
    want = operators(None)
    got = operators(ws)
    assert ws.buf is buf
    assert bool((buf[:words] == 0xA5).all()) and not bool((buf[words:] == 0xA5).all())
    assert all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.parametrize("rows", [300, 20_000])
def test_linears_and_operators_in_turn(rows, monkeypatch):
    """Bits as with a workspace of each one's own; 20000 rows take the
    streaming quantizer, whose amax pass has a word of its own."""
    monkeypatch.setitem(globals(), "M", rows)
    rnd = inputs(0)
    layer = ft.prepare_layer(W_res=rnd(N, K, std=K ** -0.5), U=rnd(K, 16, std=0.1), V=rnd(N, 16, std=0.1),
                             A=rnd(K, 16, std=0.1), B=rnd(N, 16, std=0.1), s=0.5)
    operators = made()
    want_l, want_o = linears(ft.Workspace(), layer), operators(ft.Workspace())
    x = inputs(3)(rows, K)
    want_q = ft.ft_quantize(x, ws=ft.Workspace())
    ws = ft.Workspace()
    ws.get(max(ft.ft_workspace_bytes(rows, N, K, 16, 16), 1 << 22), torch.device("cuda", 0))
    for _ in range(2):
        for got, want in ((linears(ws, layer), want_l), (operators(ws), want_o), (linears(ws, layer), want_l)):
            assert all(torch.equal(a, b) for a, b in zip(got, want))
        q = ft.ft_quantize(x, ws=ws)
        assert torch.equal(q.codes, want_q.codes) and torch.equal(q.scales, want_q.scales)
        assert torch.equal(q.tscale, want_q.tscale)
        assert all(torch.equal(a, b) for a, b in zip(operators(ws), want_o))
    torch.cuda.synchronize()
    assert ft.ft_device_error() == 0


def test_a_captured_call_owns_its_scratch():
    """A workspace may grow, and so give its memory back, while a graph that
    was captured with it lives: the graph writes neither there nor to what
    lies there afterwards."""
    operators, ws = made(), ft.Workspace()
    want = operators(None)
    operators(ws)  # sized by a call outside the graph
    size = ws.buf.numel()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = operators(ws)
    ws.buf.fill_(0xA5)
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(out, want)) and bool((ws.buf == 0xA5).all())
    ws.get(8 * size, torch.device("cuda", 0))
    others = [torch.full((size,), 7, dtype=torch.uint8, device="cuda") for _ in range(4)]
    for t in out:
        t.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(out, want)) and not ws.buf.any()
    assert all(bool((t == 7).all()) for t in others)
