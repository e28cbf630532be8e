"""Where the operators around the linears keep their sums in a workspace that
they may share with the linears: behind the words that those keep in it."""
import ctypes

from bit_quantized_lora_b200 import _lib


def words():
    """Bytes of the linears' words: what ft_workspace_qact names first lies
    right behind them, whatever the shape."""
    L = _lib.load(build_if_missing=True)
    at = set()
    for shape in ((0, 0, 0, 0, 0), (1, 256, 256, 0, 0), (4608, 1024, 4096, 64, 64)):
        out = [ctypes.c_size_t() for _ in range(3)]
        assert L.ft_workspace_qact(*shape, *(ctypes.byref(c) for c in out)) == 0
        at.add(min(c.value for c in out))
    assert len(at) == 1
    return at.pop()


def test_the_sums_lie_behind_the_words():
    L = _lib.load(build_if_missing=True)
    w = words()
    assert w >= 256 + 8 * 1024 + 16 * 8192 + 256
    # without rows: three sums per sample, of the one block's share and of the sample
    at = {L.ft_gated_norm_workspace_bytes(0, D, B) - 2 * B * 3 * D * 4 for D in (8, 1024, 8192) for B in (1, 5)}
    # as many sums as values of a head, times the same
    a, b = (L.ft_qk_rope_workspace_bytes(100, hd) for hd in (64, 128))
    at.add(a - (b - a))
    assert len(at) == 1 and w <= min(at) < w + 4096 and min(at) % 256 == 0
